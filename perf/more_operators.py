"""The operators of a feed-forward sub-layer of experts on real sizes: the RMS
norm with the residual's addition, the router with the sort of its choices, the
way of the tokens to their experts and back, and the experts' gated products.

Each is here in two forms on the same inputs: a plain one in elementary torch
operations, and the call a user makes of this package (``own = True``).
``listed()`` names the cases, ``draw(rng)`` makes another of the same ranges,
``prepare`` makes the inputs, ``run`` does one pass, ``work`` says what a pass
cannot do without and ``exact`` what it should give.

The sizes are the package's own layers (tokens x 256 of the small and the large
system, 1024 <-> 4096 of the wide model) with 8 to 64 experts, one token of the
same layers, and ragged ones.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
GROUP = 128                    # columns that share a scale of the 8-bit output
LARGEST_ROWS = 552960          # tokens of the large system
NORM_LIMIT = LARGEST_ROWS * 256
ROUTE_LIMIT = LARGEST_ROWS * 16
EXCHANGE_LIMIT = LARGEST_ROWS * 2 * 256
FLOP_LIMIT = 6 * LARGEST_ROWS * 2 * 256 * 512
WEIGHT_LIMIT = 1 << 27         # floats of all experts' weights


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # RMS norm of M rows of width N, after the residual's addition.
        # one token of the wide model: launch latency
        dict(name="rms_fwd_1x1024", op="rms_norm", kind="fwd", M=1, N=1024, residual=True),
        # a training step's norm in the small system (192 atoms x 32 neighbours)
        dict(name="rms_train_6144x256", op="rms_norm", kind="train", M=6144, N=256, residual=True),
        # a row count and a width that nothing divides, output in 8 bits
        dict(name="rms_quant_4099x1001", op="rms_norm", kind="quant", M=4099, N=1001, residual=True),
        # the large system (17,280 atoms x 32 neighbours): memory bound
        dict(name="rms_train_552960x256", op="rms_norm", kind="train", M=LARGEST_ROWS, N=256, residual=True),
        # router: the k largest of E logits, their weights, the choices sorted by expert.
        # one token: launch latency
        dict(name="route_1x8_k2", op="route", train=False, M=1, E=8, k=2, over="chosen", masked=False),
        # the large system, forward and backward: memory bound
        dict(name="route_train_552960x16_k2", op="route", train=True, M=LARGEST_ROWS, E=16, k=2, over="chosen",
             masked=False),
        # tokens to their experts and back, with gradients.
        # ragged width and count, padded tokens that go nowhere
        dict(name="exchange_train_6145x333_E7_k3", op="exchange", train=True, M=6145, N=333, E=7, k=3, masked=True),
        # the large system
        dict(name="exchange_train_552960x256_E16_k2", op="exchange", train=True, M=LARGEST_ROWS, N=256, E=16, k=2,
             masked=False),
        # the experts' gated blocks on sorted rows: M tokens, k experts each.
        # one token of the wide model: reads two experts' weights once
        dict(name="experts_fwd_1x1024x4096_E8_k2", op="experts", train=False, M=1, K=1024, F=4096, E=8, k=2,
             act="silu", mode="bf16x9"),
        # a ragged training step in the two-component mode
        dict(name="experts_train_777x260x700_E5_k3_tf32x3", op="experts", train=True, M=777, K=260, F=700, E=5, k=3,
             act="gelu_tanh", mode="tf32x3"),
        # a training step of the small system
        dict(name="experts_train_6144x256x1024_E8_k2", op="experts", train=True, M=6144, K=256, F=1024, E=8, k=2,
             act="silu", mode="bf16x9"),
        # forces on the large system need the forward over every token
        dict(name="experts_fwd_552960x256x512_E16_k2", op="experts", train=False, M=LARGEST_ROWS, K=256, F=512, E=16,
             k=2, act="silu", mode="bf16x9"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _width(rng, lo, hi):
    """A layer width: mostly a multiple of 32, sometimes of 4, sometimes odd."""
    w = _log_uniform(rng, lo, hi)
    kind = rng.random()
    if kind < 0.55:
        return max(lo, w // 32 * 32)
    if kind < 0.85:
        return max(lo, w // 4 * 4)
    return w | 1


def draw(rng):
    op = rng.choice(["rms_norm", "route", "exchange", "experts"])
    if op == "rms_norm":
        N = _width(rng, 16, 8192)
        M = _log_uniform(rng, 1, min(LARGEST_ROWS, NORM_LIMIT // N))
        return dict(op=op, kind=rng.choice(["fwd", "train", "train", "quant"]), M=M, N=N, residual=rng.random() < 0.7)
    if op == "route":
        E = _log_uniform(rng, 2, 256)
        k = rng.randint(1, min(E, 8))
        M = _log_uniform(rng, 1, min(LARGEST_ROWS, ROUTE_LIMIT // E, 2 * ROUTE_LIMIT // (E * k)))
        return dict(op=op, train=rng.random() < 0.5, M=M, E=E, k=k, over=rng.choice(["chosen", "all"]),
                    masked=rng.random() < 0.4)
    E = _log_uniform(rng, 2, 64)
    k = rng.randint(1, min(E, 8))
    if op == "exchange":
        N = _width(rng, 16, 4096)
        M = _log_uniform(rng, 1, min(LARGEST_ROWS, EXCHANGE_LIMIT // (k * N)))
        return dict(op=op, train=rng.random() < 0.6, M=M, N=N, E=E, k=k, masked=rng.random() < 0.4)
    train = rng.random() < 0.6
    K = _width(rng, 64, 2048)
    F = _width(rng, 64, min(4096, WEIGHT_LIMIT // (3 * E * K)))
    per_token = 6 * K * F * k * (3 if train else 1)
    # one token to the most that cost no more than the largest listed case
    M = _log_uniform(rng, 1, min(LARGEST_ROWS, 1 << 20, FLOP_LIMIT // per_token // 2, EXCHANGE_LIMIT // (k * max(K, F))))
    return dict(op=op, train=train, M=max(1, M), K=K, F=F, E=E, k=k, act=rng.choice(["gelu", "gelu_tanh", "silu"]),
                mode=rng.choice(["bf16x9", "tf32x3"]))


# ----------------------------------------------------------------- inputs ---
def _logits(normal, M, E, masked):
    """A router's logits: some experts are liked better than others.  Masked: the
    last tokens are padding, and single experts are closed to single tokens."""
    logits = normal(M, E).add_(normal(E, std=0.5))
    if masked:
        logits.masked_fill_(normal(M, E) > 1.6, -math.inf)
        logits[M - M // 8:] = -math.inf
    return logits


def _sorted(experts, E):
    """(slots, sources, offsets) of the choices sorted by expert, in order of the
    tokens: where each choice goes, which choice each row is, where each expert's
    rows start.  A choice of -1 goes nowhere (slot -1), and the rows behind the
    last expert's have no source (-1)."""
    flat = experts.reshape(-1).long()
    T = flat.numel()
    hot = flat[None, :] == torch.arange(E, device=flat.device)[:, None]
    rank = torch.cumsum(hot, 1)                                  # int64
    offsets = torch.zeros(E + 1, device=flat.device, dtype=torch.int64)
    offsets[1:] = torch.cumsum(rank[:, -1], 0)
    sent = flat >= 0
    at = flat.clamp(min=0)
    slots = offsets[at] + rank.gather(0, at[None, :])[0] - 1
    slots = torch.where(sent, slots, torch.full_like(slots, -1))
    sources = torch.full((T + 1,), -1, device=flat.device, dtype=torch.int64)
    sources[torch.where(sent, slots, torch.full_like(slots, T))] = torch.arange(T, device=flat.device)
    sources[T] = -1
    return slots.reshape(experts.shape).int(), sources[:T].int(), offsets.int()


def _choose(logits, k):
    """The k largest logits of each row, the lowest index first among equals:
    (experts, values); -1 and -inf where a row has no more."""
    left = logits.clone()
    index = torch.arange(logits.shape[1], device=logits.device)[None, :].expand_as(left)
    experts, values = [], []
    for _ in range(k):
        v = left.amax(1, keepdim=True)
        e = torch.where(left == v, index, torch.full_like(index, logits.shape[1])).amin(1, keepdim=True)
        experts.append(torch.where(v == -math.inf, torch.full_like(e, -1), e))
        values.append(v)
        left.scatter_(1, e, -math.inf)
    return torch.cat(experts, 1).int(), torch.cat(values, 1)


def _choice_weights(values, logits, over):
    """Softmax of the chosen values over themselves or over the whole row."""
    top = values[:, :1]
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(values - top)
    total = e.sum(1, keepdim=True) if over == "chosen" else torch.exp(logits - top).sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(mean, std, generator=g)

    s = dict(case=case)
    M = case["M"]
    if case["op"] == "rms_norm":
        N = case["N"]
        # a residual stream: channels of different offset and spread
        s["X"] = normal(M, N).mul_(normal(N, std=0.5).exp_()).add_(normal(N, std=0.3))
        s["R"] = normal(M, N) if case["residual"] else None
        s["w"] = normal(N, std=0.1, mean=1.0)
        if case["kind"] == "train":
            s["dY"] = normal(M, N)
            s["add"] = normal(M, N) if case["residual"] else None    # what reaches the stream behind the norm
        return s
    E, k = case["E"], case["k"]
    s["logits"] = _logits(normal, M, E, case.get("masked", False))
    if case["op"] == "route":
        if case["train"]:
            s["dweights"] = normal(M, k)
        return s
    experts, values = _choose(s["logits"], k)
    s["weights"] = _choice_weights(values, s["logits"], "chosen")
    s["experts"] = experts
    s["slots"], s["sources"], s["offsets"] = _sorted(experts, E)
    T = M * k
    if case["op"] == "exchange":
        N = case["N"]
        s["X"], s["Ys"], s["R"] = normal(M, N), normal(T, N), normal(M, N)
        if case["train"]:
            s["dY"], s["dXs"] = normal(M, N), normal(T, N)
    else:
        K, F = case["K"], case["F"]
        s["Xs"] = normal(T, K)
        s["Win"] = normal(E, 2 * F, K, std=K ** -0.5)      # an expert's gate rows, then its up rows
        s["Wout"] = normal(E, K, F, std=F ** -0.5)
        if case["train"]:
            s["dYs"] = normal(T, K)
    return s


# -------------------------------------------------------------- plain form ---
_C = math.sqrt(2.0 / math.pi)


def _act(name, z):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (0.5 * _C)
    t = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * (_C * (1.0 + 3 * 0.044715 * z * z))


def _dequantised(Q, scales):
    return Q.to(torch.float32) * scales.repeat_interleave(GROUP, 1)[:, :Q.shape[1]]


def _quantised(Y):
    """(Q, scales): each group's scale is the smallest power of two with the
    group's largest magnitude within 448 of it."""
    M, N = Y.shape
    G = (N + GROUP - 1) // GROUP
    padded = torch.zeros((M, G * GROUP), device=Y.device, dtype=Y.dtype)
    padded[:, :N] = Y
    top = padded.reshape(M, G, GROUP).abs().amax(2)
    mantissa, exponent = torch.frexp(top)                  # top = mantissa 2^exponent, 448 = 0.875 2^9
    exponent = torch.where(mantissa > 0.875, exponent - 8, exponent - 9)
    exponent = torch.where(top == 0, torch.full_like(exponent, -126), exponent).clamp(min=-126)
    scales = torch.ldexp(torch.ones_like(top), exponent)
    return (padded.reshape(M, G, GROUP) / scales[:, :, None]).reshape(M, -1)[:, :N].to(torch.float8_e4m3fn), scales


def _rows_at(A, index):
    """The rows of A at `index`, zeros where it is -1."""
    return torch.where((index >= 0)[..., None], A[index.long().clamp(min=0)], torch.zeros((), device=A.device))


def _plain(s):
    c = s["case"]
    if c["op"] == "rms_norm":
        S = s["X"] if s["R"] is None else s["X"] + s["R"]
        rstd = 1.0 / torch.sqrt((S * S).mean(1, keepdim=True) + EPS)
        h = S * rstd
        Y = h * s["w"]
        stream = () if s["R"] is None else (S,)
        if c["kind"] == "quant":
            return (_dequantised(*_quantised(Y)),) + stream
        if c["kind"] == "fwd":
            return (Y,) + stream
        gr = s["dY"] * s["w"]
        dX = rstd * (gr - h * (gr * h).mean(1, keepdim=True))
        if s["add"] is not None:
            dX = dX + s["add"]
        return (Y,) + stream + (dX, (s["dY"] * h).sum(0))
    if c["op"] == "route":
        logits = s["logits"]
        experts, values = _choose(logits, c["k"])
        weights = _choice_weights(values, logits, c["over"])
        out = (experts, weights) + _sorted(experts, c["E"])
        if not c["train"]:
            return out
        dw = s["dweights"]
        inner = (weights * dw).sum(1, keepdim=True)
        if c["over"] == "chosen":
            part, base = weights * (dw - inner), torch.zeros_like(logits)
        else:
            top = values[:, :1]
            e = torch.exp(logits - torch.where(top == -math.inf, torch.zeros_like(top), top))
            total = e.sum(1, keepdim=True)
            base = torch.where(total > 0, -e / total * inner, torch.zeros_like(e))
            part = weights * dw
        wide = torch.cat([base, torch.zeros_like(base[:, :1])], 1)  # a column for the choices that go nowhere
        wide.scatter_add_(1, torch.where(experts < 0, torch.full_like(experts, c["E"]), experts).long(), part)
        return out + (wide[:, :c["E"]],)
    if c["op"] == "exchange":
        slots, sources, weights, k = s["slots"], s["sources"], s["weights"], c["k"]
        token = torch.where(sources >= 0, sources // k, sources)
        Xs = _rows_at(s["X"], token)
        Y = s["R"] + (_rows_at(s["Ys"], slots) * weights[:, :, None]).sum(1)
        if not c["train"]:
            return Xs, Y
        w = torch.where(sources >= 0, weights.reshape(-1)[sources.long().clamp(min=0)], torch.zeros((), device=Y.device))
        dYs = _rows_at(s["dY"], token) * w[:, None]
        dweights = (_rows_at(s["Ys"], slots) * s["dY"][:, None, :]).sum(2)
        return Xs, Y, dYs, dweights, _rows_at(s["dXs"], slots).sum(1)
    F, t = c["F"], c["train"]
    bounds = s["offsets"].tolist()
    out = [torch.empty_like(s["Xs"])] + ([torch.empty_like(s["Xs"]), torch.empty_like(s["Win"]),
                                          torch.empty_like(s["Wout"])] if t else [])
    for e in range(c["E"]):
        rows = slice(bounds[e], bounds[e + 1])
        X, Win, Wout = s["Xs"][rows], s["Win"][e], s["Wout"][e]
        Z = X @ Win.t()
        G, U = Z[:, :F], Z[:, F:]
        A = _act(c["act"], G)
        H = A * U
        out[0][rows] = H @ Wout.t()
        if not t:
            continue
        dY = s["dYs"][rows]
        dH = dY @ Wout
        dZ = torch.cat([dH * U * _act_grad(c["act"], G), dH * A], 1)
        out[1][rows] = dZ @ Win
        out[2][e] = dZ.t() @ X
        out[3][e] = dY.t() @ H
    return tuple(out) if t else out[0]


# ---------------------------------------------------------------- own form ---
def _own(s):
    import fp32_emulated_gemm_gb300 as emu
    c = s["case"]
    if c["op"] == "rms_norm":
        if c["kind"] == "quant":
            Q, scales, *stream = emu.rms_norm_quant(s["X"], s["w"], residual=s["R"], eps=EPS)
            return (_dequantised(Q, scales), *stream)
        if c["kind"] == "fwd":
            out = emu.rms_norm_fwd(s["X"], s["w"], residual=s["R"], eps=EPS, save=False)
            return out if s["R"] is not None else (out,)
        Y, S, rstd = emu.rms_norm_fwd(s["X"], s["w"], residual=s["R"], eps=EPS)
        stream = () if s["R"] is None else (S,)
        return (Y, *stream, *emu.rms_norm_bwd(s["dY"], S, s["w"], rstd, add=s["add"]))
    if c["op"] == "route":
        plan, weights = emu.expert_route(s["logits"], c["k"], over=c["over"])
        out = (plan.experts, weights, plan.slots, plan.sources, plan.offsets)
        if not c["train"]:
            return out
        return out + (emu.expert_route_bwd(s["dweights"], s["logits"], plan, weights, over=c["over"]),)
    plan = emu.ExpertPlan(s["experts"], s["slots"], s["sources"], s["offsets"])
    if c["op"] == "exchange":
        Xs = emu.expert_dispatch(s["X"], plan)
        Y = emu.expert_combine_fwd(s["Ys"], plan, s["weights"], residual=s["R"])
        if not c["train"]:
            return Xs, Y
        dYs, dweights = emu.expert_combine_bwd(s["dY"], s["Ys"], plan, s["weights"])
        return Xs, Y, dYs, dweights, emu.expert_combine_fwd(s["dXs"], plan)
    act, mode = c["act"], c["mode"]
    if not c["train"]:
        return emu.expert_ffn_fwd(s["Xs"], s["Win"], s["Wout"], plan, act=act, mode=mode)
    Ys, D, H = emu.expert_ffn_fwd(s["Xs"], s["Win"], s["Wout"], plan, act=act, mode=mode, save=True)
    return (Ys,) + tuple(emu.expert_ffn_bwd(s["dYs"], s["Xs"], s["Win"], s["Wout"], D, H, plan, act=act, mode=mode))


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ---
def work(case):
    M = case["M"]
    if case["op"] == "rms_norm":
        N, t, r = case["N"], case["kind"] == "train", case["residual"]
        # X (and R), w -> Y (and S); and dY (and add) -> dX, dw (S counted once)
        out = N if case["kind"] != "quant" else N // 4 + (N + GROUP - 1) // GROUP
        return {"bytes": 4 * (M * (N * (1 + 2 * r) + out + t * N * (2 + r)) + N * (1 + t)), "flops": M * N * (5 + 9 * t)}
    E, k, t = case["E"], case["k"], case["train"]
    if case["op"] == "route":
        return {"bytes": 4 * (M * (E + 4 * k) + E + 1 + t * M * (E + k)), "flops": M * E * (2 + 3 * t)}
    T = M * k
    if case["op"] == "exchange":
        N = case["N"]
        # X -> Xs; Ys, R -> Y; and dY -> dYs; dXs -> dX; the plan and the weights
        rows = M * 3 + T * 2 + t * (T * 2 + M * 2)
        return {"bytes": 4 * (rows * N + (3 + t) * T), "flops": T * N * (2 + 4 * t)}
    K, F = case["K"], case["F"]
    used = min(E, T)                                 # experts that have rows
    rows = T * K * (2 + 2 * t)
    return {"bytes": 4 * (rows + 3 * F * K * (used + t * E)), "flops": 6 * T * F * K * (1 + 2 * t)}


# ------------------------------------------------------------------- exact ---
def _act64(name, z):
    """(act(z), act'(z)) in 64 bits, from the definitions."""
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if name == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh v) = expit(2 v), v = sqrt(2/pi) (z + 0.044715 z^3)
    c = 2 * math.sqrt(2 / math.pi)
    arg = c * z * (1 + 0.044715 * z.square())
    p = torch.special.expit(arg)
    return z * p, p + z * p * torch.special.expit(-arg) * c * (1 + 0.134145 * z.square())


def _exact_rms(s, c):
    D = torch.double
    M, N = c["M"], c["N"]
    block = max(1, min(M, (1 << 25) // N))
    parts, dw = [], torch.zeros(N, device="cuda", dtype=D)
    for r in range(0, M, block):
        cut = slice(r, r + block)
        x = s["X"][cut].to(D)
        if s["R"] is not None:
            x = x + s["R"][cut].to(D)
        rms = (torch.linalg.vector_norm(x, dim=1, keepdim=True).square() / N + EPS).sqrt()
        y = x / rms * s["w"].to(D)
        out = [y] if s["R"] is None else [y, x]
        if c["kind"] == "train":
            dy = s["dY"][cut].to(D)
            gr = dy * s["w"].to(D)
            dot = torch.einsum("ij,ij->i", gr, x)[:, None]
            dx = gr / rms - x * dot / (N * rms ** 3)
            out.append(dx if s["add"] is None else dx + s["add"][cut].to(D))
            dw += torch.einsum("ij,ij->j", dy, x / rms)
        parts.append(out)
    result = [torch.cat([p[i] for p in parts]) for i in range(len(parts[0]))]
    if c["kind"] == "quant":
        result[0] = None                             # rounded to 8 bits: no value of its own
    return tuple(result) + ((dw,) if c["kind"] == "train" else ())


def _exact_route(s, c):
    D = torch.double
    logits, E, k, over = s["logits"].to(D), c["E"], c["k"], c["over"]
    _, order = torch.sort(logits, dim=1, descending=True, stable=True)
    chosen = order[:, :k]
    values = logits.gather(1, chosen)
    open_ = values > -math.inf
    experts = torch.where(open_, chosen, torch.full_like(chosen, -1))
    norm = torch.logsumexp(values if over == "chosen" else logits, 1, keepdim=True)
    weights = torch.where(open_, torch.exp(values - norm), torch.zeros_like(values))
    # the sort by expert: a stable argsort, choices that go nowhere behind the others
    flat = torch.where(open_, chosen, torch.full_like(chosen, E)).reshape(-1)
    key, perm = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device), right=False)
    sources = torch.where(key < E, perm, torch.full_like(perm, -1))
    slots = torch.empty_like(flat)
    slots[perm] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(flat < E, slots, torch.full_like(slots, -1)).reshape(experts.shape)
    out = (experts.int(), weights, slots.int(), sources.int(), offsets.int())
    if not c["train"]:
        return out
    dw = s["dweights"].to(D)
    grad = torch.zeros_like(logits)
    grad.scatter_add_(1, chosen, torch.where(open_, weights * dw, torch.zeros_like(dw)))
    total = grad.sum(1, keepdim=True)
    if over == "chosen":
        soft = torch.zeros_like(logits).scatter_add_(1, chosen, weights)
    else:
        soft = torch.where(norm > -math.inf, torch.exp(logits - norm), torch.zeros_like(logits))
    return out + (grad - soft * total,)


def _exact_exchange(s, c):
    D = torch.double
    M, N, k = c["M"], c["N"], c["k"]
    if M * k * N > 1 << 29:
        return None
    slots, sources = s["slots"].long(), s["sources"].long()
    rows = sources >= 0
    Xs = torch.zeros(M * k, N, device="cuda", dtype=D)
    Xs[rows] = s["X"].to(D)[sources[rows] // k]
    Y = s["R"].to(D)
    dX, dYs = torch.zeros(M, N, device="cuda", dtype=D), torch.zeros(M * k, N, device="cuda", dtype=D)
    dweights = torch.zeros(M, k, device="cuda", dtype=D)
    for j in range(k):
        m = (slots[:, j] >= 0).nonzero()[:, 0]
        at, w = slots[m, j], s["weights"][m, j].to(D)
        Y[m] += w[:, None] * s["Ys"][at].to(D)
        if c["train"]:
            dy = s["dY"][m].to(D)
            dYs[at] = w[:, None] * dy
            dweights[m, j] = torch.einsum("ij,ij->i", dy, s["Ys"][at].to(D))
            dX[m] += s["dXs"][at].to(D)
    return (Xs, Y, dYs, dweights, dX) if c["train"] else (Xs, Y)


def _exact_experts(s, c):
    D = torch.double
    F, t = c["F"], c["train"]
    if work(c)["flops"] > 4e12:
        return None
    Ys, grads = [], ([], [], [])
    for e, n in enumerate(torch.diff(s["offsets"].long()).tolist()):
        r = sum(y.shape[0] for y in Ys)
        x, wo = s["Xs"][r:r + n].to(D), s["Wout"][e].to(D)
        wg, wu = s["Win"][e].to(D).split(F)
        a, da = _act64(c["act"], x.mm(wg.T))
        u = x.mm(wu.T)
        h = a * u
        Ys.append(h.mm(wo.T))
        if t:
            dy = s["dYs"][r:r + n].to(D)
            dh = dy.mm(wo)
            dg, du = dh * u * da, dh * a
            grads[0].append(dg.mm(wg) + du.mm(wu))
            grads[1].append(torch.cat([dg.T.mm(x), du.T.mm(x)]))
            grads[2].append(dy.T.mm(h))
    if not t:
        return torch.cat(Ys)
    return torch.cat(Ys), torch.cat(grads[0]), torch.stack(grads[1]), torch.stack(grads[2])


def exact(case, seed):
    s = prepare(case, seed)
    return {"rms_norm": _exact_rms, "route": _exact_route, "exchange": _exact_exchange,
            "experts": _exact_experts}[case["op"]](s, case)
