"""The feed-forward operators on real sizes: layer norm, the linear layer with
bias, activation and residual, and the gated feed-forward block.

Each is here in two forms on the same inputs: a plain one in elementary torch
operations (FP32 throughout), and the call a user makes of this package
(``own = True``).  ``listed()`` names the cases, ``draw(rng)`` makes another
of the same ranges, ``prepare`` makes the inputs, ``run`` does one pass,
``work`` says what a pass cannot do without and ``exact`` what it should give.

The sizes are the package's own layers (tokens x 256 -> 1024 of the small and
the large system, 1024 <-> 4096 of the wide model), one token and a few
tokens of the same layers, and ragged ones.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-5
LARGEST_ROWS = 552960          # tokens of the large system
FLOP_LIMIT = 6 * LARGEST_ROWS * 256 * 1024
LN_LIMIT = LARGEST_ROWS * 256


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # layer norm: M rows of width N.
        # inference on a handful of atoms: launch latency
        dict(name="ln_fwd_192x256", op="layer_norm", train=False, M=192, N=256),
        # one training step's norm in the small system (192 atoms x 32 neighbours)
        dict(name="ln_train_6144x256", op="layer_norm", train=True, M=6144, N=256),
        # a width and a row count that nothing divides, rows off 16-byte boundaries
        dict(name="ln_train_4099x1001", op="layer_norm", train=True, M=4099, N=1001),
        # the large system (17,280 atoms x 32 neighbours): memory bound
        dict(name="ln_train_552960x256", op="layer_norm", train=True, M=LARGEST_ROWS, N=256),
        # linear layer with its epilogue: Y = act(X W^T + b) [+ residual].
        # one token through the wide model's expanding layer: reads the weight once
        dict(name="linear_fwd_1x1024x4096_gelu", op="linear_act", train=False, M=1, K=1024, N=4096, act="gelu",
             residual=False, mode="bf16x9"),
        # the small system's expanding layer, inference, in the two-component mode
        dict(name="linear_fwd_6144x256x1024_gelu_tf32x3", op="linear_act", train=False, M=6144, K=256, N=1024,
             act="gelu", residual=False, mode="tf32x3"),
        # a ragged layer with a residual, forward and backward
        dict(name="linear_train_1537x300x500_silu_res_tf32x3", op="linear_act", train=True, M=1537, K=300, N=500,
             act="silu", residual=True, mode="tf32x3"),
        # the wide model's expanding layer, forward and backward
        dict(name="linear_train_6144x1024x4096_gelu", op="linear_act", train=True, M=6144, K=1024, N=4096,
             act="gelu", residual=False, mode="bf16x9"),
        # gated block: Y = (act(X Wg^T + bg) * (X Wu^T + bu)) Wo^T + bo + X0.
        # one token through the wide model's block
        dict(name="ffn_fwd_1x1024x4096_silu", op="gated_ffn", train=False, M=1, K=1024, F=4096, act="silu",
             mode="bf16x9"),
        # a training step of the small system's block
        dict(name="ffn_train_6144x256x1024_silu", op="gated_ffn", train=True, M=6144, K=256, F=1024, act="silu",
             mode="bf16x9"),
        # a ragged block, in the two-component mode
        dict(name="ffn_train_777x260x700_gelu_tanh_tf32x3", op="gated_ffn", train=True, M=777, K=260, F=700,
             act="gelu_tanh", mode="tf32x3"),
        # forces on the large system need the block's forward over every token
        dict(name="ffn_fwd_552960x256x1024_silu", op="gated_ffn", train=False, M=LARGEST_ROWS, K=256, F=1024,
             act="silu", mode="bf16x9"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


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
    op = rng.choice(["layer_norm", "linear_act", "gated_ffn"])
    train = rng.random() < 0.6
    if op == "layer_norm":
        N = _width(rng, 16, 8192)
        M = _log_uniform(rng, 1, max(1, min(LARGEST_ROWS, LN_LIMIT // N)))
        return dict(op=op, train=train, M=M, N=N)
    mode = rng.choice(["bf16x9", "tf32x3"])
    # relu's derivative jumps at zero, so a rounding of Z decides whole entries
    # of a gradient; its forward pass alone has one answer
    act = rng.choice(["gelu", "gelu_tanh", "silu"] + ([] if train else ["relu"]))
    K = _width(rng, 64, 2048)
    N = _width(rng, 64, 4096)
    # one token to the most rows that cost no more than the largest listed case
    per_row = 2 * K * N * (3 if op == "gated_ffn" else 1) * (3 if train else 1)
    M = _log_uniform(rng, 1, max(1, min(LARGEST_ROWS, FLOP_LIMIT // per_row // 2)))
    if op == "linear_act":
        return dict(op=op, train=train, M=M, K=K, N=N, act=act, residual=rng.random() < 0.5, mode=mode)
    return dict(op=op, train=train, M=M, K=K, F=N, act=act, mode=mode)


# ----------------------------------------------------------------- inputs ---
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(mean, std, generator=g)

    s = dict(case=case)
    M = case["M"]
    if case["op"] == "layer_norm":
        N = case["N"]
        # a residual stream: channels of different offset and spread
        s["X"] = normal(M, N).mul_(normal(N, std=0.5).exp_()).add_(normal(N, std=0.7))
        s["w"] = normal(N, std=0.1, mean=1.0)
        s["b"] = normal(N, std=0.1)
        if case["train"]:
            s["dY"] = normal(M, N)
    elif case["op"] == "linear_act":
        K, N = case["K"], case["N"]
        s["X"] = normal(M, K)
        s["W"] = normal(N, K, std=K ** -0.5)
        s["b"] = normal(N, std=0.1)
        s["R"] = normal(M, N) if case["residual"] else None
        if case["train"]:
            s["dY"] = normal(M, N)
    else:
        K, F = case["K"], case["F"]
        s["X"] = normal(M, K)
        s["Win"] = normal(2 * F, K, std=K ** -0.5)      # gate rows, then up rows
        s["bin"] = normal(2 * F, std=0.1)
        s["Wout"] = normal(K, F, std=F ** -0.5)
        s["bout"] = normal(K, std=0.1)
        s["R"] = normal(M, K)
        if case["train"]:
            s["dY"] = normal(M, K)
    return s


# -------------------------------------------------------------- plain form ---
_C = math.sqrt(2.0 / math.pi)


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z * z * z)))


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (0.5 * _C)
    t = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * (_C * (1.0 + 3 * 0.044715 * z * z))


def _plain(s):
    c = s["case"]
    if c["op"] == "layer_norm":
        X, w, b = s["X"], s["w"], s["b"]
        xc = X - X.mean(1, keepdim=True)
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
        xh = xc * rstd
        Y = xh * w + b
        if not c["train"]:
            return Y
        dY = s["dY"]
        d = dY * w
        dX = rstd * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
        return Y, dX, (dY * xh).sum(0), dY.sum(0)
    if c["op"] == "linear_act":
        X, W = s["X"], s["W"]
        Z = X @ W.t() + s["b"]
        Y = _act(c["act"], Z)
        if s["R"] is not None:
            Y = Y + s["R"]
        if not c["train"]:
            return Y
        dZ = s["dY"] * _act_grad(c["act"], Z)
        return Y, dZ @ W, dZ.t() @ X, dZ.sum(0)
    X, Win, Wout, F = s["X"], s["Win"], s["Wout"], c["F"]
    Z = X @ Win.t() + s["bin"]
    G, U = Z[:, :F], Z[:, F:]
    A = _act(c["act"], G)
    H = A * U
    Y = H @ Wout.t() + s["bout"] + s["R"]
    if not c["train"]:
        return Y
    dY = s["dY"]
    dH = dY @ Wout
    dZ = torch.cat([dH * U * _act_grad(c["act"], G), dH * A], 1)
    return Y, dZ @ Win, dZ.t() @ X, dZ.sum(0), dY.t() @ H, dY.sum(0)


# ---------------------------------------------------------------- own form ---
def _own(s):
    import fp32_emulated_gemm_gb300 as emu
    c = s["case"]
    if c["op"] == "layer_norm":
        Y, mean, rstd = emu.layer_norm_fwd(s["X"], s["w"], s["b"], eps=EPS)
        if not c["train"]:
            return Y
        return (Y,) + tuple(emu.layer_norm_bwd(s["dY"], s["X"], s["w"], mean, rstd))
    act, mode = c["act"], c["mode"]
    if c["op"] == "linear_act":
        if not c["train"]:
            return emu.linear_act_fwd(s["X"], s["W"], s["b"], act=act, residual=s["R"], mode=mode)
        Y, Z = emu.linear_act_fwd(s["X"], s["W"], s["b"], act=act, residual=s["R"], mode=mode, save=True)
        return (Y,) + tuple(emu.linear_act_bwd(s["dY"], s["X"], s["W"], Z, act=act, mode=mode))
    if not c["train"]:
        return emu.gated_ffn_fwd(s["X"], s["Win"], s["bin"], s["Wout"], s["bout"], act=act, residual=s["R"], mode=mode)
    Y, Z, H = emu.gated_ffn_fwd(s["X"], s["Win"], s["bin"], s["Wout"], s["bout"], act=act, residual=s["R"],
                                mode=mode, save=True)
    return (Y,) + tuple(emu.gated_ffn_bwd(s["dY"], s["X"], s["Win"], s["Wout"], Z, H, act=act, mode=mode))


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work ---
def work(case):
    M, t = case["M"], case["train"]
    if case["op"] == "layer_norm":
        N = case["N"]
        # X, w, b -> Y; and dY -> dX, dw, db (X counted once)
        return {"bytes": 4 * ((2 + 2 * t) * M * N + (2 + 2 * t) * N), "flops": (8 + 14 * t) * M * N}
    K = case["K"]
    if case["op"] == "linear_act":
        N = case["N"]
        rows = K + N + (N if case["residual"] else 0) + t * (N + K)
        return {"bytes": 4 * (M * rows + (1 + t) * (N * K + N)), "flops": 2 * M * N * K * (1 + 2 * t)}
    F = case["F"]
    rows = 3 * K + t * 2 * K                        # X, residual, Y; dY, dX
    return {"bytes": 4 * (M * rows + (1 + t) * (3 * F * K + 2 * F + K)), "flops": 6 * M * F * K * (1 + 2 * t)}


# ------------------------------------------------------------------- exact ---
def _phi64(z):
    return torch.special.ndtr(z)


def _act64(name, z):
    """(act(z), act'(z)) in 64 bits, from the definitions."""
    if name == "relu":
        on = (z > 0).double()
        return z * on, on
    if name == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if name == "gelu":
        density = torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        return z * _phi64(z), _phi64(z) + z * density
    # 0.5 (1 + tanh v) = expit(2 v), v = sqrt(2/pi) (z + 0.044715 z^3)
    k = 2 * math.sqrt(2 / math.pi)
    arg = k * z * (1 + 0.044715 * z.square())
    p = torch.special.expit(arg)
    return z * p, p + z * p * torch.special.expit(-arg) * k * (1 + 0.134145 * z.square())


def exact(case, seed):
    s = prepare(case, seed)
    M, t = case["M"], case["train"]
    # rows in blocks that keep the 64-bit intermediates within a few GB
    width = case["N"] if case["op"] == "layer_norm" else case.get("N", 0) + 2 * case.get("F", 0) + case["K"]
    block = max(1, min(M, (1 << 27) // max(1, width)))
    D = torch.double
    rows = []                                        # per block: the outputs that have M rows
    sums = None                                      # the outputs summed over the rows
    for r in range(0, M, block):
        cut = slice(r, min(M, r + block))
        if case["op"] == "layer_norm":
            x, w = s["X"][cut].to(D), s["w"].to(D)
            var, mu = torch.var_mean(x, 1, unbiased=False, keepdim=True)
            sd = (var + EPS).sqrt()
            n = (x - mu) / sd
            out, part = [n * w + s["b"].to(D)], []
            if t:
                dy = s["dY"][cut].to(D)
                gr = dy * w
                N = case["N"]
                out.append((gr - gr.sum(1, keepdim=True) / N - n * ((gr * n).sum(1, keepdim=True) / N)) / sd)
                part = [torch.einsum("ij,ij->j", dy, n), dy.sum(0)]
        elif case["op"] == "linear_act":
            x, w = s["X"][cut].to(D), s["W"].to(D)
            a, da = _act64(case["act"], torch.addmm(s["b"].to(D), x, w.T))
            out, part = [a if s["R"] is None else a + s["R"][cut].to(D)], []
            if t:
                dz = s["dY"][cut].to(D) * da
                out.append(dz.mm(w))
                part = [dz.T.mm(x), dz.sum(0)]
        else:
            F = case["F"]
            x, wo = s["X"][cut].to(D), s["Wout"].to(D)
            wg, wu = s["Win"].to(D).split(F)
            bg, bu = s["bin"].to(D).split(F)
            a, da = _act64(case["act"], torch.addmm(bg, x, wg.T))
            u = torch.addmm(bu, x, wu.T)
            h = a * u
            out, part = [torch.addmm(s["bout"].to(D), h, wo.T) + s["R"][cut].to(D)], []
            if t:
                dy = s["dY"][cut].to(D)
                dh = dy.mm(wo)
                dg, du = dh * u * da, dh * a
                out.append(dg.mm(wg) + du.mm(wu))
                part = [torch.cat([dg.T.mm(x), du.T.mm(x)]), torch.cat([dg.sum(0), du.sum(0)]), dy.T.mm(h), dy.sum(0)]
        rows.append(out)
        sums = part if sums is None else [p + q for p, q in zip(sums, part)]
    result = [torch.cat([o[i] for o in rows]) for i in range(len(rows[0]))] + sums
    return tuple(result) if t else result[0]
