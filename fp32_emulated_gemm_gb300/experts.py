"""Operators of a layer of experts: the RMS norm, the router, the tokens' way to
their experts' rows and back, and the experts' gated blocks on the emulated
products, each with its backward pass.

As in feed_forward.py the functions only marshal arguments (see
``include/emu_gemm.h`` for the contract).  How many rows an expert has stays on
the device: a layer runs without a synchronisation, and in a CUDA graph.
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _check, _mode
from . import feed_forward as ff
from .feed_forward import _NONE, _SIGNATURES, _act, _c_name, _empty, _flat, _float32, _fn, _Function, _new_vector
from .feed_forward import _result, _rows, _stream_of, _vector

EMU_OVER_CHOSEN, EMU_OVER_ALL = range(2)
OVER = {"chosen": EMU_OVER_CHOSEN, "all": EMU_OVER_ALL}
SCALE_GROUP = 128                       # columns that share a scale of rms_norm_quant

_SIGNATURES.update({
    "emu_rms_norm_fwd": "nnpnpnpfpnpnp",
    "emu_rms_norm_quant": "nnpnpnpfpnpnpn",
    "emu_rms_norm_bwd": "nnpnpnpppnpnp",
    "emu_expert_route": "eneepnppppp",
    "emu_expert_sort": "neepppp",
    "emu_expert_route_bwd": "eneeppnpppn",
    "emu_expert_dispatch": "nenpnpppn",
    "emu_expert_combine_fwd": "nenpnpppnpn",
    "emu_expert_combine_bwd": "nenpnpnppppnp",
    "emu_expert_ffn_fwd": "eenennnpnppnpnpnpnpn",
    "emu_expert_ffn_bwd": "enennnpnpnppnpnpnpnpnpnpnpn",
})
emu_rms_norm_fwd = _c_name("emu_rms_norm_fwd")
emu_rms_norm_quant = _c_name("emu_rms_norm_quant")
emu_rms_norm_bwd = _c_name("emu_rms_norm_bwd")
emu_expert_route = _c_name("emu_expert_route")
emu_expert_sort = _c_name("emu_expert_sort")
emu_expert_route_bwd = _c_name("emu_expert_route_bwd")
emu_expert_dispatch = _c_name("emu_expert_dispatch")
emu_expert_combine_fwd = _c_name("emu_expert_combine_fwd")
emu_expert_combine_bwd = _c_name("emu_expert_combine_bwd")
emu_expert_ffn_fwd = _c_name("emu_expert_ffn_fwd")
emu_expert_ffn_bwd = _c_name("emu_expert_ffn_bwd")

_int32 = torch.int32


def _new(M, N, device):
    """A new matrix with rows on 16-byte boundaries."""
    if not N & 3:
        t, ld = _empty((M, N), device=device, dtype=_float32), N
    else:   # (a view of a padded matrix costs the host 2.5 us more)
        ld = (N + 3) // 4 * 4
        t = torch.empty_strided((M, N), (ld, 1), device=device, dtype=_float32)
    return t, t.data_ptr(), ld


def _ints(t, name, shape):
    """(tensor, address) of an int32 tensor of this shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _int32 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA int32 tensor")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        t = t.contiguous()
    return t, t.data_ptr()


def _dense(t, name, shape):
    """(tensor, address) of a contiguous float32 matrix of this shape."""
    t, p, ld = _rows(t, name, shape)
    if not t.is_contiguous():
        t = t.contiguous()
        p = t.data_ptr()
    return t, p


def _over(over):
    try:
        return OVER[over]
    except KeyError:
        raise ValueError(f"over must be one of {', '.join(OVER)}") from None


# ------------------------------------------------------------- RMS norm ----
def _norm_inputs(X, weight, residual):
    X, px, ldx = _rows(X, "X")
    M, N = X.shape
    weight, pw = _vector(weight, "weight", N)
    residual, pr, ldr = _NONE if residual is None else _rows(residual, "residual", (M, N))
    S, ps, lds = _NONE if residual is None else (_empty((M, N), device=X.device, dtype=_float32), None, N)
    if S is not None:
        ps = S.data_ptr()
    return X, px, ldx, weight, pw, residual, pr, ldr, S, ps, lds


def rms_norm_fwd(X, weight=None, *, residual=None, eps=1e-6, save=True, out=None):
    """Y = S * rstd * weight over the rows of S = X + residual, rstd = 1 /
    sqrt(mean(S^2) + eps).  (Y, S, rstd) for rms_norm_bwd, S being X itself when
    there is no residual; without `save` (Y, S), or Y alone without a residual."""
    X, px, ldx, weight, pw, residual, pr, ldr, S, ps, lds = _norm_inputs(X, weight, residual)
    M, N = X.shape
    device = X.device
    if out is None:
        Y, ldy = _empty((M, N), device=device, dtype=_float32), N
        py = Y.data_ptr()
    else:
        Y, py, ldy = _result(out, (M, N), device, "out")
    rstd, prs = _new_vector(M, device) if save else (None, None)
    _check(_fn("emu_rms_norm_fwd")(M, N, px, ldx, pr, ldr, pw, eps, py, ldy, ps, lds, prs,
                                   _stream_of("rms_norm_fwd", X, residual, weight, Y)), "emu_rms_norm_fwd")
    if save:
        return Y, X if S is None else S, rstd
    return Y if S is None else (Y, S)


def rms_norm_quant(X, weight=None, *, residual=None, eps=1e-6):
    """rms_norm_fwd's Y in 8 bits: (Q, scales), or (Q, scales, S) with a residual.
    Q is float8_e4m3fn, and Y[m, c] stands at Q[m, c] * scales[m, c // 128]; the
    scales are powers of two."""
    X, px, ldx, weight, pw, residual, pr, ldr, S, ps, lds = _norm_inputs(X, weight, residual)
    M, N = X.shape
    groups = (N + SCALE_GROUP - 1) // SCALE_GROUP
    Q = _empty((M, N), device=X.device, dtype=torch.float8_e4m3fn)
    scales = _empty((M, groups), device=X.device, dtype=_float32)
    _check(_fn("emu_rms_norm_quant")(M, N, px, ldx, pr, ldr, pw, eps, Q.data_ptr(), N, scales.data_ptr(), groups, ps, lds,
                                     _stream_of("rms_norm_quant", X, residual, weight)), "emu_rms_norm_quant")
    return (Q, scales) if S is None else (Q, scales, S)


def rms_norm_bwd(dY, S, weight, rstd, *, add=None, need_input=True, need_weight=True):
    """(dX, dweight) of rms_norm_fwd from its S and rstd; dX is the residual's
    gradient too.  `add` (a gradient that reaches S by another way) is added to
    it.  What is not needed comes back as None."""
    S, ps, lds = _rows(S, "S")
    M, N = shape = tuple(S.shape)
    dY, pdy, lddy = _rows(dY, "dY", shape)
    add, pa, lda = _NONE if add is None else _rows(add, "add", shape)
    if add is not None and not need_input:
        raise ValueError("add needs dX")
    weight, pw = _vector(weight, "weight", N)
    rstd, pr = _vector(rstd, "rstd", M)
    if rstd is None:
        raise TypeError("rstd must be a CUDA float32 tensor")
    dX = pdx = dw = pdw = None
    if need_input:
        dX = _empty(shape, device=S.device, dtype=_float32)
        pdx = dX.data_ptr()
    if need_weight:
        dw, pdw = _new_vector(N, S.device)
    _check(_fn("emu_rms_norm_bwd")(M, N, pdy, lddy, ps, lds, pw, pr, pa, lda, pdx, N, pdw,
                                   _stream_of("rms_norm_bwd", S, dY, weight, rstd, add)), "emu_rms_norm_bwd")
    return dX, dw


# --------------------------------------------------------------- router ----
class ExpertPlan(NamedTuple):
    """Where the tokens' choices go (int32 tensors): the chosen `experts` [M, k]
    (-1: none), each choice's row `slots` [M, k] (-1: none), each row's choice
    `sources` [M k] (m k + j; -1 behind the last), and the experts' first rows
    `offsets` [E + 1]."""
    experts: torch.Tensor
    slots: torch.Tensor
    sources: torch.Tensor
    offsets: torch.Tensor


def _new_plan(M, E, k, device, experts=None):
    new = lambda *s: _empty(s, device=device, dtype=_int32)
    return ExpertPlan(new(M, k) if experts is None else experts, new(M, k), new(M * k), new(E + 1))


def expert_route(logits, k, *, over="chosen"):
    """(plan, weights): the k largest of each token's logits [M, E] (the lowest
    index first among equals), sorted by expert, and their softmax weights [M, k]
    over the chosen logits or, over="all", all of the token's.  A logit of -inf is
    closed; what a token has too few open ones for goes nowhere, with weight 0."""
    over = _over(over)
    logits, pl, ldl = _rows(logits, "logits")
    M, E = logits.shape
    k = int(k)
    if not 1 <= k <= E:
        raise ValueError(f"k must be within 1 .. {E}")
    plan = _new_plan(M, E, k, logits.device)
    weights = _empty((M, k), device=logits.device, dtype=_float32)
    _check(_fn("emu_expert_route")(over, M, E, k, pl, ldl, plan.experts.data_ptr(), weights.data_ptr(),
                                   plan.slots.data_ptr(), plan.sources.data_ptr(), plan.offsets.data_ptr(),
                                   _stream_of("expert_route", logits)), "emu_expert_route")
    return plan, weights


def expert_sort(experts, num_experts):
    """The plan of given choices (int32 [M, k]); one outside 0 .. num_experts - 1
    goes nowhere."""
    if not isinstance(experts, torch.Tensor) or experts.dim() != 2:
        raise ValueError("experts must be a matrix")
    M, k = experts.shape
    E = int(num_experts)
    experts, pe = _ints(experts, "experts", (M, k))
    plan = _new_plan(M, E, k, experts.device, experts)
    _check(_fn("emu_expert_sort")(M, E, k, pe, plan.slots.data_ptr(), plan.sources.data_ptr(), plan.offsets.data_ptr(),
                                  _stream_of("expert_sort", experts)), "emu_expert_sort")
    return plan


def expert_route_bwd(dweights, logits, plan, weights, *, over="chosen"):
    """dlogits [M, E] of expert_route from its plan and weights."""
    over = _over(over)
    logits, pl, ldl = _rows(logits, "logits")
    M, E = logits.shape
    if plan.experts.dim() != 2:
        raise ValueError("plan.experts must be a matrix")
    k = plan.experts.shape[1]
    experts, pe = _ints(plan.experts, "plan.experts", (M, k))
    weights, pw = _dense(weights, "weights", (M, k))
    dweights, pdw = _dense(dweights, "dweights", (M, k))
    dlogits = _empty((M, E), device=logits.device, dtype=_float32)
    _check(_fn("emu_expert_route_bwd")(over, M, E, k, pdw, pl, ldl, pe, pw, dlogits.data_ptr(), E,
                                       _stream_of("expert_route_bwd", logits, experts, weights, dweights)),
           "emu_expert_route_bwd")
    return dlogits


# ------------------------------------------------------------- exchange ----
def _plan_of(plan, sources=True):
    if plan.slots.dim() != 2:
        raise ValueError("plan.slots must be a matrix")
    M, k = plan.slots.shape
    slots, psl = _ints(plan.slots, "plan.slots", (M, k))
    src, psr = _ints(plan.sources, "plan.sources", (M * k,)) if sources else (None, None)
    return M, k, slots, psl, src, psr


def expert_dispatch(X, plan):
    """The tokens at their experts' rows: Xs[plan.slots[m, j]] = X[m] [M k, N];
    rows without a source are zero."""
    M, k, slots, psl, src, psr = _plan_of(plan)
    X, px, ldx = _rows(X, "X")
    N = X.shape[1]
    if X.shape[0] != M:
        raise ValueError(f"X must have the plan's {M} rows, not {X.shape[0]}")
    Xs, pxs, ldxs = _new(M * k, N, X.device)
    _check(_fn("emu_expert_dispatch")(M, k, N, px, ldx, psl, psr, pxs, ldxs, _stream_of("expert_dispatch", X, slots, src)),
           "emu_expert_dispatch")
    return Xs


def expert_combine_fwd(Ys, plan, weights=None, *, residual=None, out=None):
    """Y[m] = sum over j of weights[m, j] Ys[plan.slots[m, j]] + residual[m].
    Without weights and residual it is expert_dispatch's gradient."""
    M, k, slots, psl, _, _ = _plan_of(plan, sources=False)
    Ys, py, ldys = _rows(Ys, "Ys")
    N = Ys.shape[1]
    if Ys.shape[0] != M * k:
        raise ValueError(f"Ys must have the plan's {M * k} rows, not {Ys.shape[0]}")
    weights, pw = (None, None) if weights is None else _dense(weights, "weights", (M, k))
    residual, pr, ldr = _NONE if residual is None else _rows(residual, "residual", (M, N))
    Y, pyo, ldy = _new(M, N, Ys.device) if out is None else _result(out, (M, N), Ys.device, "out")
    _check(_fn("emu_expert_combine_fwd")(M, k, N, py, ldys, psl, pw, pr, ldr, pyo, ldy,
                                         _stream_of("expert_combine_fwd", Ys, slots, weights, residual, Y)),
           "emu_expert_combine_fwd")
    return Y


def expert_combine_bwd(dY, Ys, plan, weights, *, need=(True, True)):
    """(dYs, dweights) of expert_combine_fwd with weights (the residual's gradient
    is dY); rows of dYs without a source are zero.  `need` says which are wanted;
    Ys may be None where dweights is not."""
    M, k, slots, psl, src, psr = _plan_of(plan)
    dY, pdy, lddy = _rows(dY, "dY")
    N = dY.shape[1]
    if dY.shape[0] != M:
        raise ValueError(f"dY must have the plan's {M} rows, not {dY.shape[0]}")
    Ys, py, ldys = _rows(Ys, "Ys", (M * k, N)) if need[1] or Ys is not None else _NONE
    weights, pw = _dense(weights, "weights", (M, k))
    dYs, pdys, lddys = _new(M * k, N, dY.device) if need[0] else _NONE
    dw = pdw = None
    if need[1]:
        dw = _empty((M, k), device=dY.device, dtype=_float32)
        pdw = dw.data_ptr()
    _check(_fn("emu_expert_combine_bwd")(M, k, N, pdy, lddy, py, ldys, psl, psr, pw, pdys, lddys, pdw,
                                         _stream_of("expert_combine_bwd", dY, Ys, slots, src, weights)),
           "emu_expert_combine_bwd")
    return dYs, dw


# -------------------------------------------------------------- experts ----
def _weights3(W, name):
    """(tensor, address, row stride) of [E, R, C] weights, one matrix behind the other."""
    if not isinstance(W, torch.Tensor) or W.dtype is not _float32 or not W.is_cuda:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if W.dim() != 3:
        raise ValueError(f"{name} must have three dimensions: experts, rows, columns")
    if not W.is_contiguous():
        W = W.contiguous()
    return W, W.data_ptr(), W.shape[2]


def _expert_shapes(X, W_in, W_out, plan):
    rows, K = X.shape
    E, F2, Kw = W_in.shape
    Eo, N, F = W_out.shape
    if F2 != 2 * F:
        raise ValueError("W_in must have the gate's rows, then as many of the up projection, one each per column of W_out")
    if Kw != K:
        raise ValueError("inner dimensions differ")
    if Eo != E:
        raise ValueError("W_in and W_out must have as many experts")
    offsets, po = _ints(plan.offsets, "plan.offsets", (E + 1,))
    return rows, E, K, F, N, offsets, po


def expert_ffn_fwd(X, W_in, W_out, plan, *, act="silu", mode="bf16x9", save=False):
    """Each expert's gated block on its rows of X [rows, K] (sorted by expert,
    plan.offsets): Y = (a(X Wg^T) * (X Wu^T)) W_out^T with W_in [E, 2F, K] (Wg's
    rows, then Wu's) and W_out [E, N, F]; with `save` (Y, D, H) for
    expert_ffn_bwd.  Rows behind the last expert's are not written."""
    mode, a = _mode(mode), _act(act)
    X, px, ldx = _rows(X, "X")
    W_in, pwi, ldwi = _weights3(W_in, "W_in")
    W_out, pwo, ldwo = _weights3(W_out, "W_out")
    rows, E, K, F, N, offsets, po = _expert_shapes(X, W_in, W_out, plan)
    device = X.device
    Y, py, ldy = _new(rows, N, device)
    H, ph, ldh = _new(rows, F, device)
    D, pd, ldd = _new(rows, 2 * F, device) if save else _NONE
    s = _stream_of("expert_ffn_fwd", X, W_in, W_out, offsets)
    _check(_fn("emu_expert_ffn_fwd")(mode, a, rows, E, K, F, N, px, ldx, po, pwi, ldwi, pwo, ldwo, pd, ldd, ph, ldh, py,
                                     ldy, s), "emu_expert_ffn_fwd")
    return (Y, D, H) if save else Y


def expert_ffn_bwd(dY, X, W_in, W_out, D, H, plan, *, act="silu", mode="bf16x9", need=(True, True, True)):
    """(dX, dW_in, dW_out) of expert_ffn_fwd from its D and H; `need` says which
    are wanted.  (D holds the activation's part; `act` only has to name one.)  D
    may be None where only dW_out is wanted, H where it is not.  Rows of dX behind
    the last expert's are not written."""
    _act(act)
    X, px, ldx = _rows(X, "X")
    W_in, pwi, ldwi = _weights3(W_in, "W_in")
    W_out, pwo, ldwo = _weights3(W_out, "W_out")
    rows, E, K, F, N, offsets, po = _expert_shapes(X, W_in, W_out, plan)
    dY, pdy, lddy = _rows(dY, "dY", (rows, N))
    inner = need[0] or need[1]
    D, pd, ldd = _rows(D, "D", (rows, 2 * F)) if inner or D is not None else _NONE
    H, ph, ldh = _rows(H, "H", (rows, F)) if need[2] or H is not None else _NONE
    device = X.device
    dZ, pdz, lddz = _new(rows, 2 * F, device) if inner else _NONE
    dX, pdx, lddx = _new(rows, K, device) if need[0] else _NONE
    dWi, pdwi, lddwi = _new(E * 2 * F, K, device) if need[1] else _NONE
    dWo, pdwo, lddwo = _new(E * N, F, device) if need[2] else _NONE
    s = _stream_of("expert_ffn_bwd", dY, X, W_in, W_out, D, H, offsets)
    _check(_fn("emu_expert_ffn_bwd")(_mode(mode), rows, E, K, F, N, pdy, lddy, px, ldx, po, pwi, ldwi, pwo, ldwo, pd, ldd,
                                     ph, ldh, pdz, lddz, pdx, lddx, pdwi, lddwi, pdwo, lddwo, s), "emu_expert_ffn_bwd")
    return dX, None if dWi is None else dWi.unflatten(0, (E, 2 * F)), None if dWo is None else dWo.unflatten(0, (E, N))


# ------------------------------------------------------------- autograd ----
class EmuRMSNormFunction(_Function):
    """(Y, S): the norm and the stream behind the residual's addition (X itself
    without one), whose gradient joins in the norm's backward pass."""

    @staticmethod
    def infer(X, weight, residual, eps):
        r = rms_norm_fwd(X, weight, residual=residual, eps=eps, save=False)
        return (r, X) if residual is None else r

    @staticmethod
    def forward(ctx, X, weight, residual, eps):
        Y, S, rstd = rms_norm_fwd(X, weight, residual=residual, eps=eps)
        ctx.save_for_backward(S, weight, rstd)
        ctx.set_materialize_grads(False)
        return Y, S

    @staticmethod
    @once_differentiable
    def backward(ctx, dY, dS):
        S, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        if dY is None:
            return dS if need[0] else None, None, dS if need[2] else None, None
        inner = need[0] or need[2]
        dX, dw = rms_norm_bwd(dY, S, weight, rstd, add=dS if inner else None, need_input=inner,
                              need_weight=need[1] and weight is not None)
        return dX if need[0] else None, dw, dX if need[2] else None, None


class EmuExpertFFNFunction(_Function):
    """Each token's experts' gated blocks, weighted and summed, plus the residual."""

    @staticmethod
    def infer(X, logits, W_in, W_out, residual, k, over, act, mode):
        plan, weights = expert_route(logits, k, over=over)
        Ys = expert_ffn_fwd(expert_dispatch(X, plan), W_in, W_out, plan, act=act, mode=mode)
        return expert_combine_fwd(Ys, plan, weights, residual=residual)

    @staticmethod
    def forward(ctx, X, logits, W_in, W_out, residual, k, over, act, mode):
        plan, weights = expert_route(logits, k, over=over)
        Xs = expert_dispatch(X, plan)
        Ys, D, H = expert_ffn_fwd(Xs, W_in, W_out, plan, act=act, mode=mode, save=True)
        ctx.save_for_backward(logits, W_in, W_out, Xs, Ys, D, H, weights, *plan)
        ctx.over, ctx.act, ctx.mode = over, act, mode
        return expert_combine_fwd(Ys, plan, weights, residual=residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        logits, W_in, W_out, Xs, Ys, D, H, weights, *plan = ctx.saved_tensors
        plan = ExpertPlan(*plan)
        need = ctx.needs_input_grad
        inner = need[0] or need[2] or need[3]
        dX = dlogits = dW_in = dW_out = None
        if inner or need[1]:
            dYs, dw = expert_combine_bwd(dY, Ys, plan, weights, need=(inner, need[1]))
            if need[1]:
                dlogits = expert_route_bwd(dw, logits, plan, weights, over=ctx.over)
            if inner:
                dXs, dW_in, dW_out = expert_ffn_bwd(dYs, Xs, W_in, W_out, D, H, plan, act=ctx.act, mode=ctx.mode,
                                                    need=(need[0], need[2], need[3]))
                if need[0]:
                    dX = expert_combine_fwd(dXs, plan)
        return dX, dlogits, dW_in, dW_out, dY if need[4] else None, None, None, None, None


class EmuRMSNorm(torch.nn.Module):
    """RMS norm over the last dimension.  With a residual, forward(x, residual)
    gives (norm(x + residual), x + residual)."""

    def __init__(self, features, eps=1e-6, device=None, dtype=torch.float32):
        super().__init__()
        self.features, self.eps = features, eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        rows, residual, shape = _flat(x, residual, self.features, self.features)
        y, s = EmuRMSNormFunction.apply(rows, self.weight, residual, self.eps)
        return y.reshape(shape) if residual is None else (y.reshape(shape), s.reshape(shape))


def _token_mask(mask, x):
    if tuple(mask.shape) != tuple(x.shape[:-1]) or mask.dtype != torch.bool:
        raise ValueError(f"the mask must be bool of shape {tuple(x.shape[:-1])}")
    return mask.reshape(-1)


class EmuExpertFFN(torch.nn.Module):
    """A layer of experts: each token goes through the gated blocks of the `k`
    experts that the router's logits favour, weighted by their softmax (`over` the
    chosen logits or all).  weight_in holds each expert's gate rows, then its up
    rows."""

    def __init__(self, in_features, hidden_features, num_experts, k, out_features=None, over="chosen", act="silu",
                 mode="bf16x9", device=None, dtype=torch.float32):
        super().__init__()
        _act(act), _over(over)
        if _mode(mode) not in ff._FUSED:
            raise ValueError("mode must be bf16x9 or tf32x3")
        if not 1 <= k <= num_experts:
            raise ValueError(f"k must be within 1 .. {num_experts}")
        out_features = in_features if out_features is None else out_features
        self.in_features, self.hidden_features, self.out_features = in_features, hidden_features, out_features
        self.num_experts, self.k, self.over, self.act, self.mode = num_experts, k, over, act, mode
        self.router = ff.EmuLinearAct(in_features, num_experts, bias=False, act="none", mode=mode, device=device, dtype=dtype)
        new = lambda *s: torch.nn.Parameter(torch.empty(s, device=device, dtype=dtype))
        self.weight_in = new(num_experts, 2 * hidden_features, in_features)
        self.weight_out = new(num_experts, out_features, hidden_features)
        self.reset_parameters()

    def reset_parameters(self):
        """nn.Linear's initial values, for the router and each projection of an expert."""
        self.router.reset_parameters()
        for w in (self.weight_in, self.weight_out):
            bound = w.shape[2] ** -0.5 if w.shape[2] else 0.0
            torch.nn.init.uniform_(w, -bound, bound)

    def forward(self, x, residual=None, mask=None):
        """`mask` (x's shape without the features, False for padded tokens): tokens
        that go to no expert and get the residual alone.  What they hold, NaN too,
        reaches no other token and no weight's gradient."""
        rows, residual, shape = _flat(x, residual, self.in_features, self.out_features)
        if mask is not None:
            closed = ~_token_mask(mask, x)[:, None]
            rows = rows.masked_fill(closed, 0.0)   # (the router's weight gradient has them times 0)
        logits = self.router(rows)
        if mask is not None:
            logits = logits.masked_fill(closed, float("-inf"))
        y = EmuExpertFFNFunction.apply(rows, logits, self.weight_in, self.weight_out, residual, self.k, self.over, self.act,
                                       self.mode)
        return y.reshape(shape)


class EmuExpertFeedForward(torch.nn.Module):
    """The pre-norm sub-layer of experts: x + ffn(norm(x)), with an EmuRMSNorm and
    an EmuExpertFFN."""

    def __init__(self, features, hidden_features, num_experts, k, over="chosen", act="silu", mode="bf16x9", eps=1e-6,
                 device=None, dtype=torch.float32):
        super().__init__()
        self.norm = EmuRMSNorm(features, eps=eps, device=device, dtype=dtype)
        self.ffn = EmuExpertFFN(features, hidden_features, num_experts, k, over=over, act=act, mode=mode, device=device,
                                dtype=dtype)

    def forward(self, x, mask=None):
        rows, _, shape = _flat(x, None, self.norm.features, self.norm.features)
        if mask is None:
            y, s = EmuRMSNormFunction.apply(rows, self.norm.weight, None, self.norm.eps)
        else:   # (what padded tokens hold stays out of the norm's weight gradient too)
            mask, s = _token_mask(mask, x), rows
            y = self.norm(rows.masked_fill(~mask[:, None], 0.0))
        return self.ffn(y, residual=s, mask=mask).reshape(shape)
