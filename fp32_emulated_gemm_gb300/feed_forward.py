"""Feed-forward operators around the emulated products: layer norm, a linear
layer with bias, activation and residual in one call, and the gated
feed-forward block, each with its backward pass.

Like the rest of the binding, the functions only marshal arguments; the
computation runs in libemu_gemm.so (see ``include/emu_gemm.h`` for the
contract).  Matrices are CUDA float32 with rows of unit column stride (others
are made contiguous first).  The library copies a product's operand whose rows
do not start on 16-byte boundaries; the results of these functions have padded
rows where their width is not a multiple of 4.
"""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import EMU_MODE_BF16X9, EMU_MODE_TF32X3, _check, _mode, _new_c, _ptr, _stream, load

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
EMU_ACT_NONE, EMU_ACT_RELU, EMU_ACT_GELU, EMU_ACT_GELU_TANH, EMU_ACT_SILU = range(5)

# Argument kinds of the C entry points, stream left out: e enum, n int64, f float, p pointer.
_SIGNATURES = {
    "emu_layer_norm_fwd": "nnpnppfpnpp",
    "emu_layer_norm_bwd": "nnpnpnppppnpnpp",
    "emu_linear_act_fwd": "eennnpnpnppnpnpn",
    "emu_linear_act_bwd": "ennnpnpnpnpnpnpnpnp",
    "emu_gated_fwd": "eennnpnpnppnpn",
    "emu_gated_bwd": "ennnpnpnpnpnpnpnpnp",
    "emu_gated_ffn_fwd": "eennnnpnpnppnppnpnpnpn",
    "emu_gated_ffn_bwd": "ennnnpnpnpnpnpnpnpnpnpnppnp",
}
_CTYPES = {"e": ctypes.c_int, "n": ctypes.c_int64, "f": ctypes.c_float, "p": ctypes.c_void_p}
_CAST = {"e": int, "n": int, "f": float, "p": _ptr}
_functions = {}


def _fn(name):
    f = _functions.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes = [_CTYPES[k] for k in _SIGNATURES[name]] + [ctypes.c_void_p]
        f.restype = ctypes.c_int
        _functions[name] = f
    return f



def _c_name(name):
    kinds = _SIGNATURES[name]

    def call(*args, stream=None):
        if len(args) != len(kinds):
            raise TypeError(f"{name} takes {len(kinds)} arguments and a stream")
        _check(_fn(name)(*[_CAST[k](a) for k, a in zip(kinds, args)], _stream(stream)), name)

    call.__name__ = call.__qualname__ = name
    call.__doc__ = f"{name} of include/emu_gemm.h: its arguments in order, then stream=None (the current one)."
    return call


emu_layer_norm_fwd = _c_name("emu_layer_norm_fwd")
emu_layer_norm_bwd = _c_name("emu_layer_norm_bwd")
emu_linear_act_fwd = _c_name("emu_linear_act_fwd")
emu_linear_act_bwd = _c_name("emu_linear_act_bwd")
emu_gated_fwd = _c_name("emu_gated_fwd")
emu_gated_bwd = _c_name("emu_gated_bwd")
emu_gated_ffn_fwd = _c_name("emu_gated_ffn_fwd")
emu_gated_ffn_bwd = _c_name("emu_gated_ffn_bwd")


# ------------------------------------------------------------ arguments ----
# A small call costs as much on the host as on the GPU, so the helpers look at
# each tensor once and hand back what the call needs of it: (tensor, address,
# row stride).  A matrix that is not wanted is (None, None, 0).
_float32, _empty = torch.float32, torch.empty
_NONE = (None, None, 0)
_FUSED = (EMU_MODE_BF16X9, EMU_MODE_TF32X3)  # the modes whose products take the activations in their epilogue


def _act(act):
    try:
        return ACTS[act]
    except KeyError:
        raise ValueError(f"act must be one of {', '.join(ACTS)}") from None


def _rows(t, name, shape=None):
    """`t` as a matrix of unit column stride whose rows do not overlap."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    r, c = t.shape
    if shape is not None and (r, c) != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}, not {r} x {c}")
    if t.is_contiguous():
        return t, t.data_ptr(), c
    if (c > 1 and t.stride(1) != 1) or (r > 1 and t.stride(0) < c):
        t = t.contiguous()
        return t, t.data_ptr(), c
    return t, t.data_ptr(), t.stride(0) if r > 1 else c


def _pad4(n):
    return (n + 3) // 4 * 4


def _vector(t, name, n):
    """(tensor, address) of a vector."""
    if t is None:
        return None, None
    if not isinstance(t, torch.Tensor) or t.dtype is not _float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be a vector of {n}")
    if not t.is_contiguous():
        t = t.contiguous()
    return t, t.data_ptr()


def _new(M, N, device):
    """A new matrix with rows on 16-byte boundaries."""
    t = _empty((M, N), device=device, dtype=_float32) if not N & 3 else _new_c(M, N, device)
    return t, t.data_ptr(), _pad4(N)


def _new_vector(n, device):
    t = _empty(n, device=device, dtype=_float32)
    return t, t.data_ptr()


def _result(out, shape, device, name):
    if out is None:
        return _new(*shape, device)
    if not isinstance(out, torch.Tensor) or out.dtype is not _float32 or not out.is_cuda:
        raise TypeError(f"{name} must be a CUDA float32 tensor")
    if tuple(out.shape) != shape or (shape[1] > 1 and out.stride(1) != 1) or (shape[0] > 1 and out.stride(0) < shape[1]):
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]} with unit column stride")
    return out, out.data_ptr(), out.stride(0) if shape[0] > 1 else _pad4(shape[1])


def _stream_of(name, *tensors):
    """The current stream, for tensors that have to be on the current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: all tensors must be on the current device (cuda:{dev})")
    return _raw_stream(dev)


# (the Stream object that torch.cuda.current_stream builds costs 3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# ----------------------------------------------------------- layer norm ----
def layer_norm_fwd(X, weight=None, bias=None, *, eps=1e-5, save=True, out=None):
    """(Y, mean, rstd), or Y alone without `save`: Y = (X - mean) * rstd * weight
    + bias over the rows of X; layer_norm_bwd wants the other two."""
    X, px, ldx = _rows(X, "X")
    M, N = X.shape
    weight, pw = _vector(weight, "weight", N)
    bias, pb = _vector(bias, "bias", N)
    device = X.device
    if out is None:
        Y, ldy = _empty((M, N), device=device, dtype=_float32), N
        py = Y.data_ptr()
    else:
        Y, py, ldy = _result(out, (M, N), device, "out")
    mean = rstd = pm = pr = None
    if save:
        mean, pm = _new_vector(M, device)
        rstd, pr = _new_vector(M, device)
    _check(_fn("emu_layer_norm_fwd")(M, N, px, ldx, pw, pb, eps, py, ldy, pm, pr,
                                     _stream_of("layer_norm_fwd", X, weight, bias, Y)), "emu_layer_norm_fwd")
    return (Y, mean, rstd) if save else Y


def layer_norm_bwd(dY, X, weight, mean, rstd, *, add=None, need_input=True, need_params=True):
    """(dX, dweight, dbias) of layer_norm_fwd; `add` (a gradient that reaches X
    by another way) is added to dX.  What is not needed comes back as None."""
    X, px, ldx = _rows(X, "X")
    M, N = shape = tuple(X.shape)
    dY, pdy, lddy = _rows(dY, "dY", shape)
    add, pa, lda = _NONE if add is None else _rows(add, "add", shape)
    if add is not None and not need_input:
        raise ValueError("add needs dX")
    weight, pw = _vector(weight, "weight", N)
    mean, pm = _vector(mean, "mean", M)
    rstd, pr = _vector(rstd, "rstd", M)
    device = X.device
    dX = pdx = dw = pdw = db = pdb = None
    if need_input:
        dX = _empty(shape, device=device, dtype=_float32)
        pdx = dX.data_ptr()
    if need_params:
        dw, pdw = _new_vector(N, device)
        db, pdb = _new_vector(N, device)
    _check(_fn("emu_layer_norm_bwd")(M, N, pdy, lddy, px, ldx, pw, pm, pr, pa, lda, pdx, N, pdw, pdb,
                                     _stream_of("layer_norm_bwd", X, dY, weight, mean, rstd, add)), "emu_layer_norm_bwd")
    return dX, dw, db


# ----------------------------------------------------------- linear_act ----
def linear_act_fwd(X, W, bias=None, *, act="none", residual=None, mode="bf16x9", save=False, out=None):
    """Y = act(Z) + residual with Z = X W^T + bias (X [M,K], W [N,K]); with
    `save` (Y, D) for linear_act_bwd, D = act'(Z) (None for act "none")."""
    mode = _mode(mode)
    X, px, ldx = _rows(X, "X")
    W, pw, ldw = _rows(W, "W")
    M, K = X.shape
    N, Kw = W.shape
    if Kw != K:
        raise ValueError("inner dimensions differ")
    a = _act(act)
    bias, pb = _vector(bias, "bias", N)
    residual, pr, ldr = _NONE if residual is None else _rows(residual, "residual", (M, N))
    device = X.device
    Y, py, ldy = _result(out, (M, N), device, "out")
    D, pd, ldd = _new(M, N, device) if save and a != EMU_ACT_NONE else _NONE
    _check(_fn("emu_linear_act_fwd")(mode, a, M, N, K, px, ldx, pw, ldw, pb, pr, ldr, pd, ldd, py, ldy,
                                     _stream_of("linear_act_fwd", X, W, bias, residual, Y)), "emu_linear_act_fwd")
    return (Y, D) if save else Y


def linear_act_bwd(dY, X, W, D=None, *, act="none", mode="bf16x9", need=(True, True, True)):
    """(dX, dW, dbias) of linear_act_fwd from its D, which act "none" does not
    read (the residual's gradient is dY).  `need` says which are wanted; the
    others are None."""
    X, px, ldx = _rows(X, "X")
    W, pw, ldw = _rows(W, "W")
    M, K = X.shape
    N, Kw = W.shape
    if Kw != K:
        raise ValueError("inner dimensions differ")
    dY, pdy, lddy = _rows(dY, "dY", (M, N))
    device = X.device
    pd, ldd, pdz, lddz = None, 0, None, 0
    if _act(act) != EMU_ACT_NONE:
        if D is None:
            raise ValueError(f"act {act!r} needs D")
        D, pd, ldd = _rows(D, "D", (M, N))
        dZ, pdz, lddz = _new(M, N, device)
    else:
        D = None
    dX, pdx, lddx = _new(M, K, device) if need[0] else _NONE
    dW, pdw, lddw = _new(N, K, device) if need[1] else _NONE
    db, pdb = _new_vector(N, device) if need[2] else (None, None)
    _check(_fn("emu_linear_act_bwd")(_mode(mode), M, N, K, pdy, lddy, px, ldx, pw, ldw, pd, ldd, pdz, lddz, pdx, lddx,
                                     pdw, lddw, pdb, _stream_of("linear_act_bwd", dY, X, W, D)), "emu_linear_act_bwd")
    return dX, dW, db


# ---------------------------------------------------------------- gated ----
def _gated_shapes(X, W):
    (M, K), (F2, Kw) = X.shape, W.shape
    if F2 % 2:
        raise ValueError("W must have the gate's rows, then as many of the up projection")
    if Kw != K:
        raise ValueError("inner dimensions differ")
    return M, K, F2 // 2


def gated_fwd(X, W, bias=None, *, act="silu", mode="bf16x9", save=False):
    """H = act(G) * U with [G | U] = X W^T + bias (X [M,K]; W [2F,K]: the
    gate's rows, then the up projection's); with `save` (H, D) for
    gated_bwd, D = [U act'(G) | act(G)]."""
    mode = _mode(mode)
    X, px, ldx = _rows(X, "X")
    W, pw, ldw = _rows(W, "W")
    M, K, F = _gated_shapes(X, W)
    bias, pb = _vector(bias, "bias", 2 * F)
    H, ph, ldh = _new(M, F, X.device)
    D, pd, ldd = _new(M, 2 * F, X.device) if save or mode not in _FUSED else _NONE
    _check(_fn("emu_gated_fwd")(mode, _act(act), M, F, K, px, ldx, pw, ldw, pb, pd, ldd, ph, ldh,
                                _stream_of("gated_fwd", X, W, bias)), "emu_gated_fwd")
    return (H, D) if save else H


def gated_bwd(dH, X, W, D, *, act="silu", mode="bf16x9", need=(True, True, True)):
    """(dX, dW, dbias) of gated_fwd from its D; `need` says which are wanted.
    (D holds the activation's part; `act` only has to name one.)"""
    _act(act)
    X, px, ldx = _rows(X, "X")
    W, pw, ldw = _rows(W, "W")
    M, K, F = _gated_shapes(X, W)
    dH, pdh, lddh = _rows(dH, "dH", (M, F))
    D, pd, ldd = _rows(D, "D", (M, 2 * F))
    device = X.device
    dZ, pdz, lddz = _new(M, 2 * F, device)
    dX, pdx, lddx = _new(M, K, device) if need[0] else _NONE
    dW, pdw, lddw = _new(2 * F, K, device) if need[1] else _NONE
    db, pdb = _new_vector(2 * F, device) if need[2] else (None, None)
    _check(_fn("emu_gated_bwd")(_mode(mode), M, F, K, pdh, lddh, px, ldx, pw, ldw, pd, ldd, pdz, lddz, pdx,
                                lddx, pdw, lddw, pdb, _stream_of("gated_bwd", dH, X, W, D)), "emu_gated_bwd")
    return dX, dW, db


def _ffn_shapes(X, W_in, W_out):
    M, K, F = _gated_shapes(X, W_in)
    if W_out.shape[1] != F:
        raise ValueError("W_out must have one column per gated feature")
    return M, K, F, W_out.shape[0]


def gated_ffn_fwd(X, W_in, b_in, W_out, b_out, *, act="silu", residual=None, mode="bf16x9", save=False, out=None):
    """Y = H W_out^T + b_out + residual with H = gated_fwd(X, W_in, b_in)
    (X [M,K], W_in [2F,K], W_out [N,F]; the biases and the residual may be
    None); with `save` (Y, D, H) for gated_ffn_bwd."""
    mode = _mode(mode)
    X, px, ldx = _rows(X, "X")
    W_in, pwi, ldwi = _rows(W_in, "W_in")
    W_out, pwo, ldwo = _rows(W_out, "W_out")
    M, K, F, N = _ffn_shapes(X, W_in, W_out)
    b_in, pbi = _vector(b_in, "b_in", 2 * F)
    b_out, pbo = _vector(b_out, "b_out", N)
    residual, pr, ldr = _NONE if residual is None else _rows(residual, "residual", (M, N))
    device = X.device
    Y, py, ldy = _result(out, (M, N), device, "out")
    H, ph, ldh = _new(M, F, device)
    D, pd, ldd = _new(M, 2 * F, device) if save or mode not in _FUSED else _NONE
    s = _stream_of("gated_ffn_fwd", X, W_in, b_in, W_out, b_out, residual, Y)
    _check(_fn("emu_gated_ffn_fwd")(mode, _act(act), M, K, F, N, px, ldx, pwi, ldwi, pbi, pwo, ldwo, pbo, pr, ldr,
                                    pd, ldd, ph, ldh, py, ldy, s), "emu_gated_ffn_fwd")
    return (Y, D, H) if save else Y


def gated_ffn_bwd(dY, X, W_in, W_out, D, H, *, act="silu", mode="bf16x9", need=(True, True, True, True, True)):
    """(dX, dW_in, db_in, dW_out, db_out) of gated_ffn_fwd from its D and H
    (the residual's gradient is dY); `need` says which are wanted.  (D holds the
    activation's part; `act` only has to name one.)  D may be None where only
    dW_out and db_out are wanted, H where dW_out is not."""
    _act(act)
    X, px, ldx = _rows(X, "X")
    W_in, pwi, ldwi = _rows(W_in, "W_in")
    W_out, pwo, ldwo = _rows(W_out, "W_out")
    M, K, F, N = _ffn_shapes(X, W_in, W_out)
    dY, pdy, lddy = _rows(dY, "dY", (M, N))
    inner = any(need[:3])
    D, pd, ldd = _rows(D, "D", (M, 2 * F)) if inner or D is not None else _NONE
    H, ph, ldh = _rows(H, "H", (M, F)) if need[3] or H is not None else _NONE
    device = X.device
    dZ, pdz, lddz = _new(M, 2 * F, device) if inner else _NONE
    dX, pdx, lddx = _new(M, K, device) if need[0] else _NONE
    dWi, pdwi, lddwi = _new(2 * F, K, device) if need[1] else _NONE
    dbi, pdbi = _new_vector(2 * F, device) if need[2] else (None, None)
    dWo, pdwo, lddwo = _new(N, F, device) if need[3] else _NONE
    dbo, pdbo = _new_vector(N, device) if need[4] else (None, None)
    s = _stream_of("gated_ffn_bwd", dY, X, W_in, W_out, D, H)
    _check(_fn("emu_gated_ffn_bwd")(_mode(mode), M, K, F, N, pdy, lddy, px, ldx, pwi, ldwi, pwo, ldwo, pd, ldd,
                                    ph, ldh, pdz, lddz, pdx, lddx, pdwi, lddwi, pdbi, pdwo, lddwo, pdbo, s),
           "emu_gated_ffn_bwd")
    return dX, dWi, dbi, dWo, dbo


# ------------------------------------------------------------- autograd ----
class _Function(torch.autograd.Function):
    """With gradients off, or wanted by no argument, `apply` is the call itself,
    which stores nothing for a backward pass.  (needs_input_grad cannot tell: it
    is set for parameters with gradients off too, and inside `forward` they are
    always off.)"""

    @classmethod
    def apply(cls, *args):
        if torch.is_grad_enabled() and any(isinstance(a, torch.Tensor) and a.requires_grad for a in args):
            return super().apply(*args)
        return cls.infer(*args)


class EmuLayerNormFunction(_Function):
    @staticmethod
    def infer(X, weight, bias, eps):
        return layer_norm_fwd(X, weight, bias, eps=eps, save=False)

    @staticmethod
    def forward(ctx, X, weight, bias, eps):
        Y, mean, rstd = layer_norm_fwd(X, weight, bias, eps=eps)
        ctx.save_for_backward(X, weight, mean, rstd)
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dX, dw, db = layer_norm_bwd(dY, X, weight, mean, rstd, need_input=need[0], need_params=need[1] or need[2])
        return dX, dw if need[1] else None, db if need[2] else None, None


class EmuLinearActFunction(_Function):
    @staticmethod
    def infer(X, W, bias, residual, act, mode):
        return linear_act_fwd(X, W, bias, act=act, residual=residual, mode=mode)

    @staticmethod
    def forward(ctx, X, W, bias, residual, act, mode):
        save = act != "none" and any(ctx.needs_input_grad[:3])
        r = linear_act_fwd(X, W, bias, act=act, residual=residual, mode=mode, save=save)
        Y, D = r if save else (r, None)
        ctx.save_for_backward(X, W, D)
        ctx.act, ctx.mode = act, mode
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, W, D = ctx.saved_tensors
        need = ctx.needs_input_grad
        dX = dW = db = None
        if any(need[:3]):
            dX, dW, db = linear_act_bwd(dY, X, W, D, act=ctx.act, mode=ctx.mode, need=need[:3])
        return dX, dW, db, dY if need[3] else None, None, None


class EmuGatedFFNFunction(_Function):
    @staticmethod
    def infer(X, W_in, b_in, W_out, b_out, residual, act, mode):
        return gated_ffn_fwd(X, W_in, b_in, W_out, b_out, act=act, residual=residual, mode=mode)

    @staticmethod
    def forward(ctx, X, W_in, b_in, W_out, b_out, residual, act, mode):
        save = any(ctx.needs_input_grad[:5])
        r = gated_ffn_fwd(X, W_in, b_in, W_out, b_out, act=act, residual=residual, mode=mode, save=save)
        Y, D, H = r if save else (r, None, None)
        ctx.save_for_backward(X, W_in, W_out, D, H)
        ctx.act, ctx.mode = act, mode
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, W_in, W_out, D, H = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = (None,) * 5
        if any(need[:5]):
            grads = gated_ffn_bwd(dY, X, W_in, W_out, D, H, act=ctx.act, mode=ctx.mode, need=need[:5])
        return (*grads, dY if need[5] else None, None, None)


class EmuFeedForwardFunction(_Function):
    """x + gated_ffn(layer_norm(x)): the residual's gradient joins in the norm's
    backward pass."""

    @staticmethod
    def infer(X, norm_weight, norm_bias, W_in, b_in, W_out, b_out, eps, act, mode):
        Xn = layer_norm_fwd(X, norm_weight, norm_bias, eps=eps, save=False)
        return gated_ffn_fwd(Xn, W_in, b_in, W_out, b_out, act=act, residual=X, mode=mode)

    @staticmethod
    def forward(ctx, X, norm_weight, norm_bias, W_in, b_in, W_out, b_out, eps, act, mode):
        save = any(ctx.needs_input_grad[:7])
        Xn, mean, rstd = layer_norm_fwd(X, norm_weight, norm_bias, eps=eps)
        r = gated_ffn_fwd(Xn, W_in, b_in, W_out, b_out, act=act, residual=X, mode=mode, save=save)
        Y, D, H = r if save else (r, None, None)
        ctx.save_for_backward(X, norm_weight, mean, rstd, Xn, W_in, W_out, D, H)
        ctx.act, ctx.mode = act, mode
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, norm_weight, mean, rstd, Xn, W_in, W_out, D, H = ctx.saved_tensors
        need = ctx.needs_input_grad
        dX = dnw = dnb = None
        inner = any(need[:3])
        dXn, *grads = gated_ffn_bwd(dY, Xn, W_in, W_out, D, H, act=ctx.act, mode=ctx.mode, need=(inner, *need[3:7]))
        if inner:
            dX, dnw, dnb = layer_norm_bwd(dXn, X, norm_weight, mean, rstd, add=dY if need[0] else None,
                                          need_input=need[0], need_params=need[1] or need[2])
        return (dX, dnw if need[1] else None, dnb if need[2] else None, *grads, None, None, None)


class EmuLayerNorm(torch.nn.LayerNorm):
    """Drop-in nn.LayerNorm on the library's kernels."""

    def forward(self, x):
        n = 1
        for d in self.normalized_shape:
            n *= d
        if tuple(x.shape[x.dim() - len(self.normalized_shape):]) != tuple(self.normalized_shape):
            raise ValueError(f"the input must end in {tuple(self.normalized_shape)}")
        flat = [None if p is None else p.reshape(n) for p in (self.weight, self.bias)]
        rows = x.numel() // n if n else 0
        return EmuLayerNormFunction.apply(x.reshape(rows, n), *flat, self.eps).reshape(x.shape)


def _flat(x, residual, in_features, out_features):
    """(rows of x, rows of the residual, shape of the result).  The residual has
    that shape, or is the matrix of its rows."""
    if x.dim() < 1 or x.shape[-1] != in_features:
        raise ValueError(f"the input must have {in_features} features, not shape {tuple(x.shape)}")
    shape = (*x.shape[:-1], out_features)
    rows = math.prod(shape[:-1])
    if residual is not None:
        if tuple(residual.shape) not in (shape, (rows, out_features)):
            raise ValueError(f"the residual must be {tuple(shape)}, not {tuple(residual.shape)}")
        residual = residual.reshape(rows, out_features)
    return x.reshape(rows, in_features), residual, shape


class EmuLinearAct(torch.nn.Linear):
    """nn.Linear with an activation and an optional residual:
    act(x W^T + b) + residual."""

    def __init__(self, in_features, out_features, bias=True, act="gelu", mode="bf16x9", **kw):
        _act(act), _mode(mode)
        super().__init__(in_features, out_features, bias=bias, **kw)
        self.act, self.mode = act, mode

    def forward(self, x, residual=None):
        x, residual, shape = _flat(x, residual, self.in_features, self.out_features)
        return EmuLinearActFunction.apply(x, self.weight, self.bias, residual, self.act, self.mode).reshape(shape)


class EmuGatedFFN(torch.nn.Module):
    """The gated feed-forward block act(x Wg^T + bg) * (x Wu^T + bu), projected
    back by W_out: weight_in holds Wg's rows, then Wu's."""

    def __init__(self, in_features, hidden_features, out_features=None, bias=True, act="silu", mode="bf16x9",
                 device=None, dtype=torch.float32):
        super().__init__()
        _act(act), _mode(mode)
        out_features = in_features if out_features is None else out_features
        self.in_features, self.hidden_features, self.out_features = in_features, hidden_features, out_features
        self.act, self.mode = act, mode
        new = lambda *s: torch.nn.Parameter(torch.empty(s, device=device, dtype=dtype))
        self.weight_in, self.weight_out = new(2 * hidden_features, in_features), new(out_features, hidden_features)
        self.bias_in = new(2 * hidden_features) if bias else None
        self.bias_out = new(out_features) if bias else None
        self.reset_parameters()

    def reset_parameters(self):
        """nn.Linear's initial values, for each of the three projections."""
        for w, b in ((self.weight_in, self.bias_in), (self.weight_out, self.bias_out)):
            bound = w.shape[1] ** -0.5 if w.shape[1] else 0.0
            torch.nn.init.uniform_(w, -bound, bound)
            if b is not None:
                torch.nn.init.uniform_(b, -bound, bound)

    def forward(self, x, residual=None):
        x, residual, shape = _flat(x, residual, self.in_features, self.out_features)
        y = EmuGatedFFNFunction.apply(x, self.weight_in, self.bias_in, self.weight_out, self.bias_out, residual, self.act,
                                      self.mode)
        return y.reshape(shape)


class EmuFeedForward(torch.nn.Module):
    """The pre-norm feed-forward sub-layer of a transformer:
    x + ffn(norm(x)), with an EmuLayerNorm and an EmuGatedFFN."""

    def __init__(self, features, hidden_features, bias=True, act="silu", mode="bf16x9", eps=1e-5, device=None,
                 dtype=torch.float32):
        super().__init__()
        self.norm = EmuLayerNorm(features, eps=eps, device=device, dtype=dtype)
        self.ffn = EmuGatedFFN(features, hidden_features, bias=bias, act=act, mode=mode, device=device, dtype=dtype)

    def forward(self, x):
        f = self.ffn
        x, _, shape = _flat(x, None, f.in_features, f.out_features)
        y = EmuFeedForwardFunction.apply(x, self.norm.weight, self.norm.bias, f.weight_in, f.bias_in, f.weight_out,
                                         f.bias_out, self.norm.eps, f.act, f.mode)
        return y.reshape(shape)
