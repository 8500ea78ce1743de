"""64-bit values with a bound on what FP32 code may differ from them.

A `V` holds a float64 array and, elementwise, how far a correct FP32
evaluation may be from it.  Each operation computes the exact result of the
values and the first-order bound: what the inputs' own bounds become, plus
the roundings of the operation itself (u = 2^-24).  The tests build an
operator's definition from these, so that every tolerance follows from the
definition, the sizes and the accuracy stated for the products, before
anything runs.
"""
from __future__ import annotations

import numpy as np
from scipy import special

U = 2.0 ** -24


class V:
    def __init__(self, val, err=0.0):
        self.val = np.asarray(val, np.float64)
        self.err = np.broadcast_to(np.asarray(err, np.float64), self.val.shape)

    def __add__(self, o):
        o = as_v(o)
        v = self.val + o.val
        return V(v, self.err + o.err + U * np.abs(v))

    def __sub__(self, o):
        o = as_v(o)
        v = self.val - o.val
        return V(v, self.err + o.err + U * np.abs(v))

    def __mul__(self, o):
        o = as_v(o)
        v = self.val * o.val
        return V(v, self.err * np.abs(o.val) + np.abs(self.val) * o.err + U * np.abs(v))

    @property
    def T(self):
        return V(self.val.T, self.err.T)

    def cols(self, a, b):
        return V(self.val[:, a:b], self.err[:, a:b])

    def check(self, got, what):
        got = np.asarray(got, np.float64)
        assert got.shape == self.val.shape, f"{what}: shape {got.shape}, not {self.val.shape}"
        assert np.all(np.isfinite(got)), f"{what}: {int((~np.isfinite(got)).sum())} values are not finite"
        over = np.abs(got - self.val) - (self.err + U * np.abs(self.val) + 1e-37)
        if over.size and over.max() > 0:
            i = np.unravel_index(int(over.argmax()), over.shape)
            raise AssertionError(f"{what}: at {i} {got[i]!r}, exactly {self.val[i]!r}, allowed {self.err[i]:.3e} "
                                 f"({int((over > 0).sum())} of {over.size} values out of bounds)")


def as_v(x):
    return x if isinstance(x, V) else V(x)


# accuracy of a product in units of u |A||B| per term (include/emu_gemm.h; "+8"
# covers the FP32 chains of very short products)
TERMS = {"bf16x9": lambda k: 2 * k + 8, "tf32x3": lambda k: 4 * k + 8, "fp32": lambda k: k + 8,
         "bf16x6": lambda k: 2 * k + 8 + 16 * 2 ** -20 / U / 16, "tf32x1": lambda k: 2 * k + 8 + 2 ** -10 / U}


def product(A, B, mode, bias=None):
    """A B (+ bias) of 2-D values in an emulated mode."""
    A, B = as_v(A), as_v(B)
    k = A.val.shape[1]
    mag = np.abs(A.val) @ np.abs(B.val)
    v = A.val @ B.val
    if bias is not None:
        v = v + bias
        mag = mag + np.abs(bias)
    return V(v, TERMS[mode](k) * U * mag + A.err @ np.abs(B.val) + np.abs(A.val) @ B.err)


def column_sum(A):
    """Sum over the rows: chains of at most rows / 32 + 96 terms."""
    A = as_v(A)
    m = A.val.shape[0]
    return V(A.val.sum(0), A.err.sum(0) + (m / 32 + 96) * U * np.abs(A.val).sum(0))


# Activations: |a'| <= 1.13 and |a''| <= 0.8 for all of them (relu: no second
# derivative; its jump is handled by the caller).  The FP32 evaluation itself:
# a few units in the last place of z times a factor of at most 1.
def act_value(name, z):
    a, _ = act64(name, z.val)
    return V(a, 1.13 * z.err + 16 * U * np.abs(z.val))


def act_grad(name, z):
    _, d = act64(name, z.val)
    return V(d, 0.8 * z.err + 16 * U * (1 + np.abs(z.val)))


def act64(name, z):
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if name == "silu":
        s = special.expit(z)
        return z * s, s + z * s * special.expit(-z)
    if name == "gelu":
        s = special.ndtr(z)
        return z * s, s + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    k = 2 * np.sqrt(2 / np.pi)
    arg = k * (z + 0.044715 * z ** 3)
    s = special.expit(arg)
    return z * s, s + z * s * special.expit(-arg) * k * (1 + 3 * 0.044715 * z * z)


def layer_norm(x, w, b, eps):
    """(y, xh, rstd) with bounds: sums of at most N / 32 + 16 terms a chain."""
    n = x.shape[1]
    c = 2 * (n / 32 + 16) * U
    mu = x.mean(1, keepdims=True)
    rs = 1 / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + eps)
    xh = V((x - mu) * rs, c * rs * (np.abs(x) + np.abs(x).mean(1, keepdims=True)))
    y = xh if w is None else xh * w
    return (y if b is None else y + b), xh, rs


def layer_norm_grads(dy, x, w, eps, add=None):
    n = x.shape[1]
    c = 3 * (n / 32 + 16) * U
    _, xh, rs = layer_norm(x, w, None, eps)
    dy = as_v(dy)
    g = dy if w is None else dy * w
    gx = g * xh
    mean = lambda a: a.mean(1, keepdims=True)
    v = rs * (g.val - mean(g.val) - xh.val * mean(gx.val))
    mag = np.abs(g.val) + mean(np.abs(g.val)) + np.abs(xh.val) * mean(np.abs(gx.val))
    err = rs * (c * mag + g.err + mean(g.err) + xh.err * np.abs(mean(gx.val)) + np.abs(xh.val) * mean(gx.err))
    dx = V(v, err)
    return (dx if add is None else dx + add), column_sum(dy * xh), column_sum(dy)
