"""The experts' operators' host side, without a GPU: the binding matches the
header, argument errors are answered before any device work, and the modules
call what they should."""
import ctypes
import os
import re

import pytest
import torch
import torch.nn.functional as F

import fp32_emulated_gemm_gb300 as emu
from fp32_emulated_gemm_gb300 import build as emu_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, NOT_SUPPORTED = 1, 2
BIG = 2 ** 31


@pytest.fixture(scope="module")
def ex():
    emu_build.build()
    from fp32_emulated_gemm_gb300 import experts
    return experts


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_float * 64)()
    yield (ctypes.cast(buf, ctypes.c_void_p).value + 15) & ~15


def test_binding_signatures_match_the_header(ex):
    header = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "emu_gemm.h")).read(), flags=re.S)
    names = [n for n in emu._EXPERTS if n.startswith("emu_")]
    assert len(names) == 11
    for name in names:
        args = re.search(name + r"\((.*?)\)", header, re.S).group(1).split(",")
        assert args[-1].split()[0] == "emu_stream_t"
        want = "".join("p" if "*" in a else "n" if "int64_t" in a else "f" if "float" in a else "e" for a in args[:-1])
        assert ex._SIGNATURES[name] == want, name
    enum = {m.group(1): int(m.group(2)) for m in re.finditer(r"(EMU_OVER_\w+)\s*=\s*(\d+)", header)}
    assert enum == {"EMU_OVER_" + k.upper(): v for k, v in emu.OVER.items()}
    for name, value in enum.items():
        assert getattr(emu, name) == value


def test_exports():
    for name in emu._EXPERTS:
        assert name in emu.__all__ and getattr(emu, name) is not None


def test_norm_checks(ex, p):
    fn = lambda name, *a: ex._fn(name)(*a, None)
    f = lambda M=4, N=4, X=p, ldx=4, R=None, ldr=0, eps=1e-6, Y=p, ldy=4, S=None, lds=0: fn(
        "emu_rms_norm_fwd", M, N, X, ldx, R, ldr, p, eps, Y, ldy, S, lds, p)
    assert f(M=-1) == INVALID and f(N=-1) == INVALID and f(X=None) == INVALID and f(ldx=3) == INVALID
    assert f(Y=None) == INVALID and f(ldy=3) == INVALID and f(R=p, ldr=3) == INVALID and f(S=p, lds=3) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(N=BIG, ldx=BIG, ldy=BIG) == NOT_SUPPORTED
    assert f(M=0, X=None) == 0 and f(N=0, X=None) == 0
    q = lambda Q=p, ldq=4, s=p, lds=1, N=4: fn("emu_rms_norm_quant", 4, N, p, 400, None, 0, p, 1e-6, Q, ldq, s, lds, None, 0)
    assert q(Q=None) == INVALID and q(ldq=3) == INVALID and q(s=None) == INVALID and q(lds=0) == INVALID
    assert q(N=129, ldq=129, lds=1) == INVALID
    b = lambda M=4, N=4, S=p, r=p, dX=p, lddx=4, add=None, lda=4: fn(
        "emu_rms_norm_bwd", M, N, p, 4, S, 4, p, r, add, lda, dX, lddx, p)
    assert b(M=-1) == INVALID and b(S=None) == INVALID and b(r=None) == INVALID and b(lddx=3) == INVALID
    assert b(dX=None, add=p) == INVALID and b(add=p, lda=3) == INVALID and b(N=BIG) == NOT_SUPPORTED and b(N=0) == 0


def test_router_checks(ex, p):
    fn = lambda name, *a: ex._fn(name)(*a, None)
    r = lambda over=0, M=4, E=4, k=2, logits=p, ldl=4, out=p: fn(
        "emu_expert_route", over, M, E, k, logits, ldl, out, p, p, p, p)
    assert r(over=2) == INVALID and r(over=-1) == INVALID and r(M=-1) == INVALID and r(E=0) == INVALID
    assert r(k=0) == INVALID and r(k=5) == INVALID and r(ldl=3) == INVALID and r(logits=None) == INVALID and r(out=None) == INVALID
    assert r(E=1025, ldl=1025) == NOT_SUPPORTED and r(E=64, k=33, ldl=64) == NOT_SUPPORTED
    assert r(M=2 ** 30, k=2) == NOT_SUPPORTED and r(M=BIG - 256, k=1) == NOT_SUPPORTED
    s = lambda M=4, E=4, k=2, e=p, slots=p: fn("emu_expert_sort", M, E, k, e, slots, p, p)
    assert s(M=-1) == INVALID and s(E=0) == INVALID and s(k=0) == INVALID and s(e=None) == INVALID and s(slots=None) == INVALID
    assert s(E=1025) == NOT_SUPPORTED and s(k=33) == NOT_SUPPORTED and s(M=2 ** 30) == NOT_SUPPORTED
    b = lambda over=0, k=2, logits=p, dl=p, lddl=4, M=4: fn(
        "emu_expert_route_bwd", over, M, 4, k, p, logits, 4, p, p, dl, lddl)
    assert b(over=2) == INVALID and b(k=5) == INVALID and b(dl=None) == INVALID and b(lddl=3) == INVALID
    assert b(over=1, logits=None) == INVALID and b(M=0) == 0 and b(M=0, logits=None) == 0


def test_exchange_checks(ex, p):
    fn = lambda name, *a: ex._fn(name)(*a, None)
    d = lambda M=4, k=2, N=4, X=p, ldx=4, src=p, ldo=4: fn("emu_expert_dispatch", M, k, N, X, ldx, p, src, p, ldo)
    assert d(M=-1) == INVALID and d(k=0) == INVALID and d(N=-1) == INVALID and d(X=None) == INVALID and d(ldx=3) == INVALID
    assert d(src=None) == INVALID and d(ldo=3) == INVALID and d(k=33) == NOT_SUPPORTED and d(M=2 ** 30) == NOT_SUPPORTED
    assert d(M=0) == 0 and d(N=0) == 0
    c = lambda Ys=p, ldys=4, slots=p, R=None, ldr=0, ldy=4: fn("emu_expert_combine_fwd", 4, 2, 4, Ys, ldys, slots, None, R, ldr, p, ldy)
    assert c(Ys=None) == INVALID and c(ldys=3) == INVALID and c(slots=None) == INVALID and c(R=p, ldr=3) == INVALID
    assert c(ldy=3) == INVALID
    b = lambda dY=p, Ys=p, src=p, w=p, dYs=p, lddys=4, dw=p: fn(
        "emu_expert_combine_bwd", 4, 2, 4, dY, 4, Ys, 4, p, src, w, dYs, lddys, dw)
    assert b(dY=None) == INVALID and b(Ys=None) == INVALID and b(src=None) == INVALID and b(w=None) == INVALID
    assert b(lddys=3) == INVALID and b(dYs=None, dw=None) == 0


def test_expert_products_checks(ex, p):
    fn = lambda name, *a: ex._fn(name)(*a, None)
    f = lambda mode=0, act=4, rows=40, E=2, K=4, F=4, N=4, X=p, ldx=4, o=p, ldwi=4, D=None, ldd=0, H=p, ldh=4, Y=p, ldy=4: fn(
        "emu_expert_ffn_fwd", mode, act, rows, E, K, F, N, X, ldx, o, p, ldwi, p, 4, D, ldd, H, ldh, Y, ldy)
    assert f(act=5) == INVALID and f(rows=-1) == INVALID and f(E=0) == INVALID and f(K=0) == INVALID and f(F=0) == INVALID
    assert f(N=0) == INVALID and f(X=None) == INVALID and f(o=None) == INVALID and f(ldx=3) == INVALID and f(ldwi=3) == INVALID
    assert f(H=None) == INVALID and f(ldh=3) == INVALID and f(Y=None) == INVALID and f(ldy=3) == INVALID and f(D=p, ldd=7) == INVALID
    assert f(mode=4) == NOT_SUPPORTED and f(mode=2) == NOT_SUPPORTED and f(mode=9) == NOT_SUPPORTED
    assert f(E=1025) == NOT_SUPPORTED and f(F=2 ** 30, ldh=2 ** 30) == NOT_SUPPORTED and f(rows=BIG) == NOT_SUPPORTED
    assert f(Y=p + 4) == NOT_SUPPORTED and f(ldy=6) == NOT_SUPPORTED and f(ldh=6) == NOT_SUPPORTED and f(D=p + 4, ldd=8) == NOT_SUPPORTED
    assert f(rows=0, X=None) == 0
    # the checks come before the copies of odd operands, which need the device
    assert f(X=p + 4, ldx=5, ldy=6) == NOT_SUPPORTED and f(X=p + 4, ldx=5, ldwi=3) == INVALID
    b = lambda mode=0, dY=p, D=p, dZ=p, dX=p, lddx=4, X=p, dWi=p, lddwi=4, H=p, dWo=p, lddwo=4: fn(
        "emu_expert_ffn_bwd", mode, 40, 2, 4, 4, 4, dY, 4, X, 4, p, p, 4, p, 4, D, 8, H, 4, dZ, 8, dX, lddx, dWi, lddwi, dWo, lddwo)
    assert b(mode=4) == NOT_SUPPORTED and b(dY=None) == INVALID and b(D=None) == INVALID and b(dZ=None) == INVALID
    assert b(lddx=3) == INVALID and b(X=None) == INVALID and b(lddwi=3) == INVALID and b(H=None) == INVALID and b(lddwo=3) == INVALID
    assert b(lddx=6) == NOT_SUPPORTED and b(lddwi=6) == NOT_SUPPORTED and b(dWo=p + 4) == NOT_SUPPORTED
    assert b(D=None, dZ=None, dX=None, dWi=None, lddwo=6) == NOT_SUPPORTED       # what is not wanted needs nothing
    assert b(H=None, dWo=None, X=None, dWi=None, lddx=6) == NOT_SUPPORTED
    assert b(dX=None, dWi=None, dWo=None) == 0


def test_expert_products_sizes_that_overflow(ex, p):
    """Sizes whose products leave 64 bits are refused like other large ones, also
    where there are no rows."""
    fn = lambda name, *a: ex._fn(name)(*a, None)
    for rows in (0, 40):
        for E, K, F, N in ((1, 4, 2 ** 62, 4), (2, 4, 2 ** 62, 4), (1, 4, 2 ** 63 - 4, 4), (4, 4, 4, 2 ** 62), (1, 2 ** 62, 4, 4)):
            assert fn("emu_expert_ffn_fwd", 0, 4, rows, E, K, F, N, p, K, p, p, K, p, F, None, 0, p, F, p, N) == NOT_SUPPORTED
            assert fn("emu_expert_ffn_bwd", 0, rows, E, K, F, N, p, N, p, K, p, p, K, p, F, p, 2 ** 62, p, F, p, 2 ** 62, p, K, None, 0,
                      None, 0) == NOT_SUPPORTED


@pytest.fixture
def plain(monkeypatch):
    """The functional calls replaced by plain ones on the CPU that record how they
    were called."""
    from fp32_emulated_gemm_gb300 import experts as ex
    from fp32_emulated_gemm_gb300 import feed_forward as ff
    made = []

    def linear_act_fwd(X, W, bias=None, *, act="none", residual=None, mode="bf16x9", save=False, out=None):
        return F.linear(X, W, bias)

    def rms_norm_fwd(X, weight=None, *, residual=None, eps=1e-6, save=True, out=None):
        made.append(("rms_norm", save))
        S = X if residual is None else X + residual
        rstd = (S.square().mean(1) + eps).rsqrt()
        Y = S * rstd[:, None] * weight
        return (Y, S, rstd) if save else Y if residual is None else (Y, S)

    def expert_route(logits, k, *, over="chosen"):
        top = torch.topk(logits, k, 1)
        w = torch.softmax(top.values, 1)
        M, E = logits.shape
        e = top.indices.int()
        order = torch.sort(e.reshape(-1), stable=True).indices
        slots = torch.empty(M * k, dtype=torch.int32)
        slots[order] = torch.arange(M * k, dtype=torch.int32)
        offsets = torch.searchsorted(e.reshape(-1)[order].contiguous(), torch.arange(E + 1, dtype=torch.int32))
        return emu.ExpertPlan(e, slots.reshape(M, k), order.int(), offsets.int()), w

    def expert_dispatch(X, plan):
        return X[plan.sources.long() // plan.slots.shape[1]]

    def expert_combine_fwd(Ys, plan, weights=None, *, residual=None, out=None):
        y = (Ys[plan.slots.long()] * weights[:, :, None]).sum(1)
        return y if residual is None else y + residual

    def expert_ffn_fwd(X, W_in, W_out, plan, *, act="silu", mode="bf16x9", save=False):
        made.append(("experts", save))
        o, parts = plan.offsets.tolist(), []
        for e in range(len(W_in)):
            g, u = (X[o[e]:o[e + 1]] @ W_in[e].T).chunk(2, 1)
            parts.append((F.silu(g) * u) @ W_out[e].T)
        Y = torch.cat(parts)
        return (Y, X.new_zeros(len(X), W_in.shape[1]), X.new_zeros(len(X), W_out.shape[2])) if save else Y

    monkeypatch.setattr(ff, "linear_act_fwd", linear_act_fwd)
    for f in (rms_norm_fwd, expert_route, expert_dispatch, expert_combine_fwd, expert_ffn_fwd):
        monkeypatch.setattr(ex, f.__name__, f)
    return made


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_saved_with_gradients_off(plain, off):
    torch.manual_seed(0)
    m, x = emu.EmuExpertFeedForward(6, 8, 4, 2), torch.randn(5, 6)
    trained = m(x)
    assert trained.requires_grad and [s for _, s in plain] == [True, True]
    plain.clear()
    with off():
        y = m(x)
    assert not y.requires_grad and torch.equal(y, trained.detach())
    assert [s for _, s in plain] == [False, False]
    plain.clear()
    m.requires_grad_(False)
    assert not m(x).requires_grad and [s for _, s in plain] == [False, False]


def test_module_shapes_and_refusals(plain):
    m = emu.EmuExpertFFN(6, 8, 4, 2, out_features=5)
    assert m(torch.randn(2, 3, 6)).shape == (2, 3, 5) and m(torch.randn(2, 3, 6), torch.randn(2, 3, 5)).shape == (2, 3, 5)
    assert [tuple(q.shape) for q in m.parameters()] == [(4, 16, 6), (4, 5, 8), (4, 6)]
    for bad in (lambda: m(torch.randn(2, 7)), lambda: m(torch.randn(3, 6), torch.randn(3, 6)),
                lambda: m(torch.randn(2, 3, 6), mask=torch.ones(6, dtype=torch.bool)),
                lambda: m(torch.randn(2, 3, 6), mask=torch.ones(2, 3)),
                lambda: emu.EmuExpertFFN(6, 8, 4, 5), lambda: emu.EmuExpertFFN(6, 8, 4, 0),
                lambda: emu.EmuExpertFFN(6, 8, 4, 2, over="some"), lambda: emu.EmuExpertFFN(6, 8, 4, 2, act="tanh"),
                lambda: emu.EmuExpertFFN(6, 8, 4, 2, mode="fp32"), lambda: emu.EmuRMSNorm(6)(torch.randn(5, 7))):
        with pytest.raises(ValueError):
            bad()
    f = emu.EmuExpertFeedForward(6, 8, 4, 2)
    assert f(torch.randn(2, 3, 6)).shape == (2, 3, 6)
    for mask in (torch.ones(3, 2, dtype=torch.bool), torch.ones(6, dtype=torch.bool), torch.ones(2, 3)):
        with pytest.raises(ValueError):
            f(torch.randn(2, 3, 6), mask)
    n = emu.EmuRMSNorm(6)
    y, s = n(torch.randn(2, 3, 6), torch.randn(2, 3, 6))
    assert y.shape == s.shape == (2, 3, 6) and n(torch.randn(2, 6)).shape == (2, 6)
