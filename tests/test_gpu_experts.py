"""The operators of a layer of experts against their definitions in 64 bits.

Tolerances are running error bounds (tests/_running.py): the roundings of a
definition's own operations and the products' stated accuracy, before anything
runs.  Choices, places and copies have to be equal.
"""
import numpy as np
import pytest

from tests import _gpu
from tests import _running as R
from tests._running import U, V
from tests.test_gpu_feed_forward import dev, done, f32, host, rng_of

pytestmark = pytest.mark.gpu
EPS = 1e-6
INF = float("inf")


def ints(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(_gpu.device())


def padded(x, left=0, right=3, fill=np.nan):
    """A device view of x whose rows start `left` words into rows of other values."""
    buf = np.full((x.shape[0] + 2, left + x.shape[1] + right), fill, np.float32)
    buf[1:-1, left:left + x.shape[1]] = x
    return _gpu.to_dev(buf)[1:-1, left:left + x.shape[1]]


# --------------------------------------------------------------- RMS norm --
def norm_terms(n):
    """Relative error of 1 / sqrt(mean s^2 + eps): half the sum's (chains of at
    most n / 32 + 16 positive terms) and the operations around it."""
    return (n / 64 + 16) * U


def rms_norm(x, q, w):
    """(Y, S, rstd) with bounds; S is one rounding."""
    s = V(x.astype(np.float64)) if q is None else V(x) + q
    n = x.shape[1]
    r = 1 / np.sqrt((s.val ** 2).mean(1, keepdims=True) + EPS)
    y = s.val * r * (1 if w is None else w.astype(np.float64))
    return V(y, np.abs(y) * (norm_terms(n) + 4 * U) + np.abs(r * (1 if w is None else w)) * s.err), s, r[:, 0]


def rms_grads(dy, s, w, rstd, add):
    """(dX, dweight) with bounds, of the S and rstd that the call was given."""
    n = s.shape[1]
    c = 3 * (n / 32 + 16) * U
    h = V(s * rstd[:, None], U * np.abs(s * rstd[:, None]))
    g = V(dy) if w is None else V(dy) * w
    m = (g.val * h.val).mean(1, keepdims=True)
    mag = np.abs(g.val) + np.abs(h.val) * np.abs(g.val * h.val).mean(1, keepdims=True)
    dx = V(rstd[:, None] * (g.val - h.val * m), rstd[:, None] * c * mag)
    return dx if add is None else dx + add, R.column_sum(V(dy) * h)


def check_quant(y, Q, scales):
    """e4m3 of y / scale: half a step of the value (2^-4 of it) or, below e4m3's
    smallest normal number 2^-6, of its steps of 2^-9; the scale the smallest power
    of two that keeps the group in range (either of two where y's bound leaves it open)."""
    M, N = y.val.shape
    wide = np.repeat(scales.astype(np.float64), 128, 1)[:, :N]
    assert np.all(np.log2(scales) == np.round(np.log2(scales))) and scales.min() >= 2.0 ** -126
    over = np.abs(Q * wide - y.val) - (2.0 ** -4 * (np.abs(y.val) + y.err) + 2.0 ** -10 * wide + y.err)
    assert over.max() <= 0, f"Q: {int((over > 0).sum())} values off"
    for g in range(scales.shape[1]):
        cut = slice(128 * g, 128 * g + 128)
        top, err = np.abs(y.val[:, cut]).max(1), y.err[:, cut].max(1)
        f = scales[:, g].astype(np.float64)
        assert np.all(top - err <= 448 * f) and np.all((top + err > 224 * f) | (f == 2.0 ** -126)), f"scales of group {g}"


RMS_SHAPES = [(1, 1), (3, 2), (65, 4), (50, 16), (77, 13), (33, 17), (130, 32), (5, 31), (129, 61), (33, 64), (40, 128),
              (7, 129), (1, 256), (192, 256), (700, 257), (65, 512), (40, 1000), (37, 1001), (9, 1024), (20, 2048), (12, 2050),
              (5, 4096), (3, 8192), (4, 9001), (3, 16384), (2, 16383), (2, 20000), (2, 40003)]


@pytest.mark.parametrize("M,N", RMS_SHAPES)
@pytest.mark.parametrize("kind", ["all", "plain", "odd"])
def test_rms_norm(M, N, kind):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("rms", M, N)
    x = (f32(rng, M, N, std=1.5, mean=0.5) * np.exp(f32(rng, N, std=0.5))).astype(np.float32)
    q, w = (f32(rng, M, N), f32(rng, N, std=0.2, mean=1.0)) if kind != "plain" else (None, None)
    dy, add = f32(rng, M, N), f32(rng, M, N)
    put = (lambda a: None if a is None else padded(a, 1)) if kind == "odd" else dev
    want, s64, r64 = rms_norm(x, q, w)
    y, s, rstd = emu.rms_norm_fwd(put(x), dev(w), residual=put(q), eps=EPS)
    only = emu.rms_norm_fwd(put(x), dev(w), residual=put(q), eps=EPS, save=False)
    Q, scales, *more = emu.rms_norm_quant(put(x), dev(w), residual=put(q), eps=EPS)
    dx, dw = emu.rms_norm_bwd(put(dy), s, dev(w), rstd, add=put(add))
    dx0, none = emu.rms_norm_bwd(put(dy), s, dev(w), rstd, need_weight=False)
    none2, dw1 = emu.rms_norm_bwd(put(dy), s, dev(w), rstd, need_input=False)
    done()
    want.check(host(y), "Y")
    V(r64, r64 * norm_terms(N)).check(host(rstd), "rstd")
    s64.check(host(s), "S")
    if q is None:
        only, stream = (only, s), []
    else:
        stream = more
        assert len(more) == 1
    assert none is None and none2 is None and not np.any(host(only[0]) != host(y)) and not np.any(host(only[1]) != host(s))
    for t in stream:
        s64.check(host(t), "S beside Q")
    check_quant(want, host(Q.float()).astype(np.float64), host(scales))
    sg, rg, w64 = host(s).astype(np.float64), host(rstd).astype(np.float64), None if w is None else w.astype(np.float64)
    want_dx, want_dw = rms_grads(dy, sg, w64, rg, add)
    want_dx.check(host(dx), "dX")
    want_dw.check(host(dw), "dweight")
    want_dw.check(host(dw1), "dweight alone")
    rms_grads(dy, sg, w64, rg, None)[0].check(host(dx0), "dX without add")


@pytest.mark.parametrize("N", [7, 256, 1001, 5000, 17000])
def test_rms_norm_quant_keeps_nan_in_its_row(N):
    """A NaN makes its row NaN, an infinity itself (as the FP32 output's); the other
    rows and all scales are as without them."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("nanquant", N)
    x = f32(rng, 5, N)
    want = [host(t.float()) for t in emu.rms_norm_quant(dev(x), eps=EPS)]
    x[1, N // 2], x[3, N - 1] = np.nan, INF
    y = host(emu.rms_norm_fwd(dev(x), eps=EPS, save=False))
    Q, s = (host(t.float()) for t in emu.rms_norm_quant(dev(x), eps=EPS))
    done()
    assert np.isnan(Q[1]).all() and np.isnan(y[1]).all() and np.array_equal(np.isnan(Q[3]), np.isnan(y[3])) and np.isnan(Q[3, N - 1])
    keep = [0, 2, 4]
    assert np.array_equal(Q[keep], want[0][keep]) and np.array_equal(s[keep], want[1][keep]) and np.isfinite(s).all()


@pytest.mark.parametrize("N", [7, 256, 1001, 5000, 17000])
def test_rms_norm_hard_rows(N):
    """Rows that are zero, constant, huge, tiny, or hold one outlier; a residual
    that cancels; NaN stays in its row."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("hardrms", N)
    x = np.stack([np.zeros(N), np.full(N, 7.0), f32(rng, N) * 1e15, f32(rng, N) * 1e-15, f32(rng, N) + 4096.0,
                  np.where(np.arange(N) == N // 2, 1e6, 1e-3), f32(rng, N) * 1e-30]).astype(np.float32)
    w, dy = f32(rng, N, mean=1.0, std=0.1), f32(rng, len(x), N)
    want, s64, _ = rms_norm(x, None, w)
    y, s, rstd = emu.rms_norm_fwd(dev(x), dev(w), eps=EPS)
    Q, scales = emu.rms_norm_quant(dev(x), dev(w), eps=EPS)
    dx, dw = emu.rms_norm_bwd(dev(dy), s, dev(w), rstd)
    cancel = emu.rms_norm_fwd(dev(x), dev(w), residual=dev(-x), eps=EPS, save=False)
    bad = x.copy()
    bad[3, N // 3] = np.nan
    yb = host(emu.rms_norm_fwd(dev(bad), dev(w), eps=EPS, save=False))
    done()
    want.check(host(y), "Y")
    check_quant(want, host(Q.float()).astype(np.float64), host(scales))
    for got, ref, name in zip((dx, dw), rms_grads(dy, x.astype(np.float64), w, host(rstd).astype(np.float64), None), ("dX", "dw")):
        ref.check(host(got), name)
    assert not np.any(host(cancel[0])) and not np.any(host(cancel[1]))
    assert np.isnan(yb[3]).all() and np.array_equal(np.delete(yb, 3, 0), np.delete(host(y), 3, 0))


@pytest.mark.parametrize("N", [7, 256, 1001, 5000, 17000])
def test_rms_norm_of_rows_whose_squares_overflow(N):
    """The sum of squares is infinite: 1 / sqrt of it is 0, and so are the row, its
    gradient and its part of the weight's; an infinity itself becomes NaN."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("overflow", N)
    x, dy = f32(rng, 4, N), f32(rng, 4, N)
    x[1, N // 2], x[2], x[3, 0] = 1e30, 1.7e19, INF   # (one square beyond FP32's range; the sum of all; infinity)
    y, s, rstd = emu.rms_norm_fwd(dev(x), eps=EPS)
    Q, scales = emu.rms_norm_quant(dev(x), eps=EPS)
    dx, dw = emu.rms_norm_bwd(dev(dy[:3]), s[:3], None, rstd[:3])
    dx0, dw0 = emu.rms_norm_bwd(dev(dy[:1]), s[:1], None, rstd[:1])
    done()
    y, Q, r = host(y), host(Q.float()), host(rstd)
    assert np.isfinite(r).all() and not r[1:].any() and r[0] > 0
    assert not y[1:3].any() and not Q[1:3].any() and not y[3, 1:].any() and np.isnan(y[3, 0]) and np.isnan(Q[3, 0])
    assert np.isfinite(host(scales)).all()
    assert not host(dx)[1:].any() and np.array_equal(host(dx)[0], host(dx0)[0]) and np.array_equal(host(dw), host(dw0))


def test_rms_norm_many_rows_and_repeatable():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("manyrms")
    M, N = 30011, 96
    x, q, dy, w = f32(rng, M, N, mean=0.3), f32(rng, M, N), f32(rng, M, N), f32(rng, N)
    y, s, rstd = emu.rms_norm_fwd(dev(x), dev(w), residual=dev(q), eps=EPS)
    first = emu.rms_norm_bwd(dev(dy), s, dev(w), rstd, add=dev(q))
    again = emu.rms_norm_bwd(dev(dy), s, dev(w), rstd, add=dev(q))
    done()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    rms_norm(x, q, w)[0].check(host(y), "Y")
    want = rms_grads(dy, host(s).astype(np.float64), w, host(rstd).astype(np.float64), q)
    want[0].check(host(first[0]), "dX")
    want[1].check(host(first[1]), "dweight")


# ----------------------------------------------------------------- router --
def sort_oracle(experts, E):
    M, k = experts.shape
    flat = experts.reshape(-1)
    sent = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(sent, flat, E), kind="stable")[:sent.sum()]
    slots, sources = np.full(M * k, -1), np.full(M * k, -1)
    slots[order] = np.arange(len(order))
    sources[:len(order)] = order
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[sent], minlength=E))])
    return slots.reshape(M, k), sources, offsets


def route_oracle(l, k, over):
    """(experts, weights with bounds): softmax over fewer than E + k terms, each
    exp of a difference (its rounding times exp's argument) and exp's own error."""
    M, E = l.shape
    l = l.astype(np.float64)
    order = np.argsort(-l, axis=1, kind="stable")[:, :k]
    v = np.take_along_axis(l, order, 1)
    open_ = v > -INF
    experts = np.where(open_, order, -1)
    top = np.where(open_[:, :1], v[:, :1], 0)
    e = np.where(open_, np.exp(v - top), 0)
    total = e.sum(1, keepdims=True) if over == "chosen" else np.exp(l - top).sum(1, keepdims=True)
    w = np.divide(e, total, out=np.zeros_like(e), where=open_)
    span = np.where(open_, top - v, 0).max(1, keepdims=True)
    rel = (span + (k if over == "chosen" else E) + 16) * U
    if over == "all":   # a term's difference is rounded in proportion to it, and exp's small values weigh little: x e^-x <= 1
        rel = rel + U
    return experts, V(w, rel * w)


def check_plan(plan, experts, E, what=""):
    slots, sources, offsets = sort_oracle(experts, E)
    for name, got, want in (("experts", plan.experts, experts), ("slots", plan.slots, slots), ("sources", plan.sources, sources),
                            ("offsets", plan.offsets, offsets)):
        assert np.array_equal(host(got), want), f"{what} {name}"


ROUTE_SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 7, 3), (64, 16, 2), (200, 13, 4), (1000, 8, 1), (333, 33, 9), (4099, 16, 2),
                (2000, 64, 8), (777, 100, 17), (500, 128, 32), (300, 129, 6), (257, 256, 8), (60, 300, 5), (40, 1000, 3),
                (33, 1024, 32), (30001, 6, 2), (70003, 2, 1), (9000, 1024, 2)]


@pytest.mark.parametrize("M,E,k", ROUTE_SHAPES)
@pytest.mark.parametrize("over", ["chosen", "all"])
@pytest.mark.parametrize("masked", [False, True])
def test_expert_route(M, E, k, over, masked):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("route", M, E, k)
    l = f32(rng, M, E, std=2.0) + f32(rng, E)
    l = np.round(l * 8).astype(np.float32) / 8 if M % 2 else l      # many ties
    if masked:
        l[rng.random((M, E)) < 0.3] = -INF
        l[M - M // 5:] = -INF
        l[0] = -INF
    dw = f32(rng, M, k)
    ld = padded(l, 1, 2, 9.0) if M % 3 == 0 else dev(l)
    plan, w = emu.expert_route(ld, k, over=over)
    dl = emu.expert_route_bwd(dev(dw), ld, plan, w, over=over)
    again = emu.expert_sort(plan.experts, E)
    done()
    experts, want = route_oracle(l, k, over)
    check_plan(plan, experts, E)
    check_plan(again, experts, E, "sorted alone")
    want.check(host(w), "weights")
    # the gradient, of the weights as given: sums of k terms; over all, p_e has the weights' bound
    wg, dwd = host(w).astype(np.float64), dw.astype(np.float64)
    inner, mag = (wg * dwd).sum(1, keepdims=True), np.abs(wg * dwd).sum(1, keepdims=True)
    ref, err = np.zeros((M, E + 1)), np.zeros((M, E + 1))
    at = np.where(experts < 0, E, experts)
    rows = np.arange(M)[:, None]
    part = wg * dwd - (wg * inner if over == "chosen" else 0)
    np.add.at(ref, (rows, at), part)
    np.add.at(err, (rows, at), (k + 8) * U * (np.abs(wg * dwd) + (wg * mag if over == "chosen" else 0)))
    if over == "all":
        l64 = l.astype(np.float64)
        top = np.where(experts[:, :1] >= 0, l64.max(1, keepdims=True), 0)
        e = np.exp(l64 - top)
        p = np.divide(e, e.sum(1, keepdims=True), out=np.zeros_like(e), where=e.sum(1, keepdims=True) > 0)
        span = np.where(l64 > -INF, top - l64, 0)
        ref[:, :E] -= p * inner
        err[:, :E] += p * mag * (span + want.err.max(initial=0) / U + E + k + 32) * U
    V(ref[:, :E], err[:, :E] + 2 * U * np.abs(ref[:, :E])).check(host(dl), "dlogits")


def test_expert_route_special_values():
    """Equal rows, +0 and -0 as equals, the type's lowest value open, infinities and
    NaN: NaN first, then +inf, and both show in the row's weights alone."""
    import fp32_emulated_gemm_gb300 as emu
    low = np.finfo(np.float32).min
    l = np.array([[0, 0, 0, 0, 0], [-0.0, 0.0, -0.0, -1, -1], [low, -INF, low, -INF, -INF], [1, INF, 2, 3, 0],
                  [1, np.nan, INF, 3, 0], [-INF, -INF, -INF, -INF, 5], [1e30, -1e30, 3, 1e30, 2]], np.float32)
    for over in ("chosen", "all"):
        plan, w = emu.expert_route(dev(l), 3, over=over)
        done()
        e, w = host(plan.experts), host(w)
        assert e.tolist() == [[0, 1, 2], [0, 1, 2], [0, 2, -1], [1, 3, 2], [1, 2, 3], [4, -1, -1], [0, 3, 2]]
        check_plan(plan, e, 5)
        assert np.isnan(w[3]).any() and np.isnan(w[4]).any() and np.isfinite(np.delete(w, (3, 4), 0)).all()
        assert w[2].tolist() == [0.5, 0.5, 0] and w[5].tolist() == [1, 0, 0] and w[6].tolist() == [0.5, 0.5, 0]


@pytest.mark.parametrize("M,E,k", [(1, 4, 1), (50, 3, 2), (3000, 40, 6), (20000, 300, 3)])
def test_expert_sort_takes_any_choices(M, E, k):
    """Choices outside the experts go nowhere; an expert may come twice; one may
    take everything."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("sort", M, E, k)
    for e in (rng.integers(-2, E + 2, (M, k)), np.full((M, k), E - 1), np.full((M, k), -1),
              np.where(rng.random((M, k)) < 0.5, 2 ** 31 - 1, -2 ** 31)):
        plan = emu.expert_sort(ints(e), E)
        done()
        check_plan(plan, e, E)


# --------------------------------------------------------------- exchange --
EXCHANGE_SHAPES = [(1, 1, 1), (1, 1024, 2), (5, 3, 3), (77, 16, 2), (60, 20, 4), (300, 31, 1), (129, 64, 3), (100, 65, 8),
                   (64, 128, 2), (1000, 256, 2), (333, 333, 3), (50, 512, 32), (40, 1001, 5), (9, 4099, 2), (20000, 24, 2),
                   (12, 8, 32), (700, 300, 3), (1300, 1030, 2), (1217, 4100, 1), (30, 2000, 4), (610, 2049, 3)]


@pytest.mark.parametrize("M,N,k", EXCHANGE_SHAPES)
@pytest.mark.parametrize("kind", ["full", "masked", "odd"])
def test_exchange(M, N, k, kind):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("exchange", M, N, k)
    E = 6
    e = rng.integers(0, E, (M, k))
    if kind != "full":
        e[rng.random((M, k)) < 0.3] = -1
        e[M - M // 4:] = -1
    plan = emu.expert_sort(ints(e), E)
    slots, sources, offsets = sort_oracle(e, E)
    T, sent = M * k, int(offsets[-1])
    x, ys, r, dy, dxs, w = f32(rng, M, N), f32(rng, T, N), f32(rng, M, N), f32(rng, M, N), f32(rng, T, N), f32(rng, M, k)
    ys[sent:], dxs[sent:] = np.nan, np.nan                           # rows that no choice reads
    put = (lambda a: padded(a, 1)) if kind == "odd" else dev
    xs = emu.expert_dispatch(put(x), plan)
    y = emu.expert_combine_fwd(put(ys), plan, dev(w), residual=put(r))
    y0 = emu.expert_combine_fwd(put(ys), plan, dev(w))
    dx = emu.expert_combine_fwd(put(dxs), plan)
    dys, dw = emu.expert_combine_bwd(put(dy), put(ys), plan, dev(w))
    dys1, none = emu.expert_combine_bwd(put(dy), None, plan, dev(w), need=(True, False))
    none2, dw1 = emu.expert_combine_bwd(put(dy), put(ys), plan, dev(w), need=(False, True))
    done()
    assert none is None and none2 is None
    token = np.where(sources >= 0, sources // k, 0)
    assert np.array_equal(host(xs), np.where((sources >= 0)[:, None], x[token], 0))
    wrow = np.where(sources >= 0, w.reshape(-1)[np.maximum(sources, 0)], 0).astype(np.float32)
    want_dys = np.where((sources >= 0)[:, None], dy[token] * wrow[:, None], 0)
    assert np.array_equal(host(dys), want_dys) and np.array_equal(host(dys1), want_dys)
    on = (slots >= 0)[:, :, None]
    at = np.maximum(slots, 0)
    w64 = w.astype(np.float64)[:, :, None]
    terms = np.where(on, w64 * np.nan_to_num(ys)[at], 0)
    s = V(terms.sum(1), (k + 1) * U * np.abs(terms).sum(1))
    s.check(host(y0), "Y without residual")
    (s + r).check(host(y), "Y")
    terms = np.where(on, np.nan_to_num(dxs)[at].astype(np.float64), 0)
    V(terms.sum(1), (k + 1) * U * np.abs(terms).sum(1)).check(host(dx), "dX")
    terms = np.where(on, dy[:, None, :].astype(np.float64) * np.nan_to_num(ys)[at], 0)
    want = V(terms.sum(2), (N / 16 + 24) * U * np.abs(terms).sum(2))
    want.check(host(dw), "dweights")
    want.check(host(dw1), "dweights alone")


@pytest.mark.parametrize("N", [16, 333, 1024])
def test_exchange_of_padded_tokens_that_hold_nan(N):
    """Tokens that go nowhere may hold anything: it reaches no row, no other token,
    and no weight's gradient."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("nan", N)
    M, k, E = 50, 3, 4
    e = rng.integers(0, E, (M, k))
    e[40:] = -1
    e[7, 1] = -1
    plan = emu.expert_sort(ints(e), E)
    x, dy, ys, w = f32(rng, M, N), f32(rng, M, N), f32(rng, M * k, N), f32(rng, M, k)
    want = [host(t) for t in (emu.expert_dispatch(dev(x), plan), *emu.expert_combine_bwd(dev(dy), dev(ys), plan, dev(w)))]
    x[40:], dy[40:], w[40:] = np.nan, INF, np.nan
    got = [host(t) for t in (emu.expert_dispatch(dev(x), plan), *emu.expert_combine_bwd(dev(dy), dev(ys), plan, dev(w)))]
    y = host(emu.expert_combine_fwd(dev(ys), plan, dev(w)))
    done()
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert not got[2][40:].any() and got[2][7, 1] == 0 and not y[40:].any() and np.isfinite(y).all()


def test_exchange_leaves_out_wrong_slots():
    """Slots outside the rows count as none: nothing is read or written there."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    M, k, N = 6, 2, 20
    plan = emu.expert_sort(ints(np.zeros((M, k))), 1)
    plan.slots[1, 0], plan.slots[4, 1], plan.slots[5, 0] = 12, -7, 2 ** 31 - 1
    x = torch.randn(M, N, device="cuda")
    buf = torch.full((M * k + 2, N), 7.0, device="cuda")
    emu.emu_expert_dispatch(M, k, N, x, N, plan.slots, plan.sources, buf[1:-1], N)
    ys = torch.randn(M * k, N, device="cuda")
    y = emu.expert_combine_fwd(ys, plan)
    done()
    want = torch.full_like(buf, 7.0)
    rows = ys.new_zeros(M, N)
    for m in range(M):
        for j in range(k):
            s = int(plan.slots[m, j])
            if 0 <= s < M * k:
                want[1 + s] = x[m]
                rows[m] += ys[s]
    assert torch.equal(buf, want) and torch.equal(y, rows)


@pytest.mark.parametrize("M,E,k", [(7, 1024, 2), (8, 1000, 9), (5, 700, 1)])
def test_many_experts_and_few_tokens(M, E, k):
    """One block, whose counts of all experts take more shared memory than a launch
    has by itself."""
    import fp32_emulated_gemm_gb300 as emu
    l = f32(rng_of("fewmany", M, E), M, E)
    plan, w = emu.expert_route(dev(l), k)
    done()
    experts, want = route_oracle(l, k, "chosen")
    check_plan(plan, experts, E)
    want.check(host(w), "weights")


# ---------------------------------------- offsets that 32 bits do not hold --
def last(n, count=64):
    """Places among n: the first, some between, the last ones."""
    return np.unique(np.concatenate([[0, 1, n // 2], np.arange(n - count, n)]))


def test_rms_norm_beyond_32_bits():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    M, N = 1100000, 2048
    x = torch.randn(M, N, device="cuda")
    w = torch.randn(N, device="cuda")
    y, s, rstd = emu.rms_norm_fwd(x, w, residual=x, eps=EPS)
    Q, scales = emu.rms_norm_quant(x, w, residual=x, eps=EPS)[:2]
    at = torch.from_numpy(last(M)).cuda()
    xs = host(x[at])
    want, s64, r = rms_norm(xs, xs, host(w))
    assert np.array_equal(host(s[at]), s64.val.astype(np.float32))
    want.check(host(y[at]), "Y")
    check_quant(want, host(Q[at].float()).astype(np.float64), host(scales[at]))
    del y, Q
    dx, dw = emu.rms_norm_bwd(x, s, w, rstd, add=x)
    rms_grads(xs, s64.val, host(w), host(rstd[at]).astype(np.float64), xs)[0].check(host(dx[at]), "dX")
    # dweight, here the sum of 2 x^2 rstd: chains of at most 4096 positive terms (a block's rows, then the blocks)
    size = sum((2 * x[i:i + 50000].double().square() * rstd[i:i + 50000, None].double()).sum(0) for i in range(0, M, 50000))
    done()
    assert float(((dw.double() - size) / size).abs().max()) < 4100 * U


def test_route_and_exchange_beyond_32_bits():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    M, E, k = 2200000, 1000, 2
    logits = torch.randn(M, E, device="cuda")
    plan, w = emu.expert_route(logits, k)
    at = torch.from_numpy(last(M)).cuda()
    experts, want = route_oracle(host(logits[at]), k, "chosen")
    assert np.array_equal(host(plan.experts[at]), experts)
    want.check(host(w[at]), "weights")
    check_plan(plan, host(plan.experts), E)
    dl = emu.expert_route_bwd(torch.ones_like(w), logits, plan, w)
    done()
    assert float(dl[at].abs().max()) <= 8 * U
    del dl, logits
    N = 512                                  # M k N > 2^31
    x = torch.randn(M, N, device="cuda")
    xs = emu.expert_dispatch(x, plan)
    rows = torch.from_numpy(last(M * k)).cuda()
    assert torch.equal(xs[rows], x[plan.sources[rows].long() // k]) and torch.equal(xs[plan.slots[at].long()], x[at, None].expand(-1, k, -1))
    y = emu.expert_combine_fwd(xs, plan, w, residual=x)
    dys, dw = emu.expert_combine_bwd(x, xs, plan, w)
    done()
    xa, wa = x[at].double(), w[at].double()
    assert bool(((y[at].double() - xa * (1 + wa.sum(1, keepdim=True))).abs() <= 6 * U * xa.abs() * 2).all())
    assert torch.equal(dys[plan.slots[at].long()], w[at][..., None] * x[at, None])
    n2 = xa.square().sum(1, keepdim=True)
    assert bool(((dw[at].double() - n2).abs() <= 40 * U * n2).all())     # chains of N / 32 + 8 positive terms


def test_expert_ffn_of_rows_beyond_32_bits():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(3)
    rows, K, F, N, E = 1100000, 8, 1024, 12, 3             # rows 2F > 2^31
    offsets = [0, 1099000, 1099700, rows]
    x, dy = torch.randn(rows, K, device="cuda"), torch.randn(rows, N, device="cuda")
    wi, wo = torch.randn(E, 2 * F, K, device="cuda") / K ** 0.5, torch.randn(E, N, F, device="cuda") / F ** 0.5
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
    dx, dwi, dwo = emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
    done()
    for e in range(E):
        r = slice(max(offsets[e], offsets[e + 1] - 400), offsets[e + 1])
        want = expert_reference(host(x[r]), host(wi[e]), host(wo[e]), "silu", "bf16x9", host(dy[r]))
        for got, ref, name in zip((y[r], h[r], dx[r]), want, ("Y", "H", "dX")):
            ref.check(host(got), f"expert {e} {name}")
    r = slice(offsets[2], rows)
    want = expert_reference(host(x[r]), host(wi[2]), host(wo[2]), "silu", "bf16x9", host(dy[r]))
    want[3].check(host(dwi[2]), "dW_in")
    want[4].check(host(dwo[2]), "dW_out")


@pytest.mark.parametrize("counts", [[2, 0, 3], [39800, 0, 200]])
def test_expert_ffn_of_weights_beyond_32_bits(counts):
    """On the CUDA cores, and in tiles."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(4)
    E, K, F, N = 600, 1800, 1024, 8                        # E 2F K > 2^31
    first, _, tail = counts
    rows = first + tail
    offsets = np.full(E + 1, first)
    offsets[0], offsets[-1] = 0, rows
    x, dy = torch.randn(rows, K, device="cuda"), torch.randn(rows, N, device="cuda")
    wi, wo = torch.randn(E, 2 * F, K, device="cuda") / K ** 0.5, torch.randn(E, N, F, device="cuda") / F ** 0.5
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
    dx, dwi, dwo = emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
    done()
    r = slice(first, rows)
    want = expert_reference(host(x[r]), host(wi[-1]), host(wo[-1]), "silu", "bf16x9", host(dy[r]))
    for got, ref, name in zip((y[r], h[r], dx[r], dwi[-1], dwo[-1]), want, ("Y", "H", "dX", "dW_in", "dW_out")):
        ref.check(host(got), name)
    assert not bool(dwi[1:-1].any()) and not bool(dwo[1:-1].any())


# ---------------------------------------------------------------- experts --
def expert_reference(x, wi, wo, act, mode, dy=None):
    """One expert's rows: (Y, D halves, H) and with dy (dX, dW_in, dW_out)."""
    F = wo.shape[1]
    z = R.product(x, wi.T, mode)
    g, u = z.cols(0, F), z.cols(F, 2 * F)
    a = R.act_value(act, g) if act != "none" else g
    d = R.act_grad(act, g) if act != "none" else V(np.ones_like(g.val))
    h = a * u
    y = R.product(h, wo.T, mode)
    if dy is None:
        return y, h
    dh = R.product(dy, wo, mode)
    d0 = u * d
    dg, du = dh * d0, dh * a
    dz = V(np.concatenate([dg.val, du.val], 1), np.concatenate([dg.err, du.err], 1))
    return y, h, R.product(dz, wi, mode), R.product(dz.T, x, mode), R.product(V(dy).T, h, mode)


COUNTS = {"one": [1], "few": [1, 0, 2, 0, 0, 1], "few_uneven": [0, 0, 9, 0, 1, 0], "many_for_one": [0, 300, 0, 0],
          "edges": [256, 0, 257, 1, 255, 31, 33], "ragged": [70, 513, 0, 5, 130], "last_empty": [40, 200, 0, 0],
          "nothing": [0, 0, 0], "tall": [5000, 0, 257, 3300]}


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("K,F,N,act", [(72, 100, 60, "silu"), (37, 131, 45, "gelu"), (256, 129, 4, "gelu_tanh"), (4, 3, 300, "none"),
                                       (1, 1, 1, "silu"), (600, 400, 404, "silu"), (601, 403, 397, "gelu")])
@pytest.mark.parametrize("counts", COUNTS)
def test_expert_ffn(counts, K, F, N, act, mode):
    """Rows beyond the last expert's are there too: they hold NaN and stay out.  (The
    forward passes with the counts "tall" run in tiles, most others on the CUDA
    cores.)"""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    counts = COUNTS[counts]
    rng = rng_of("ffn", len(counts), sum(counts), K, F)
    E, offsets = len(counts), np.concatenate([[0], np.cumsum(counts)])
    behind = 3 if counts[-1] == 0 else 0
    rows = int(offsets[-1]) + behind
    x, dy = f32(rng, rows, K), f32(rng, rows, N)
    x[rows - behind:], dy[rows - behind:] = np.nan, np.nan
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    put = lambda a: dev(a) if K % 2 == 0 else padded(a, 1)
    y0 = emu.expert_ffn_fwd(put(x), dev(wi), dev(wo), plan, act=act, mode=mode)
    y, d, h = emu.expert_ffn_fwd(put(x), dev(wi), dev(wo), plan, act=act, mode=mode, save=True)
    dx, dwi, dwo = emu.expert_ffn_bwd(put(dy), put(x), dev(wi), dev(wo), d, h, plan, act=act, mode=mode)
    again = emu.expert_ffn_bwd(put(dy), put(x), dev(wi), dev(wo), d, h, plan, act=act, mode=mode)
    done()
    assert dwi.shape == (E, 2 * F, K) and dwo.shape == (E, N, F)
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        y_, h_, dx_, dwi_, dwo_ = expert_reference(x[r], wi[e], wo[e], act, mode, dy[r])
        for got, want, name in ((y[r], y_, "Y"), (y0[r], y_, "Y without D"), (h[r], h_, "H"), (dx[r], dx_, "dX"),
                                (dwi[e], dwi_, "dW_in"), (dwo[e], dwo_, "dW_out"), (again[0][r], dx_, "dX again")):
            want.check(host(got), f"expert {e} {name}")
    assert torch.equal(dwi, again[1]) and torch.equal(dwo, again[2])


@pytest.mark.parametrize("E,K,F,N,most", [(70, 64, 160, 96, 700), (3, 2300, 300, 70, 260), (2, 40, 70, 2300, 4000), (300, 33, 17, 20, 60),
                                          (1024, 8, 8, 8, 30), (40, 256, 512, 260, 1500), (9, 1030, 700, 36, 900)])
def test_expert_ffn_uneven_experts(E, K, F, N, most):
    """Many experts of very different sizes; tiles of very many and of few stages,
    whose stages several pairs share."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("uneven", E, K, F)
    counts = (most * rng.random(E) ** 6).astype(np.int64)
    counts[E // 2] = most
    if E > 8 * 3:
        counts[:3] = 0
    offsets = np.concatenate([[0], np.cumsum(counts)])
    rows = int(offsets[-1])
    x, dy = f32(rng, rows, K), f32(rng, rows, N)
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    y, d, h = emu.expert_ffn_fwd(dev(x), dev(wi), dev(wo), plan, save=True)
    dx, dwi, dwo = emu.expert_ffn_bwd(dev(dy), dev(x), dev(wi), dev(wo), d, h, plan)
    done()
    got = [host(t) for t in (y, h, dx, dwi, dwo)]
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        want = expert_reference(x[r], wi[e], wo[e], "silu", "bf16x9", dy[r])
        for g, w, name in zip((got[0][r], got[1][r], got[2][r], got[3][e], got[4][e]), want, ("Y", "H", "dX", "dW_in", "dW_out")):
            w.check(g, f"expert {e} {name}")


@pytest.mark.parametrize("counts,K,F,N", [([1, 0, 0, 0, 0, 0, 0, 1], 700, 1500, 1026), ([0, 3, 1, 0], 1030, 2050, 515),
                                          ([0, 3, 2, 4], 1030, 2050, 515), ([0, 13, 3], 515, 1030, 771), ([9, 0, 2, 1, 0], 300, 1111, 2300),
                                          ([0] * 20 + [1] + [0] * 11 + [2], 260, 700, 1300)])
def test_expert_ffn_few_rows_of_long_contractions(counts, K, F, N):
    """The CUDA cores' backward products, several blocks to a contraction, with rows
    before and behind the experts'; the same results from a graph and in each wanted
    gradient alone."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("long", sum(counts), K, F)
    E, offsets = len(counts), 1 + np.concatenate([[0], np.cumsum(counts)])
    rows = int(offsets[-1]) + 1
    x, dy = f32(rng, rows, K), f32(rng, rows, N)
    x[0], dy[0], x[-1], dy[-1] = (np.nan,) * 4
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    X, DY, WI, WO = dev(x), dev(dy), dev(wi), dev(wo)
    y, d, h = emu.expert_ffn_fwd(X, WI, WO, plan, save=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = emu.expert_ffn_bwd(DY, X, WI, WO, d, h, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        replayed = emu.expert_ffn_bwd(DY, X, WI, WO, d, h, plan)
    graph.replay()
    done()
    alone = [emu.expert_ffn_bwd(DY, X, WI, WO, d if i < 2 else None, h if i == 2 else None, plan, need=[j == i for j in range(3)])[i]
             for i in range(3)]
    done()
    own = slice(int(offsets[0]), int(offsets[-1]))
    for a, b, c in zip(got, replayed, alone):
        cut = own if a.shape[0] == rows else slice(None)
        assert torch.equal(a[cut], b[cut]) and torch.equal(a[cut], c[cut])
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        want = expert_reference(x[r], wi[e], wo[e], "silu", "bf16x9", dy[r])
        for g, w, name in zip((y[r], h[r], got[0][r], got[1][e], got[2][e]), want, ("Y", "H", "dX", "dW_in", "dW_out")):
            w.check(host(g), f"expert {e} {name}")


@pytest.mark.parametrize("counts,K,F,N,act", [
    ([0, 13, 64, 33, 1, 90, 16, 31], 1028, 1540, 129, "silu"), ([0, 13, 64, 33, 1, 90, 16, 31], 36, 2052, 1030, "gelu"),
    ([40, 17, 5, 33], 36, 2052, 1030, "gelu_tanh"), ([200, 0, 7, 120, 65, 31], 256, 512, 260, "silu"),
    ([200, 0, 7, 120, 65, 31], 1028, 260, 516, "none"), ([9] * 30 + [0, 33], 1028, 1540, 129, "gelu"),
    ([9] * 30 + [0, 33], 2052, 640, 65, "silu")])
def test_expert_ffn_of_some_rows(counts, K, F, N, act):
    """Between few and many rows an expert: the CUDA cores' products through shared
    memory, blocks of 1 to 32 rows, shared contractions; the rows before and behind the
    experts' hold NaN and their outputs, as all around, stay what they were."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("some", sum(counts), K, F)
    E, offsets = len(counts), 1 + np.concatenate([[0], np.cumsum(counts)])
    rows = int(offsets[-1]) + 2
    x = f32(rng, rows, K)
    x[0], x[-2:] = np.nan, np.nan
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    X, WI, WO, o = dev(x), dev(wi), dev(wo), ints(offsets)
    G, up = 7.25, lambda n: (n + 3) // 4 * 4
    widths = (2 * F, F, N)
    bufs = [torch.full((rows + 2, up(c) + 8), G, device="cuda") for c in widths]
    d, h, y = (b[1:-1, 4:4 + c] for b, c in zip(bufs, widths))
    emu.emu_expert_ffn_fwd(0, emu.ACTS[act], rows, E, K, F, N, X, K, o, WI, K, WO, F,
                           d, d.stride(0), h, h.stride(0), y, y.stride(0))
    plan = emu.ExpertPlan(None, None, None, o)
    y0 = emu.expert_ffn_fwd(X, WI, WO, plan, act=act)
    y1, d1, h1 = emu.expert_ffn_fwd(X, WI, WO, plan, act=act, save=True)
    done()
    own = slice(1, rows - 2)
    assert all(torch.equal(a[own], b[own]) for a, b in ((y, y0), (y, y1), (h, h1), (d, d1)))
    for b, c in zip(bufs, widths):
        rim = b.clone()
        rim[2:rows - 1, 4:4 + c] = G
        assert bool((rim == G).all())
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        for g, w, name in zip((y[r], h[r]), expert_reference(x[r], wi[e], wo[e], act, "bf16x9"), ("Y", "H")):
            w.check(host(g), f"expert {e} {name}")


def test_expert_ffn_only_wanted_gradients():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("wanted")
    E, K, F, N, rows = 3, 40, 64, 52, 400
    plan = emu.ExpertPlan(None, None, None, ints([0, 150, 150, 400]))
    x, dy, wi, wo = (dev(f32(rng, *s)) for s in ((rows, K), (rows, N), (E, 2 * F, K), (E, N, F)))
    y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
    full = emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
    for i in range(3):
        need = [j == i for j in range(3)]
        got = emu.expert_ffn_bwd(dy, x, wi, wo, d if i < 2 else None, h if i == 2 else None, plan, need=need)
        assert torch.equal(got[i], full[i]) and [g is None for g in got] == [j != i for j in range(3)]
    assert emu.expert_ffn_bwd(dy, x, wi, wo, None, None, plan, need=(False,) * 3) == (None, None, None)
    none = emu.ExpertPlan(None, None, None, ints([0, 0, 0, 0]))
    e = torch.empty
    y, d, h = emu.expert_ffn_fwd(x[:0], wi, wo, none, save=True)
    dx, dwi, dwo = emu.expert_ffn_bwd(dy[:0], x[:0], wi, wo, d, h, none)
    done()
    assert y.shape == (0, N) and dx.shape == (0, K) and not dwi.any() and not dwo.any()


@pytest.mark.parametrize("rows,K,F,N", [(12, 36, 40, 24), (700, 36, 40, 24), (1000, 600, 400, 404)])
def test_expert_ffn_stays_within_its_rows(rows, K, F, N):
    """Rows outside the offsets are left as they were, in every output, and so are
    the words around the outputs; offsets that do not ascend or leave the rows are
    taken as if clipped."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("within", rows)
    E = 4
    x, dy, wi, wo = (dev(f32(rng, *s)) for s in ((rows, K), (rows, N), (E, 2 * F, K), (E, N, F)))
    G = 7.25
    a, b = rows // 4, rows // 2

    def run(offsets):
        o = ints(offsets)
        new = lambda r, c: torch.full((r + 2, c + 8), G, device="cuda")
        bufs = dict(y=new(rows, N), h=new(rows, F), d=new(rows, 2 * F), dz=new(rows, 2 * F), dx=new(rows, K), dwi=new(E * 2 * F, K),
                    dwo=new(E * N, F))
        v = {n: t[1:-1, 4:-4] for n, t in bufs.items()}
        emu.emu_expert_ffn_fwd(0, 4, rows, E, K, F, N, x, K, o, wi, K, wo, F, v["d"], 2 * F + 8, v["h"], F + 8, v["y"], N + 8)
        emu.emu_expert_ffn_bwd(0, rows, E, K, F, N, dy, N, x, K, o, wi, K, wo, F, v["d"], 2 * F + 8, v["h"], F + 8, v["dz"], 2 * F + 8,
                               v["dx"], K + 8, v["dwi"], K + 8, v["dwo"], F + 8)
        done()
        return bufs, v

    good, v = run([1, a, a, b, rows - 2])
    for n, t in good.items():
        rim = t.clone()
        rim[1:-1, 4:-4] = G
        assert bool((rim == G).all()), n
        if not n.startswith("dw"):
            assert bool((v[n][0] == G).all()) and bool((v[n][rows - 2:] == G).all()), n
            assert not bool((v[n][1:rows - 2] == G).any()), n
    # not ascending, negative, beyond the rows: as the clipped ones
    for wrong, clipped in (([1, a, 0, b, rows - 2], [1, a, a, b, rows - 2]), ([-5, a, a, b, 2 ** 31 - 1], [0, a, a, b, rows]),
                           ([b, a, a, a, a], [b, b, b, b, b]), ([2 ** 31 - 1] * 5, [rows] * 5), ([-2 ** 31] * 5, [0] * 5)):
        one, two = run(wrong)[0], run(clipped)[0]
        for n in one:
            assert torch.equal(one[n], two[n]), (wrong, n)


def test_expert_ffn_equals_the_block_of_one_expert():
    """One expert with every row is the gated block, bit for bit where the launch
    plans sum alike (the backward of a dense block splits its sums)."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("oneexpert")
    M, K, F = 2048, 256, 512
    x, wi, wo = dev(f32(rng, M, K)), dev(f32(rng, 1, 2 * F, K, std=0.06)), dev(f32(rng, 1, K, F, std=0.04))
    plan = emu.ExpertPlan(None, None, None, ints([0, M]))
    for mode in ("bf16x9", "tf32x3"):
        y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, mode=mode, save=True)
        h2, d2 = emu.gated_fwd(x, wi[0], mode=mode, save=True)
        done()
        want = R.product(host(x), host(wi[0]).T, mode)
        assert float((h - h2).abs().max()) <= 4 * float(want.err.max()) * float(host(h).max())
        assert h.shape == h2.shape and d.shape == d2.shape


# ------------------------------------------------- gradients, the sub-layer --
def plain_layer(p, x, k, over, mask=None, pre="ffn.", res=None):
    """EmuExpertFFN in torch's own operations (float64 on the CPU)."""
    import torch
    import torch.nn.functional as F
    logits = x @ p[pre + "router.weight"].T
    if mask is not None:
        logits = logits.masked_fill(~mask[:, None], -INF)
    v, e = torch.topk(logits, k, 1)
    w = torch.softmax(v, 1) if over == "chosen" else torch.softmax(logits, 1).gather(1, e)
    w = torch.where(torch.isnan(w) | (v == -INF), torch.zeros_like(w), w)
    y = torch.zeros_like(x @ p[pre + "weight_out"][0] @ p[pre + "weight_out"][0].T)
    for j in range(k):
        for n in range(len(p[pre + "weight_in"])):
            m = ((e[:, j] == n) & (v[:, j] > -INF)).nonzero()[:, 0]
            g, u = (x[m] @ p[pre + "weight_in"][n].T).chunk(2, 1)
            y = y.index_add(0, m, w[m, j, None] * ((F.silu(g) * u) @ p[pre + "weight_out"][n].T))
    return y if res is None else y + res


def rms64(x, w):
    import torch
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * w


@pytest.mark.parametrize("M,over,mode,masked", [(300, "chosen", "bf16x9", False), (301, "all", "tf32x3", True), (3, "chosen", "bf16x9", True),
                                                (1, "all", "bf16x9", False)])
def test_sub_layer_and_its_gradients(M, over, mode, masked):
    """x + experts(norm(x)) as it is used, forward and backward, against the same
    layer in float64."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(M)
    m = emu.EmuExpertFeedForward(48, 40, 6, 2, over=over, mode=mode).cuda()
    x = torch.randn(M, 48, device="cuda").requires_grad_()
    mask = torch.arange(M, device="cuda") < M - M // 3 if masked else None
    g = torch.randn(M, 48, device="cuda")
    y = m(x, mask)
    y.backward(g)
    with torch.no_grad():
        assert torch.equal(m(x, mask), y.detach())
    done()
    p = {n: t.detach().double().cpu().requires_grad_() for n, t in m.named_parameters()}
    x64 = x.detach().double().cpu().requires_grad_()
    h = rms64(x64, p["norm.weight"])
    y64 = plain_layer(p, h, 2, over, None if mask is None else mask.cpu(), res=x64)
    y64.backward(g.double().cpu())
    for name, a, b in [("y", y, y64), ("dx", x.grad, x64.grad)] + [(n, t.grad, p[n].grad) for n, t in m.named_parameters()]:
        assert a.shape == b.shape
        a, b = a.detach().double().cpu(), b.detach()
        assert float((a - b).abs().max()) <= 1e-5 * float(b.abs().max()), name
    if mask is not None:
        assert torch.equal(y.detach()[~mask], x.detach()[~mask])


@pytest.mark.parametrize("M,over", [(300, "chosen"), (5, "all")])
@pytest.mark.parametrize("fill", [float("nan"), INF, -3e38])
def test_padded_tokens_reach_nothing(M, over, fill):
    """Whatever padded tokens and their gradients hold: the others' outputs and
    gradients and the weights' gradients are those of zeros in their place."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(M)
    for layer in (emu.EmuExpertFeedForward(48, 40, 6, 2, over=over).cuda(), emu.EmuExpertFFN(48, 40, 6, 2, over=over).cuda()):
        mask = torch.arange(M, device="cuda") % 3 != 1
        x, g = torch.randn(M, 48, device="cuda"), torch.randn(M, 48, device="cuda")
        results = []
        for value in (0.0, fill):
            a = x.masked_fill(~mask[:, None], value).requires_grad_()
            y = layer(a, mask=mask)
            layer.zero_grad()
            y.backward(g.masked_fill(~mask[:, None], value))
            results.append([y.detach()[mask], a.grad[mask]] + [p.grad.clone() for p in layer.parameters()])
            with torch.no_grad():
                assert torch.equal(layer(a, mask=mask)[mask], y.detach()[mask])
        done()
        for want, got in zip(*results):
            assert bool(torch.isfinite(want).all()) and torch.equal(want, got)


def test_sub_layer_against_differences():
    """The gradient along a direction against central differences of the layer
    itself in float64 arithmetic of its own forward (the choices held fixed)."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(5)
    m = emu.EmuExpertFeedForward(32, 24, 4, 2).cuda()
    x = torch.randn(60, 32, device="cuda").requires_grad_()
    g = torch.randn(60, 32, device="cuda")
    (m(x) * g).sum().backward()
    done()
    p = {n: t.detach().double().cpu() for n, t in m.named_parameters()}
    d = torch.randn(60, 32, dtype=torch.float64)
    f = lambda t: float((plain_layer(p, rms64(t, p["norm.weight"]), 2, "chosen", res=t) * g.double().cpu()).sum())
    x64, h = x.detach().double().cpu(), 1e-6
    want = (f(x64 + h * d) - f(x64 - h * d)) / (2 * h)
    got = float((x.grad.double().cpu() * d).sum())
    # differences: h^2 of the third derivative and 2^-52 |f| / h; the gradient's own 1e-5 of its size
    assert abs(got - want) <= 1e-5 * float((x.grad.double().cpu() * d).abs().sum()) + 1e-7 * max(1.0, abs(f(x64)))


def test_no_tokens_and_no_open_experts():
    """An empty batch, and one whose tokens are all padding: the residual alone, and
    zero gradients of the experts."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(2)
    m = emu.EmuExpertFeedForward(32, 24, 4, 2).cuda()
    for M, mask in ((0, None), (5, torch.zeros(5, dtype=torch.bool, device="cuda")),
                    (400, torch.zeros(400, dtype=torch.bool, device="cuda"))):
        x = torch.randn(M, 32, device="cuda", requires_grad=True)
        m.zero_grad()
        y = m(x, mask)
        y.backward(torch.ones_like(y))
        done()
        assert torch.equal(y, x) and bool((x.grad == 1).all())
        for n, p in m.named_parameters():
            assert p.grad.shape == p.shape and not p.grad.any(), (M, n)


def test_modules_want_only_some_gradients():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(1)
    m = emu.EmuExpertFeedForward(32, 40, 4, 2).cuda()
    x = torch.randn(2, 50, 32, device="cuda")
    m(x).sum().backward()                    # an expanded upstream gradient
    full = {n: p.grad.clone() for n, p in m.named_parameters()}
    for keep in full:
        m.zero_grad()
        for n, p in m.named_parameters():
            p.requires_grad_(n == keep)
        m(x).sum().backward()
        assert torch.equal(dict(m.named_parameters())[keep].grad, full[keep]), keep
    m.requires_grad_(False)
    xg = x.clone().requires_grad_()
    m(xg).sum().backward()
    assert xg.grad.shape == x.shape and bool(torch.isfinite(xg.grad).all())
    norm = emu.EmuRMSNorm(32).cuda()
    a, b = torch.randn(7, 32, device="cuda", requires_grad=True), torch.randn(7, 32, device="cuda", requires_grad=True)
    y, s = norm(a, b)
    s.sum().backward()                       # the stream alone
    assert bool((a.grad == 1).all()) and bool((b.grad == 1).all()) and norm.weight.grad is None
    done()


# ------------------------------------------------- graphs, streams, buffers --
def test_layer_in_a_graph():
    """Captured once, replayed on other tokens with other choices: the rows of each
    expert are the device's to find."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(3)
    m = emu.EmuExpertFeedForward(64, 48, 5, 2).cuda()
    for M in (1, 900):
        x = torch.randn(M, 64, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.no_grad():
            m(x)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s), torch.no_grad():
            y = m(x)
        for seed in range(3):
            new = torch.randn(M, 64, device="cuda") * (1 + seed)
            x.copy_(new)
            graph.replay()
            torch.cuda.synchronize()
            with torch.no_grad():
                assert torch.equal(y, m(new))
    done()


def test_training_step_in_a_graph():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("stepgraph")
    M, K, F, E, k = 500, 40, 36, 4, 2
    x, dy, logits = dev(f32(rng, M, K)), dev(f32(rng, M, K)), dev(f32(rng, M, E))
    wi, wo, w = dev(f32(rng, E, 2 * F, K)), dev(f32(rng, E, K, F)), dev(f32(rng, K, mean=1.0))

    def step():
        n, s, rstd = emu.rms_norm_fwd(x, w)
        plan, wt = emu.expert_route(logits, k)
        xs = emu.expert_dispatch(n, plan)
        ys, d, h = emu.expert_ffn_fwd(xs, wi, wo, plan, save=True)
        y = emu.expert_combine_fwd(ys, plan, wt, residual=x)
        dys, dwt = emu.expert_combine_bwd(dy, ys, plan, wt)
        dl = emu.expert_route_bwd(dwt, logits, plan, wt)
        dxs, dwi, dwo = emu.expert_ffn_bwd(dys, xs, wi, wo, d, h, plan)
        dx, dw = emu.rms_norm_bwd(emu.expert_combine_fwd(dxs, plan), s, w, rstd, add=dy)
        return y, dl, dwi, dwo, dx, dw

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for seed in range(3):
        logits.copy_(dev(f32(rng, M, E)))
        x.copy_(dev(f32(rng, M, K)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    done()


def test_training_of_the_module_in_a_graph():
    """The module's forward and backward pass captured as torch does it: the
    parameters' gradients of each replay are those of the tokens of the time."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(6)
    m = emu.EmuExpertFeedForward(48, 40, 5, 2).cuda()
    x, g = torch.randn(600, 48, device="cuda"), torch.randn(600, 48, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            m.zero_grad(set_to_none=True)
            m(x).backward(g)
    torch.cuda.current_stream().wait_stream(s)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = m(x)
        y.backward(g)
    static = {n: p.grad for n, p in m.named_parameters()}
    for seed in range(3):
        x.copy_(torch.randn(600, 48, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in static.items()}
        twin = emu.EmuExpertFeedForward(48, 40, 5, 2).cuda()
        twin.load_state_dict(m.state_dict())
        want = twin(x)
        want.backward(g)
        assert torch.equal(y, want)
        for n, p in twin.named_parameters():
            assert torch.equal(got[n], p.grad), n
    done()


@pytest.mark.parametrize("own_stream", [False, True])
def test_threads_on_one_stream(own_stream):
    """Several host threads call on one stream: a call's launches, which share the
    stream's buffers, follow one another."""
    import contextlib
    import threading
    import torch
    import fp32_emulated_gemm_gb300 as emu

    def calls(seed):
        rng = rng_of("threads", seed)
        E, K, F, N, M = 4 + seed, 300 + 64 * seed, 260, 301, 900 + 100 * seed
        logits, x = dev(f32(rng, 9000 + seed, 12)), dev(f32(rng, 2 * M, K))
        wi, wo, dy = dev(f32(rng, E, 2 * F, K)), dev(f32(rng, E, N, F)), dev(f32(rng, 2 * M, N))
        plan = emu.expert_route(dev(f32(rng, M, E)), 2)[0]
        y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
        rstd = dev(f32(rng, 2 * M))
        return [lambda: emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan), lambda: [*emu.expert_route(logits, 3)[0][1:]],
                lambda: emu.rms_norm_bwd(x, x, None, rstd), lambda: [emu.expert_ffn_fwd(x, wi, wo, plan)]]

    sets = [calls(seed) for seed in range(3)]
    want = [[[t.clone() for t in call()] for call in s] for s in sets]
    torch.cuda.synchronize()
    emu.emu_shutdown()                       # the buffers grow again while the threads run
    stream = torch.cuda.Stream()
    wrong, start = [], threading.Barrier(len(sets))

    def worker(i):
        try:
            with torch.cuda.stream(stream) if own_stream else contextlib.nullcontext():
                start.wait(60)
                for rep in range(40):
                    k = (rep + i) % len(sets[i])
                    for j, (got, w) in enumerate(zip(sets[i][k](), want[i][k])):
                        if not torch.equal(got, w):
                            wrong.append((i, rep, k, j))
        except Exception as e:
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(300)
    assert not any(t.is_alive() for t in threads)
    assert not wrong, wrong[:8]
    assert emu.emu_stream_check(stream if own_stream else None) == 0


def test_two_streams_at_once():
    """Two layers on two streams: each has its own buffers."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(4)
    layers = [emu.EmuExpertFeedForward(64, 80 + 16 * i, 6, 2).cuda() for i in range(2)]
    xs = [torch.randn(2500 + 100 * i, 64, device="cuda") for i in range(2)]
    with torch.no_grad():
        want = [m(x) for m, x in zip(layers, xs)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(10):
            got = []
            for m, x, s in zip(layers, xs, streams):
                with torch.cuda.stream(s):
                    got.append(m(x))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    done()


def test_allocation_failure_enqueues_nothing():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("allocx")
    E, K, F, rows = 3, 601, 400, 1000       # (tiles, and an odd operand: copies, lists, shared sums)
    plan = emu.ExpertPlan(None, None, None, ints([0, 400, 400, 1000]))
    x, wi, wo = dev(f32(rng, rows, K)), dev(f32(rng, E, 2 * F, K)), dev(f32(rng, E, K, F))
    y = torch.full((rows, 604), 7.0, device="cuda")
    h = torch.full((rows, F), 7.0, device="cuda")
    logits = dev(f32(rng, 20000, 8))
    outs = [torch.full((20000, 2), 7, device="cuda", dtype=torch.int32) for _ in range(3)] + [
        torch.full((20000, 2), 7.0, device="cuda"), torch.full((9,), 7, device="cuda", dtype=torch.int32)]
    calls = [(2, lambda: emu.emu_expert_ffn_fwd(0, 4, rows, E, K, F, K, x, K, plan.offsets, wi, K, wo, F, None, 0, h, F, y, 604)),
             (1, lambda: emu.emu_expert_route(0, 20000, 8, 2, logits, 8, outs[0], outs[3], outs[1], outs[2], outs[4]))]
    for n, call in calls:
        for _ in range(n):                    # the n-th of the call's allocations
            emu.emu_shutdown()
            emu.emu_debug_fail_allocations(1)
            try:
                with pytest.raises(emu.EmuError) as e:
                    call()
                assert e.value.status == 4
            finally:
                emu.emu_debug_fail_allocations(0)
            done()
            assert bool((y == 7).all()) and bool((h == 7).all()) and all(bool((t == 7).all()) for t in outs)
    for _, call in calls:
        call()
    done()


def test_allocation_failure_of_the_backward_buffers_enqueues_nothing():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("allocb")
    E, K, F, N, rows = 4, 515, 1030, 771, 8   # (few rows: copies of odd operands, shares of contractions)
    o = ints([0, 3, 3, 4, 8])
    x, dy, wi, wo, d, h = (dev(f32(rng, *s)) for s in ((rows, K), (rows, N), (E, 2 * F, K), (E, N, F), (rows, 2 * F), (rows, F)))
    new = lambda r, c: torch.full((r, c), 7.0, device="cuda")
    dz, dx, dwi, dwo = new(rows, 2 * F), new(rows, 516), new(E * 2 * F, 516), new(E * N, 1032)
    call = lambda: emu.emu_expert_ffn_bwd(0, rows, E, K, F, N, dy, N, x, K, o, wi, K, wo, F, d, 2 * F, h, F, dz, 2 * F, dx, 516, dwi,
                                          516, dwo, 1032)
    emu.emu_shutdown()
    emu.emu_debug_fail_allocations(1)
    try:
        with pytest.raises(emu.EmuError) as e:
            call()
        assert e.value.status == 4
    finally:
        emu.emu_debug_fail_allocations(0)
    done()
    assert all(bool((t == 7).all()) for t in (dz, dx, dwi, dwo))
    call()
    done()
    assert not any(bool((t[:, :c] == 7).any()) for t, c in ((dz, 2 * F), (dx, K), (dwi, K), (dwo, F)))


def test_refusals():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    new = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    x = new(6, 8)
    plan = emu.expert_sort(ints(np.zeros((6, 2))), 3)
    wi, wo = new(3, 10, 8), new(3, 4, 5)
    xs = new(12, 8)
    for bad in (lambda: emu.rms_norm_fwd(new(8)), lambda: emu.rms_norm_fwd(x, new(7)), lambda: emu.rms_norm_fwd(x, residual=new(6, 7)),
                lambda: emu.rms_norm_fwd(x, out=new(5, 8)), lambda: emu.rms_norm_quant(x, residual=new(5, 8)),
                lambda: emu.rms_norm_bwd(new(6, 7), x, None, new(6)), lambda: emu.rms_norm_bwd(x, x, None, new(5)),
                lambda: emu.rms_norm_bwd(x, x, None, new(6), add=x, need_input=False),
                lambda: emu.expert_route(new(8), 1), lambda: emu.expert_route(x, 0), lambda: emu.expert_route(x, 9),
                lambda: emu.expert_route(x, 2, over="some"), lambda: emu.expert_sort(new(6, dtype=torch.int32), 3),
                lambda: emu.expert_route_bwd(new(6, 3), new(6, 3), plan, new(6, 2)),
                lambda: emu.expert_dispatch(new(5, 8), plan), lambda: emu.expert_combine_fwd(new(11, 8), plan),
                lambda: emu.expert_combine_fwd(xs, plan, new(6, 3)), lambda: emu.expert_combine_fwd(xs, plan, residual=new(5, 8)),
                lambda: emu.expert_combine_bwd(x, new(11, 8), plan, new(6, 2)), lambda: emu.expert_combine_bwd(new(5, 8), xs, plan, new(6, 2)),
                lambda: emu.expert_ffn_fwd(xs, new(3, 9, 8), wo, plan), lambda: emu.expert_ffn_fwd(xs, new(3, 10, 7), wo, plan),
                lambda: emu.expert_ffn_fwd(xs, wi, new(4, 4, 5), plan), lambda: emu.expert_ffn_fwd(xs, wi[0], wo, plan),
                lambda: emu.expert_ffn_fwd(xs, new(2, 10, 8), new(2, 4, 5), plan), lambda: emu.expert_ffn_fwd(xs, wi, wo, plan, act="tanh"),
                lambda: emu.expert_ffn_bwd(new(12, 5), xs, wi, wo, new(12, 10), new(12, 5), plan)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: emu.rms_norm_fwd(x.double()), lambda: emu.rms_norm_fwd(x.cpu()), lambda: emu.rms_norm_bwd(x, x, None, None),
                lambda: emu.expert_sort(torch.zeros(6, 2, dtype=torch.int64, device="cuda"), 3),
                lambda: emu.expert_sort(torch.zeros(6, 2, dtype=torch.int32), 3),
                lambda: emu.expert_ffn_fwd(xs, wi.half(), wo, plan), lambda: emu.expert_ffn_bwd(new(12, 4), xs, wi, wo, None, new(12, 5), plan)):
        with pytest.raises(TypeError):
            bad()
    for status, bad in ((1, lambda: emu.rms_norm_fwd(x, eps=-1.0)), (2, lambda: emu.expert_ffn_fwd(xs, wi, wo, plan, mode="fp32")),
                        (2, lambda: emu.expert_route(new(2, 1025), 1)), (2, lambda: emu.expert_route(new(2, 64), 33)),
                        (2, lambda: emu.expert_sort(ints(np.zeros((2, 1))), 1025)), (1, lambda: emu.expert_sort(ints(np.zeros((2, 1))), 0))):
        with pytest.raises(emu.EmuError) as e:
            bad()
        assert e.value.status == status
    done()
