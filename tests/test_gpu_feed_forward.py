"""The feed-forward operators against their definitions in 64 bits.

Every tolerance is the running error bound of tests/_running.py: the
products' stated accuracy and the roundings of what is around them, carried
through the definition.  Gradients are checked against the formulas and
against differences of the definition.
"""
import numpy as np
import pytest

from tests import _gpu
from tests import _running as R
from tests._running import V

pytestmark = pytest.mark.gpu
EPS = 1e-5
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def rng_of(*key):
    return np.random.default_rng([abs(hash_(k)) for k in key])


def hash_(k):
    return k if isinstance(k, int) else int.from_bytes(str(k).encode()[:8].ljust(8, b"_"), "little")


def f32(rng, *shape, std=1.0, mean=0.0):
    return (rng.standard_normal(shape) * std + mean).astype(np.float32)


def dev(x):
    return None if x is None else _gpu.to_dev(x)


def host(t):
    return t.detach().cpu().numpy()


def done():
    import fp32_emulated_gemm_gb300 as emu
    st = emu.emu_stream_check()
    assert st == 0, emu.emu_status_string(st)


# ------------------------------------------------------------- layer norm --
LN_SHAPES = [(1, 1), (3, 2), (65, 4), (50, 16), (77, 13), (33, 17), (130, 32), (5, 31), (129, 61), (33, 64), (40, 128),
             (1, 256), (192, 256), (700, 257), (65, 512), (40, 1000), (37, 1001), (9, 1024), (20, 2048), (12, 2050),
             (5, 4096), (3, 8192), (4, 9001), (3, 16384), (2, 16383), (2, 20000), (2, 40003)]


@pytest.mark.parametrize("M,N", LN_SHAPES)
@pytest.mark.parametrize("affine", ["both", "weight", "none"])
def test_layer_norm(M, N, affine):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("ln", M, N)
    x = f32(rng, M, N, std=1.5, mean=0.5) * np.exp(f32(rng, N, std=0.5)) + f32(rng, N)
    x = x.astype(np.float32)
    w = f32(rng, N, std=0.2, mean=1.0) if affine != "none" else None
    b = f32(rng, N) if affine == "both" else None
    dy, add = f32(rng, M, N), f32(rng, M, N)
    y, mean, rstd = emu.layer_norm_fwd(dev(x), dev(w), dev(b), eps=EPS)
    dx, dw, db = emu.layer_norm_bwd(dev(dy), dev(x), dev(w), mean, rstd, add=dev(add))
    dx0, _, _ = emu.layer_norm_bwd(dev(dy), dev(x), dev(w), mean, rstd, need_params=False)
    done()
    x64, w64 = x.astype(np.float64), None if w is None else w.astype(np.float64)
    R.layer_norm(x64, w64, b, EPS)[0].check(host(y), "Y")
    want = R.layer_norm_grads(dy, x64, w64, EPS, add)
    want[0].check(host(dx), "dX")
    want[1].check(host(dw), "dweight")
    want[2].check(host(db), "dbias")
    R.layer_norm_grads(dy, x64, w64, EPS)[0].check(host(dx0), "dX without add")


@pytest.mark.parametrize("N", [7, 256, 1001, 5000])
def test_layer_norm_hard_rows(N):
    """Rows that are constant, huge, tiny, far from zero, or hold one outlier."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("hard", N)
    rows = [np.zeros(N), np.full(N, 7.0), f32(rng, N) * 1e15, f32(rng, N) * 1e-15, f32(rng, N) + 4096.0,
            np.where(np.arange(N) == N // 2, 1e6, 1e-3)]
    x = np.stack(rows).astype(np.float32)
    w, b, dy = f32(rng, N, mean=1.0, std=0.1), f32(rng, N), f32(rng, len(rows), N)
    y, mean, rstd = emu.layer_norm_fwd(dev(x), dev(w), dev(b), eps=EPS)
    dx, dw, db = emu.layer_norm_bwd(dev(dy), dev(x), dev(w), mean, rstd)
    done()
    x64 = x.astype(np.float64)
    R.layer_norm(x64, w, b, EPS)[0].check(host(y), "Y")
    for got, want, name in zip((dx, dw, db), R.layer_norm_grads(dy, x64, w, EPS), ("dX", "dweight", "dbias")):
        want.check(host(got), name)


def test_layer_norm_many_rows_and_repeatable():
    """More rows than the GPU takes at once; the sums over rows are the same
    bits on every run."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("many")
    M, N = 30011, 96
    x, dy, w, b = f32(rng, M, N, mean=0.3), f32(rng, M, N), f32(rng, N), f32(rng, N)
    xd, dyd, wd = dev(x), dev(dy), dev(w)
    y, mean, rstd = emu.layer_norm_fwd(xd, wd, dev(b))
    first = emu.layer_norm_bwd(dyd, xd, wd, mean, rstd)
    again = emu.layer_norm_bwd(dyd, xd, wd, mean, rstd)
    done()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    x64 = x.astype(np.float64)
    R.layer_norm(x64, w, b, EPS)[0].check(host(y), "Y")
    for got, want, name in zip(first, R.layer_norm_grads(dy, x64, w, EPS), ("dX", "dweight", "dbias")):
        want.check(host(got), name)


# ------------------------------------------------------------- linear_act --
def linear_act_reference(x, w, b, act, r, dy, mode, d_gpu=None):
    z = R.product(x, w.T, mode, b)
    y = R.act_value(act, z) if act != "none" else z
    if r is not None:
        y = y + r
    if act == "none":
        d = V(np.ones_like(z.val))
    else:
        d = R.act_grad(act, z)
        if act == "relu" and d_gpu is not None:  # the derivative jumps: where Z is within its error of 0, the GPU's own sign stands
            d = V(np.where(np.abs(z.val) <= z.err, d_gpu > 0, z.val > 0))
    if dy is None:
        return y, d
    dz = V(dy) * d
    return y, d, R.product(dz, w, mode), R.product(dz.T, x, mode), R.column_sum(dz)


LINEAR_SHAPES = [(1, 1, 1), (1, 300, 64), (1, 64, 1024), (2, 129, 33), (5, 96, 100), (8, 257, 260), (9, 40, 7),
                 (16, 512, 128), (17, 100, 36), (40, 30, 500), (300, 260, 200), (257, 1, 64), (130, 131, 37),
                 (1100, 520, 72), (1025, 1, 1), (1030, 129, 33), (1100, 257, 260), (1281, 40, 7), (1025, 131, 37),
                 (71, 1024, 770), (72, 1024, 770), (8, 4000, 2000)]


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear_act(M, N, K, act, mode):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("linear", M, N, K, act)
    x, w = f32(rng, M, K), f32(rng, N, K, std=K ** -0.5)
    b = f32(rng, N, std=0.1) if (M + N) % 2 else None
    r = f32(rng, M, N) if (M + K) % 2 else None
    dy = f32(rng, M, N)
    y0 = emu.linear_act_fwd(dev(x), dev(w), dev(b), act=act, residual=dev(r), mode=mode)
    y, d = emu.linear_act_fwd(dev(x), dev(w), dev(b), act=act, residual=dev(r), mode=mode, save=True)
    dx, dw, db = emu.linear_act_bwd(dev(dy), dev(x), dev(w), d, act=act, mode=mode)
    done()
    assert (d is None) == (act == "none")
    want = linear_act_reference(x, w, b, act, r, dy, mode, None if d is None else host(d))
    want[0].check(host(y0), "Y")
    for got, v, name in zip((y, d, dx, dw, db), want, ("Y, saving D", "D", "dX", "dW", "dbias")):
        if got is not None:
            v.check(host(got), name)


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("M,N,K", [(6144, 1024, 256), (2000, 2500, 200), (300, 260, 3000), (520, 300, 6000)])
def test_linear_act_every_plan(M, N, K, mode):
    """Products whose tiles are chained between CTA pairs, and ones whose
    tiles are split along k into few and into many pieces: each applies the
    epilogue once, to the whole sum."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("plans", M, N, K)
    x, w, b, r = f32(rng, M, K), f32(rng, N, K, std=K ** -0.5), f32(rng, N, std=0.1), f32(rng, M, N)
    y, d = emu.linear_act_fwd(dev(x), dev(w), dev(b), act="gelu", residual=dev(r), mode=mode, save=True)
    y0 = emu.linear_act_fwd(dev(x), dev(w), dev(b), act="gelu", residual=dev(r), mode=mode)
    done()
    rows = np.unique(np.concatenate([np.arange(0, M, 37), np.arange(max(0, M - 40), M)]))
    wy, wd = linear_act_reference(x[rows], w, b, "gelu", r[rows], None, mode)
    wy.check(host(y)[rows], "Y")
    wd.check(host(d)[rows], "D")
    assert np.array_equal(host(y), host(y0))


@pytest.mark.parametrize("mode", ["fp32", "bf16x6", "tf32x1"])
def test_linear_act_and_block_in_the_other_modes(mode):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("other modes")
    M, N, K, F = 150, 140, 100, 60  # (these modes have no few-row form)
    x, w, b, dy = f32(rng, M, K), f32(rng, N, K, std=0.1), f32(rng, N), f32(rng, M, N)
    y, d = emu.linear_act_fwd(dev(x), dev(w), dev(b), act="silu", mode=mode, save=True)
    g = emu.linear_act_bwd(dev(dy), dev(x), dev(w), d, act="silu", mode=mode)
    done()
    for got, v, name in zip((y, d, *g), linear_act_reference(x, w, b, "silu", None, dy, mode), ("Y", "D", "dX", "dW", "db")):
        v.check(host(got), name)
    check_ffn(rng, 70, 44, F, 52, "silu", mode, residual=True)


# ----------------------------------------------------------- gated blocks --
def beside(p, q):
    return V(np.concatenate([p.val, q.val], 1), np.concatenate([p.err, q.err], 1))


def gated_reference(x, w, b, act, mode, d_gpu=None):
    """(H, D)"""
    F = w.shape[0] // 2
    z = R.product(x, w.T, mode, b)
    g, u = z.cols(0, F), z.cols(F, 2 * F)
    slope = R.act_grad(act, g)
    if act == "relu":  # (as in linear_act_reference; U = 0 leaves the sign open, and the product zero)
        on = g.val > 0 if d_gpu is None else np.where(np.abs(g.val) <= g.err, d_gpu[:, :F] != 0, g.val > 0)
        slope = V(on.astype(np.float64))
    a = R.act_value(act, g)
    return a * u, beside(u * slope, a)


def gated_grads(dh, x, w, mode, d):
    F = w.shape[0] // 2
    dz = beside(dh * d.cols(0, F), dh * d.cols(F, 2 * F))
    return R.product(dz, w, mode), R.product(dz.T, x, mode), R.column_sum(dz)


def check_ffn(rng, M, K, F, N, act, mode, residual, bias=True, lay=None):
    import fp32_emulated_gemm_gb300 as emu
    mat = lay or dev
    x, wi, wo = f32(rng, M, K), f32(rng, 2 * F, K, std=K ** -0.5), f32(rng, N, F, std=F ** -0.5)
    bi, bo = (f32(rng, 2 * F, std=0.1), f32(rng, N, std=0.1)) if bias else (None, None)
    r, dy = f32(rng, M, N) if residual else None, f32(rng, M, N)
    args = (mat(x), mat(wi), dev(bi), mat(wo), dev(bo))
    y0 = emu.gated_ffn_fwd(*args, act=act, residual=None if r is None else mat(r), mode=mode)
    y, d, h = emu.gated_ffn_fwd(*args, act=act, residual=None if r is None else mat(r), mode=mode, save=True)
    grads = emu.gated_ffn_bwd(mat(dy), args[0], args[1], args[3], d, h, act=act, mode=mode)
    done()
    wh, wd = gated_reference(x, wi, bi, act, mode, host(d))
    wy = R.product(wh, wo.T, mode, bo)
    if r is not None:
        wy = wy + r
    dh = R.product(dy, wo, mode)
    dx, dwi, dbi = gated_grads(dh, x, wi, mode, wd)
    wy.check(host(y0), "Y")
    want = (wy, wd, wh, dx, dwi, dbi, R.product(V(dy).T, wh, mode), R.column_sum(dy))
    names = ("Y, saving", "D", "H", "dX", "dW_in", "db_in", "dW_out", "db_out")
    for got, v, name in zip((y, d, h, *grads), want, names):
        v.check(host(got), name)


FFN_SHAPES = [(1, 1, 1, 1), (1, 64, 100, 64), (1, 1024, 300, 256), (3, 33, 65, 31), (8, 128, 256, 128), (9, 20, 20, 20),
              (20, 100, 130, 60), (70, 40, 129, 36), (300, 72, 260, 72), (1030, 64, 150, 32), (261, 37, 41, 43), (1025, 1, 1, 1),
          (1030, 33, 65, 31), (1100, 100, 130, 60), (1281, 20, 20, 20), (1100, 72, 260, 72), (1025, 37, 41, 43)]


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("M,K,F,N", FFN_SHAPES)
def test_gated_ffn(M, K, F, N, act, mode):
    check_ffn(rng_of("ffn", M, K, F, N, act), M, K, F, N, act, mode, residual=(M + K) % 2 == 0, bias=F % 2 == 0)


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("M,K,F", [(6144, 256, 300), (300, 3000, 200), (520, 6000, 100), (2600, 96, 1400)])
def test_gated_every_plan(M, K, F, mode):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("gated plans", M, K, F)
    x, w, b, dh = f32(rng, M, K), f32(rng, 2 * F, K, std=K ** -0.5), f32(rng, 2 * F, std=0.1), f32(rng, M, F)
    h, d = emu.gated_fwd(dev(x), dev(w), dev(b), mode=mode, save=True)
    h0 = emu.gated_fwd(dev(x), dev(w), dev(b), mode=mode)
    dx, dw, db = emu.gated_bwd(dev(dh), dev(x), dev(w), d, mode=mode)
    done()
    assert np.array_equal(host(h), host(h0))
    rows = np.unique(np.concatenate([np.arange(0, M, 29), np.arange(max(0, M - 40), M)]))
    wh, wd = gated_reference(x, w, b, "silu", mode)
    V(wh.val[rows], wh.err[rows]).check(host(h)[rows], "H")
    V(wd.val[rows], wd.err[rows]).check(host(d)[rows], "D")
    for got, v, name in zip((dx, dw, db), gated_grads(V(dh), x, w, mode, wd), ("dX", "dW", "db")):
        v.check(host(got), name)


@pytest.mark.parametrize("M,K,F,N", [(6144, 64, 300, 96), (6144, 16, 1000, 64), (700, 96, 520, 2100), (333, 40, 50, 2500)])
@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
def test_gated_ffn_backward_every_plan(M, K, F, N, mode):
    """The block's backward pass where dY W_out is chained or split."""
    check_ffn(rng_of("ffn plans", M, K, F, N), M, K, F, N, "silu", mode, residual=True)


@pytest.mark.parametrize("act", ACTS)
def test_large_preactivations_stay_finite(act):
    """Pre-activations of any finite size: values and derivatives are finite
    and at their limits."""
    import fp32_emulated_gemm_gb300 as emu
    z = np.array([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 30.0, -30.0, 104.0, -104.0, 1e4, -1e4, 3e18, -3e18, 1e30, -1e30,
                  3e38, -3e38], np.float32)
    n = z.size
    x, w = np.ones((1, 4), np.float32), np.zeros((n, 4), np.float32)
    dy = np.ones((1, n), np.float32)
    for rows in (1, 1040):                       # the few-row form and the tiles
        xr, dyr = np.repeat(x, rows, 0), np.repeat(dy, rows, 0)
        y, zz = emu.linear_act_fwd(dev(xr), dev(w), dev(z), act=act, save=True)
        dx, dw, db = emu.linear_act_bwd(dev(dyr), dev(xr), dev(w), zz, act=act)
        h = emu.gated_fwd(dev(xr), dev(np.concatenate([w, w])), dev(np.concatenate([z, np.ones(n, np.float32)])), act=act)
        done()
        a, d = R.act64(act, z.astype(np.float64).clip(-1e30, 1e30) if act == "gelu_tanh" else z.astype(np.float64))
        a = np.where(np.isfinite(a), a, np.maximum(z, 0)).astype(np.float64)
        d = np.where(np.isfinite(d), d, z > 0)
        a = np.where(np.abs(z) > 1e18, z if act == "none" else np.maximum(z, 0), a)
        d = np.where(np.abs(z) > 1e18, 1.0 if act == "none" else z > 0, d)
        # relative to the value, and in the negative tail, where 1 + erf and
        # exp of a rounded argument have only absolute accuracy, to |z| <= 6
        # (beyond it all of them are below u)
        bound = 16 * R.U * (np.abs(a) + np.abs(z).clip(0, 6))
        V(np.repeat(a[None], rows, 0), bound).check(host(y), "Y")
        V(np.repeat(a[None], rows, 0), bound).check(host(h), "H")
        V(d * rows, 64 * R.U * rows * (1 + np.abs(z).clip(0, 100))).check(host(db), "db")


# ------------------------------------------------------------ differences --
def directional(f, args, i, rng, h):
    """(direction, central difference of the scalar f along it in args[i])."""
    v = rng.standard_normal(args[i].shape)
    plus, minus = list(args), list(args)
    plus[i], minus[i] = args[i] + h * v, args[i] - h * v
    return v, (f(*plus) - f(*minus)) / (2 * h)


def check_differences(f, args, grads, names, rng):
    """The gradients against differences of the definition along random
    directions: h = 1e-4 leaves a truncation error of about h^2 and a
    rounding error of about 1e-16 / h of f's terms; the FP32 gradients' own
    error is their bound."""
    for i, (g, name) in enumerate(zip(grads, names)):
        got, bound = g
        v, d = directional(f, args, i, rng, 1e-4)
        allowed = float((bound * np.abs(v)).sum()) + 1e-6 * float((np.abs(got) * np.abs(v)).sum()) + 1e-9
        assert abs(float((got * v).sum()) - d) <= allowed, f"{name}: {float((got * v).sum())} against {d} +- {allowed}"


def test_layer_norm_gradient_against_differences():
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("ln differences")
    M, N = 6, 50
    x, w, b, c = f32(rng, M, N), f32(rng, N, mean=1.0, std=0.2), f32(rng, N), f32(rng, M, N)
    y, mean, rstd = emu.layer_norm_fwd(dev(x), dev(w), dev(b))
    got = [host(t).astype(np.float64) for t in emu.layer_norm_bwd(dev(c), dev(x), dev(w), mean, rstd)]
    want = R.layer_norm_grads(c, x.astype(np.float64), w, EPS)

    def f(x, w, b):
        mu = x.mean(1, keepdims=True)
        return float((((x - mu) / np.sqrt(((x - mu) ** 2).mean(1, keepdims=True) + EPS) * w + b) * c).sum())

    args = [a.astype(np.float64) for a in (x, w, b)]
    check_differences(f, args, [(g, v.err) for g, v in zip(got, want)], ("dX", "dweight", "dbias"), rng)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gated_ffn_gradient_against_differences(act):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("ffn differences", act)
    M, K, F, N = 10, 24, 36, 20
    x, wi, bi, wo, bo, c = (f32(rng, M, K), f32(rng, 2 * F, K, std=0.3), f32(rng, 2 * F), f32(rng, N, F, std=0.3),
                            f32(rng, N), f32(rng, M, N))
    y, d, h = emu.gated_ffn_fwd(*(dev(a) for a in (x, wi, bi, wo, bo)), act=act, save=True)
    got = [host(t).astype(np.float64) for t in emu.gated_ffn_bwd(dev(c), dev(x), dev(wi), dev(wo), d, h, act=act)]
    wh, wd = gated_reference(x, wi, bi, act, "bf16x9")
    dh = R.product(c, wo, "bf16x9")
    want = (*gated_grads(dh, x, wi, "bf16x9", wd), R.product(V(c).T, wh, "bf16x9"), R.column_sum(c))

    def f(x, wi, bi, wo, bo):
        z = x @ wi.T + bi
        return float(((R.act64(act, z[:, :F])[0] * z[:, F:]) @ wo.T + bo).ravel() @ c.astype(np.float64).ravel())

    args = [a.astype(np.float64) for a in (x, wi, bi, wo, bo)]
    check_differences(f, args, [(a, v.err) for a, v in zip(got, want)], ("dX", "dW_in", "db_in", "dW_out", "db_out"), rng)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "none"])
def test_linear_act_gradient_against_differences(act):
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("linear differences", act)
    M, K, N = 12, 28, 20
    x, w, b, c = f32(rng, M, K), f32(rng, N, K, std=0.3), f32(rng, N), f32(rng, M, N)
    y, z = emu.linear_act_fwd(dev(x), dev(w), dev(b), act=act, save=True)
    got = [host(t).astype(np.float64) for t in emu.linear_act_bwd(dev(c), dev(x), dev(w), z, act=act)]
    want = linear_act_reference(x, w, b, act, None, c, "bf16x9")[2:]
    f = lambda x, w, b: float((R.act64(act, x @ w.T + b)[0] * c).sum())
    args = [a.astype(np.float64) for a in (x, w, b)]
    check_differences(f, args, [(a, v.err) for a, v in zip(got, want)], ("dX", "dW", "db"), rng)


# ------------------------------------------- strides, alignment, streams --
def strided(a, how):
    """`a` on the device under another layout with the same values."""
    import torch
    r, c = a.shape
    if how == "padded":
        buf = torch.full((r, c + 8 - c % 4), float("nan"), device=_gpu.device())
        v = buf[:, :c]
    elif how == "offset":                      # rows off 16-byte boundaries
        buf = torch.full((r, c + 3), float("nan"), device=_gpu.device())
        v = buf[:, 1:c + 1]
    else:                                      # columns contiguous
        buf = torch.full((c, r), float("nan"), device=_gpu.device())
        v = buf.t()
    v.copy_(torch.from_numpy(a))
    return v


@pytest.mark.parametrize("how", ["padded", "offset", "transposed"])
def test_layouts(how):
    """Padded rows, unaligned rows and transposed matrices: nothing reads the
    padding (NaN), and the tiles give what dense matrices do, bit for bit."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    lay = lambda a: strided(a, how)
    for M, K, F, N in ((1, 32, 24, 40), (5, 32, 24, 40), (4, 35, 23, 41), (70, 37, 23, 45), (1070, 36, 24, 44), (1070, 37, 23, 45)):
        check_ffn(rng_of("layouts", M, K), M, K, F, N, "silu", "bf16x9", residual=True, lay=lay)
    rng = rng_of("layouts")
    M, K, F = 1070, 36, 24
    x, wi, dh, b = f32(rng, M, K), f32(rng, 2 * F, K), f32(rng, M, F), f32(rng, 2 * F + 1)

    def run(m):
        h, z = emu.gated_fwd(m(x), m(wi), dev(b)[1:], save=True)
        return [h, z, *emu.gated_bwd(m(dh), m(x), m(wi), z), *emu.linear_act_fwd(m(x), m(wi), dev(b)[1:], act="gelu", save=True)]

    for p, q in zip(run(dev), run(lay)):
        assert torch.equal(p, q)
    # what the forward pass saved, in another layout
    wo, dy = f32(rng, 45, F), f32(rng, M, 45)
    y, d, h = emu.gated_ffn_fwd(dev(x), dev(wi), None, dev(wo), dev(b)[1:46], save=True)
    ya, da = emu.linear_act_fwd(dev(x), dev(wi), act="silu", save=True)
    want = [*emu.gated_ffn_bwd(dev(dy), dev(x), dev(wi), dev(wo), d, h), *emu.linear_act_bwd(d, dev(x), dev(wi), da, act="silu")]
    sd, sh, sa = (lay(host(t)) for t in (d, h, da))
    got = [*emu.gated_ffn_bwd(lay(dy), lay(x), lay(wi), lay(wo), sd, sh), *emu.linear_act_bwd(sd, lay(x), lay(wi), sa, act="silu")]
    for i, (p, q) in enumerate(zip(want, got)):
        if i == 7:                             # the layer's bias gradient: row sums of unaligned rows, another order
            np.testing.assert_allclose(host(p), host(q), rtol=0, atol=2 * (M / 32 + 96) * R.U * float((d * da).abs().sum(0).max()))
        else:
            assert torch.equal(p, q), i
    for N in (36, 300, 2000):
        x, dy, w = f32(rng, 9, N), f32(rng, 9, N), f32(rng, N)
        y, mean, rstd = emu.layer_norm_fwd(lay(x), dev(w))
        got = emu.layer_norm_bwd(lay(dy), lay(x), dev(w), mean, rstd, add=lay(x))
        R.layer_norm(x.astype(np.float64), w, None, EPS)[0].check(host(y), "Y")
        for g, v, name in zip(got, R.layer_norm_grads(dy, x.astype(np.float64), w, EPS, x), ("dX", "dweight", "dbias")):
            v.check(host(g), name)
    done()


def test_outputs_stay_inside_their_matrix():
    """`out` in the middle of a guarded buffer: nothing outside it changes."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("guard")
    for M, K, F, N in ((3, 20, 20, 33), (150, 40, 70, 131), (1150, 40, 70, 131)):
        x, w, wi, wo = f32(rng, M, K), f32(rng, N, K), f32(rng, 2 * F, K), f32(rng, N, F)
        guard = torch.full((M + 2, N + 8 - N % 4), 7.5, device=_gpu.device())
        view = guard[1:M + 1, :N]
        calls = [lambda o: emu.linear_act_fwd(dev(x), dev(w), act="silu", out=o),
                 lambda o: emu.gated_ffn_fwd(dev(x), dev(wi), None, dev(wo), None, out=o),
                 lambda o: emu.layer_norm_fwd(dev(f32(rng_of("g", M), M, N)), out=o)[0]]
        for call in calls:
            guard.fill_(7.5)
            got = call(view)
            assert got.data_ptr() == view.data_ptr() and torch.equal(view, call(None))
            rest = guard.clone()
            rest[1:M + 1, :N] = 7.5
            assert bool((rest == 7.5).all())
    done()


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("M,K,F,N", [(5, 36, 23, 31), (1061, 36, 71, 33), (1150, 40, 128, 256), (700, 260, 901, 300)])
def test_every_output_stays_inside_its_matrix(M, K, F, N, mode):
    """Through the C entry points, every output in the middle of a buffer whose
    other words hold a pattern: none of them changes, and every output word
    is written."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("guards", M, K, F, N)
    pattern = torch.from_numpy(np.array([0x7FC0DEAD], np.uint32).view(np.float32)).to(_gpu.device())
    made = []

    def out(r, c):
        ld = (c + 3) // 4 * 4 + 8
        buf = pattern.expand((r + 2) * ld).contiguous()
        made.append((buf, r, c, ld))
        return buf[ld + 4:], ld               # (a view: its address is the matrix's)

    x, wi, wo = dev(f32(rng, M, K)), dev(f32(rng, 2 * F, K, std=0.2)), dev(f32(rng, N, F, std=0.2))
    bi, bo, dy, w = dev(f32(rng, 2 * F)), dev(f32(rng, N)), dev(f32(rng, M, N)), dev(f32(rng, K))
    (d, ldd), (h, ldh), (y, ldy), (dz, lddz) = out(M, 2 * F), out(M, F), out(M, N), out(M, 2 * F)
    (dx, lddx), (dwi, lddwi), (dbi, _), (dwo, lddwo), (dbo, _) = out(M, K), out(2 * F, K), out(1, 2 * F), out(N, F), out(1, N)
    m = emu.MODES[mode]
    emu.emu_gated_ffn_fwd(m, emu.EMU_ACT_SILU, M, K, F, N, x, K, wi, K, bi, wo, F, bo, None, 0, d, ldd, h, ldh, y, ldy)
    emu.emu_gated_ffn_bwd(m, M, K, F, N, dy, N, x, K, wi, K, wo, F, d, ldd, h, ldh, dz, lddz, dx, lddx, dwi, lddwi, dbi,
                          dwo, lddwo, dbo)
    (d2, ldd2), (y2, ldy2), (dz2, lddz2), (db2, _) = out(M, N), out(M, N), out(M, N), out(1, N)
    emu.emu_linear_act_fwd(m, emu.EMU_ACT_GELU, M, N, K, x, K, wi if N <= 2 * F else dev(f32(rng, N, K)), K, None, dy, N, d2,
                           ldd2, y2, ldy2)
    emu.emu_linear_act_bwd(m, M, N, K, dy, N, x, K, wi, K, d2, ldd2, dz2, lddz2, None, 0, None, 0, db2)
    (n, ldn), (dn, lddn), (dw, _), (db, _), (mean, _), (rstd, _) = (out(M, K), out(M, K), out(1, K), out(1, K), out(1, M),
                                                                    out(1, M))
    emu.emu_layer_norm_fwd(M, K, x, K, w, None, 1e-5, n, ldn, mean, rstd)
    emu.emu_layer_norm_bwd(M, K, x, K, x, K, w, mean, rstd, None, 0, dn, lddn, dw, db)
    done()
    for i, (buf, r, c, ld) in enumerate(made):
        words = buf.cpu().numpy().view(np.uint32)
        inside = np.zeros(words.size, bool)
        for k in range(r):
            inside[ld + 4 + k * ld:ld + 4 + k * ld + c] = True
        assert np.all(words[~inside] == 0x7FC0DEAD), f"output {i}: a store outside the matrix"
        assert np.all(np.isfinite(words[inside].view(np.float32))), f"output {i}: not all written"


def test_other_stream():
    """The calls run on the current stream: work queued there before and
    after them is ordered with them."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("stream")
    M, K, F = 1600, 128, 96
    x, wi, wo, dy = f32(rng, M, K), f32(rng, 2 * F, K, std=0.1), f32(rng, K, F, std=0.1), f32(rng, M, K)
    args = [dev(a) for a in (x, wi, wo, dy)]

    def step(x, wi, wo, dy):
        y, z, h = emu.gated_ffn_fwd(x, wi, None, wo, None, residual=x, save=True)
        g = emu.gated_ffn_bwd(dy, x, wi, wo, z, h)
        n, mean, rstd = emu.layer_norm_fwd(y)
        return [y, n, *[t for t in g if t is not None], *emu.layer_norm_bwd(dy, y, None, mean, rstd)]

    want = step(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.zeros(1 << 26, device=_gpu.device())
        late = [torch.zeros_like(a) for a in args]
        for _ in range(4):
            big.add_(1.0)                      # keeps the stream busy before the inputs are written
        for d, a in zip(late, args):
            d.copy_(a)
        got = step(*late)
        for d in late:
            d.fill_(float("nan"))
    side.synchronize()
    assert emu.emu_stream_check(side) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
def test_backward_products_side_by_side(mode):
    """The two products of a backward pass that share the GPU (small ones) and
    the ones that run in turn (many waves): right either way, and the calls
    after them wait for both."""
    import fp32_emulated_gemm_gb300 as emu
    for M, N, K in ((1100, 300, 500), (64, 1024, 700), (5000, 96, 80), (3000, 1500, 700)):
        rng = rng_of("side", M, N, K)
        x, w, dy = f32(rng, M, K), f32(rng, N, K, std=K ** -0.5), f32(rng, M, N)
        xd, wd, dyd = dev(x), dev(w), dev(dy)
        outs = []
        for rep in range(3):
            dx, dw, db = emu.linear_act_bwd(dyd, xd, wd, mode=mode)
            outs.append([host(emu.linear_fwd(dx, wd, mode=mode)), host(dx), host(dw), host(db)])  # dX used at once
        done()
        for other in outs[1:]:
            for p, q in zip(outs[0], other):
                assert np.array_equal(p, q)
        rows = np.arange(0, M, max(1, M // 200))
        R.product(V(dy[rows]), w, mode).check(outs[0][1][rows], "dX")
        cols = np.arange(0, N, max(1, N // 60))
        R.product(V(dy[:, cols]).T, x, mode).check(outs[0][2][cols], "dW")
        R.column_sum(V(dy)).check(outs[0][3], "db")


def test_captured_in_a_graph():
    """A training step captured after a warm-up on the capturing stream: each
    replay gives what the calls give on the inputs then in place."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("graph")
    M, K, F = 1400, 96, 130
    x, wi, wo, dy = (dev(f32(rng, *s)) for s in ((M, K), (2 * F, K), (K, F), (M, K)))

    def step():
        n, mean, rstd = emu.layer_norm_fwd(x)
        y, d, h = emu.gated_ffn_fwd(n, wi, None, wo, None, residual=x, save=True)
        g = emu.gated_ffn_bwd(dy, n, wi, wo, d, h)
        dx, dw, db = emu.layer_norm_bwd(g[0], x, None, mean, rstd, add=dy)
        return [y, dx, *g[1:], emu.linear_act_fwd(dx, wi, act="gelu")]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for rep in range(3):
        x.copy_(dev(f32(rng, M, K)))
        dy.copy_(dev(f32(rng, M, K)))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    done()


def test_offsets_beyond_32_bits():
    """Matrices of more than 2^31 elements: the last rows are right and the
    first ones too."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("long")
    M, K, F = 530_000, 12, 2048                    # D and dZ: 2.17e9 elements
    rows = np.concatenate([np.arange(0, M, 100_003), np.arange(M - 5, M)])
    x, w, b = f32(rng, M, K), f32(rng, 2 * F, K, std=0.3), f32(rng, 2 * F, std=0.1)
    dh = torch.zeros((M, F), device=_gpu.device())
    some = f32(rng, len(rows), F)
    dh[torch.from_numpy(rows).to(_gpu.device())] = dev(some)
    xd, wd = dev(x), dev(w)
    h, d = emu.gated_fwd(xd, wd, dev(b), save=True)
    at = torch.from_numpy(rows).to(_gpu.device())
    wh, wd64 = gated_reference(x[rows], w, b, "silu", "bf16x9")
    wh.check(host(h[at]), "H")
    wd64.check(host(d[at]), "D")
    dx, dw, db = emu.gated_bwd(dh, xd, wd, d)
    done()
    want = gated_grads(V(some), x[rows], w, "bf16x9", wd64)
    want[0].check(host(dx[at]), "dX")
    # the other rows of dH are zero; the products' bound counts all of them
    dz = beside(V(some) * wd64.cols(0, F), V(some) * wd64.cols(F, 2 * F))
    V(want[1].val, dz.err.T @ np.abs(x[rows]) + R.TERMS["bf16x9"](M) * R.U * (np.abs(dz.val).T @ np.abs(x[rows]))).check(host(dw), "dW")
    V(want[2].val, dz.err.sum(0) + (M / 32 + 96) * R.U * np.abs(dz.val).sum(0)).check(host(db), "db")
    del h, d, dh, dx, dw
    N = 4112                                       # 2.18e9 elements
    x = torch.empty((M, N), device=_gpu.device()).normal_()
    wn, bn = f32(rng, N), f32(rng, N)
    y, mean, rstd = emu.layer_norm_fwd(x, dev(wn), dev(bn))
    xs = host(x[at]).astype(np.float64)
    R.layer_norm(xs, wn, bn, EPS)[0].check(host(y[at]), "Y")
    dx, dwn, dbn = emu.layer_norm_bwd(y, x, dev(wn), mean, rstd)
    done()
    ys = host(y[at])
    R.layer_norm_grads(ys, xs, wn, EPS)[0].check(host(dx[at]), "dX of the norm")


def test_degenerate_sizes():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    new = lambda *s: torch.ones(s, device=_gpu.device())
    y, mean, rstd = emu.layer_norm_fwd(new(0, 8), new(8), new(8))
    assert y.shape == (0, 8)
    dx, dw, db = emu.layer_norm_bwd(new(0, 8), new(0, 8), new(8), mean, rstd)
    assert dx.shape == (0, 8) and not dw.any() and not db.any()
    assert emu.layer_norm_fwd(new(3, 0))[0].shape == (3, 0)
    for M in (0, 3, 1040):
        # no input features: the bias alone
        y = emu.linear_act_fwd(new(M, 0), new(5, 0), new(5) * 2, act="silu", residual=new(M, 5))
        want = 2 / (1 + np.exp(-2.0)) + 1
        assert y.shape == (M, 5) and bool((abs(y - want) < 1e-6).all())
        # no rows, or no hidden features: zero sums and the output bias
        z = torch.empty((M, 0), device=_gpu.device())
        y, z, h = emu.gated_ffn_fwd(new(M, 4), new(0, 4), new(0), new(6, 0), new(6) * 3, residual=new(M, 6), save=True)
        assert y.shape == (M, 6) and bool((y == 4).all())
        g = emu.gated_ffn_bwd(new(M, 6), new(M, 4), new(0, 4), new(6, 0), z, h)
        assert not g[0].any() and g[1].shape == (0, 4) and bool((g[4] == M).all())
    y, z = emu.linear_act_fwd(new(0, 4), new(6, 4), new(6), act="gelu", save=True)
    dx, dw, db = emu.linear_act_bwd(new(0, 6), new(0, 4), new(6, 4), z, act="gelu")
    assert dx.shape == (0, 4) and not dw.any() and not db.any()
    assert emu.linear_act_fwd(new(3, 4), new(0, 4)).shape == (3, 0)
    done()


def test_allocation_failure_enqueues_nothing():
    """Each operator makes sure of its buffers first: with the library's next
    allocation made to fail it returns the status and writes nothing."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("alloc")
    M, K, N = 300, 3000, 260
    x, w, dy = dev(f32(rng, M, K)), dev(f32(rng, N, K)), dev(f32(rng, M, N))
    out = torch.full((M, N), 7.0, device=_gpu.device())
    calls = [lambda: emu.linear_act_fwd(x, w, act="gelu", out=out),
             lambda: emu.linear_act_bwd(dy, x, w, dy, act="gelu"),
             lambda: emu.gated_ffn_fwd(x, w, None, dev(f32(rng, N, N // 2)), None, out=out)]
    for call in calls:
        emu.emu_shutdown()
        emu.emu_debug_fail_allocations(1)
        try:
            with pytest.raises(emu.EmuError) as e:
                call()
            assert e.value.status == 4
        finally:
            emu.emu_debug_fail_allocations(0)
        done()
        assert bool((out == 7).all())
        call()
        done()
        out.fill_(7.0)


def test_refusals():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    new = lambda *s, **k: torch.zeros(s, device=_gpu.device(), **k)
    x, w = new(6, 8), new(10, 8)
    with pytest.raises(ValueError):
        emu.linear_act_fwd(x, new(10, 9))
    with pytest.raises(ValueError):
        emu.linear_act_fwd(x, w, act="tanh")
    with pytest.raises(ValueError):
        emu.linear_act_fwd(x, w, new(9))
    with pytest.raises(ValueError):
        emu.linear_act_fwd(x, w, residual=new(6, 9))
    with pytest.raises(ValueError):
        emu.linear_act_fwd(x, w, out=new(5, 10))
    with pytest.raises(ValueError):
        emu.linear_act_bwd(new(6, 10), x, w, None, act="silu")
    with pytest.raises(TypeError):
        emu.linear_act_fwd(x.double(), w)
    with pytest.raises(TypeError):
        emu.linear_act_fwd(x.cpu(), w)
    with pytest.raises(ValueError):
        emu.gated_fwd(x, new(9, 8))
    with pytest.raises(ValueError):
        emu.gated_ffn_fwd(x, w, None, new(4, 6), None)
    with pytest.raises(ValueError):
        emu.layer_norm_fwd(new(8))
    with pytest.raises(ValueError):
        emu.layer_norm_fwd(x, new(7))
    with pytest.raises(KeyError):
        emu.linear_act_fwd(x, w, mode="fp64")
    with pytest.raises(emu.EmuError) as e:
        emu.layer_norm_fwd(x, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(emu.EmuError) as e:      # an output off the 16-byte boundary, in a product of many rows
        emu.linear_act_fwd(new(1040, 8), w, out=new(1040, 12)[:, 1:11])
    assert e.value.status == 2
    done()


# ---------------------------------------------------------------- modules --
def test_modules_match_torch():
    """EmuLayerNorm, EmuLinearAct, EmuGatedFFN and EmuFeedForward, forward and
    backward, against the same layers in float64 on the CPU."""
    import torch
    import torch.nn.functional as F
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(0)

    def compare(module, reference, *inputs):
        ins = [torch.randn(s, device="cuda").requires_grad_() for s in inputs]
        y = module(*ins)
        g = torch.randn_like(y)
        y.backward(g)
        m64 = {n: p.detach().double().cpu().requires_grad_() for n, p in module.named_parameters()}
        ins64 = [t.detach().double().cpu().requires_grad_() for t in ins]
        y64 = reference(m64, *ins64)
        y64.backward(g.double().cpu())
        pairs = [(y, y64)] + [(a.grad, b.grad) for a, b in zip(ins, ins64)]
        pairs += [(p.grad, m64[n].grad) for n, p in module.named_parameters()]
        for a, b in pairs:
            assert a.shape == b.shape
            assert float((a.detach().double().cpu() - b).abs().max()) <= 1e-5 * float(b.abs().max())

    compare(emu.EmuLayerNorm(96).cuda(), lambda p, x: F.layer_norm(x, (96,), p["weight"], p["bias"]), (2, 30, 96))
    compare(emu.EmuLayerNorm((4, 24)).cuda(), lambda p, x: F.layer_norm(x, (4, 24), p["weight"], p["bias"]), (50, 4, 24))
    compare(emu.EmuLinearAct(64, 80, act="gelu").cuda(),
            lambda p, x, r: F.gelu(x @ p["weight"].T + p["bias"]) + r, (3, 70, 64), (3, 70, 80))
    compare(emu.EmuLinearAct(64, 80, act="gelu_tanh", bias=False).cuda(),
            lambda p, x: F.gelu(x @ p["weight"].T, approximate="tanh"), (130, 64))

    def ffn(p, x, pre=""):
        z = x @ p[pre + "weight_in"].T + p[pre + "bias_in"]
        g, u = z.chunk(2, -1)
        return (F.silu(g) * u) @ p[pre + "weight_out"].T + p[pre + "bias_out"]

    compare(emu.EmuGatedFFN(64, 100, 48).cuda(), ffn, (2, 33, 64))
    compare(emu.EmuFeedForward(64, 100, mode="tf32x3").cuda(),
            lambda p, x: x + ffn(p, F.layer_norm(x, (64,), p["norm.weight"], p["norm.bias"]), "ffn."), (2, 65, 64))
    done()


def test_module_wants_only_some_gradients():
    """Frozen parameters and inputs without gradients; a broadcast upstream
    gradient (expanded, stride 0)."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(1)
    m = emu.EmuFeedForward(32, 40).cuda()
    x = torch.randn(50, 32, device="cuda")
    m(x).sum().backward()
    full = {n: p.grad.clone() for n, p in m.named_parameters()}
    m.zero_grad()
    for n, p in m.named_parameters():
        p.requires_grad_(n.startswith("ffn.weight_out") or n == "norm.bias")
    m(x).sum().backward()
    for n, p in m.named_parameters():
        if p.requires_grad:
            assert torch.equal(p.grad, full[n]), n
        else:
            assert p.grad is None
    xg = x.clone().requires_grad_()
    for p in m.parameters():
        p.requires_grad_(False)
    m(xg).sum().backward()
    assert xg.grad.shape == x.shape and bool(torch.isfinite(xg.grad).all())
    with torch.no_grad():
        assert torch.equal(m(x), m(xg).detach())
    done()


def test_block_trains():
    """The sub-layer as it is used: a few steps of gradient descent on a
    regression lower the loss as the same layer in float64 does."""
    import torch
    import torch.nn.functional as F
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(2)
    m = emu.EmuFeedForward(48, 96).cuda()
    p64 = {n: p.detach().double().cpu().requires_grad_() for n, p in m.named_parameters()}
    x, t = torch.randn(400, 48, device="cuda"), torch.randn(400, 48, device="cuda")
    x64, t64 = x.double().cpu(), t.double().cpu()
    opt, opt64 = torch.optim.SGD(m.parameters(), 0.5), torch.optim.SGD(p64.values(), 0.5)
    losses = []
    for _ in range(8):
        opt.zero_grad(), opt64.zero_grad()
        loss = ((m(x) - t) ** 2).mean()
        loss.backward()
        opt.step()
        z = F.layer_norm(x64, (48,), p64["norm.weight"], p64["norm.bias"]) @ p64["ffn.weight_in"].T + p64["ffn.bias_in"]
        g, u = z.chunk(2, -1)
        y = x64 + (F.silu(g) * u) @ p64["ffn.weight_out"].T + p64["ffn.bias_out"]
        loss64 = ((y - t64) ** 2).mean()
        loss64.backward()
        opt64.step()
        losses.append((float(loss.detach()), float(loss64.detach())))
    assert losses[-1][0] < losses[0][0]
    for a, b in losses:
        assert abs(a - b) <= 1e-5 * b
    done()
