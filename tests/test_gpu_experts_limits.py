"""The operators of a layer of experts where calls meet limits or one another."""
import threading

import numpy as np
import pytest

from tests import _running as R
from tests._running import U, V
from tests.test_gpu_experts import EPS, check_plan, expert_reference, ints, route_oracle
from tests.test_gpu_feed_forward import dev, done, f32, host, rng_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [8, 200])
def test_routes_of_many_experts_from_several_threads(M):
    """Calls on streams of their own, with more shared memory than a launch may have
    without asking and different amounts of it (one block; two launches): none takes
    another's away."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    sizes = [1024, 700, 1000, 690]
    sets = []
    for E in sizes:
        l = f32(rng_of("limits", M, E), M, E)
        plan, weights = emu.expert_route(dev(l), 2)
        done()
        check_plan(plan, route_oracle(l, 2, "chosen")[0], E)
        sets.append((dev(l), [t.clone() for t in (*plan, weights)]))
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(sizes))

    def worker(i):
        try:
            logits, want = sets[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                emu.expert_route(logits, 2)
                start.wait(60)
                for rep in range(1500):
                    plan, weights = emu.expert_route(logits, 2)
                    if rep % 100 == 0 and not all(torch.equal(a, b) for a, b in zip((*plan, weights), want)):
                        wrong.append((i, rep))
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(300)
    assert not any(t.is_alive() for t in threads)
    assert not wrong, wrong[:8]
    done()


@pytest.mark.parametrize("E,rows,K,F", [(8, 16, 256, 512), (64, 4, 64, 64), (8, 300, 128, 256)])
def test_passes_without_rows_end_before_what_follows(E, rows, K, F):
    """No expert has rows, and the next call on the stream gives the offsets other
    values: the pass before it reads the old ones alone and writes nothing.  (Forward
    on the CUDA cores: lots a warp, streaming, through shared memory.)"""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("norows", E, rows)
    x, wi, wo = dev(f32(rng, rows, K)), dev(f32(rng, E, 2 * F, K)), dev(f32(rng, E, K, F))
    some, none = ints([rows] * (E + 1)), ints([0] * (E + 1))
    full = ints([0] + [rows] * E)
    offsets = none.clone()
    h, y, d = (torch.full((rows, n), 7.0, device="cuda") for n in (F, K, 2 * F))
    for i in range(200):
        offsets.copy_(some if i % 2 else none)
        emu.emu_expert_ffn_fwd(0, 4, rows, E, K, F, K, x, K, offsets, wi, K, wo, F, d, 2 * F, h, F, y, K)
        offsets.copy_(full)
    done()
    assert all(bool((t == 7).all()) for t in (h, y, d))


@pytest.mark.parametrize("counts,K,F,N", [([3, 0, 9, 1], 256, 512, 260), ([2] * 40 + [70], 64, 64, 64), ([5, 200, 0, 40], 132, 65, 36)])
def test_backward_passes_that_write_the_same_dz(counts, K, F, N):
    """Passes of different inputs one behind the other, on the CUDA cores, into one dZ
    and one set of gradients: each reads its own dZ, not the last one's."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("samedz", sum(counts), K)
    E, offsets = len(counts), ints(np.concatenate([[0], np.cumsum(counts)]))
    rows, pad = sum(counts), lambda n: (n + 3) // 4 * 4
    wi, wo = dev(f32(rng, E, 2 * F, K)), dev(f32(rng, E, N, F))
    plan = emu.ExpertPlan(None, None, None, offsets)
    sets = []
    for _ in range(3):
        x, dy = dev(f32(rng, rows, K)), dev(f32(rng, rows, N))
        y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
        sets.append((x, dy, d, h, emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)))
    done()
    new = lambda r, c: torch.empty_strided((r, c), (pad(c), 1), device="cuda")
    dz, dx, dwi, dwo = new(rows, 2 * F), new(rows, K), new(E * 2 * F, K), new(E * N, F)
    for i in range(60):
        x, dy, d, h, want = sets[i % 3]
        emu.emu_expert_ffn_bwd(0, rows, E, K, F, N, dy, N, x, K, offsets, wi, K, wo, F, d, d.stride(0), h, h.stride(0), dz, pad(2 * F),
                               dx, pad(K), dwi, pad(K), dwo, pad(F))
        got = dx, dwi.unflatten(0, (E, 2 * F)), dwo.unflatten(0, (E, N))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    done()


def skewed(E, rows, hot, rng):
    """Counts of `rows` rows, all but a few of them expert `hot`'s."""
    counts = np.zeros(E, np.int64)
    others = rng.integers(0, E, size=min(E // 2, rows // 8))
    np.add.at(counts, others, 1)
    counts[hot] += rows - counts.sum()
    return counts


@pytest.mark.parametrize("E,rows,K,F,N", [(64, 2500, 64, 64, 64), (256, 9000, 36, 33, 20), (1024, 9000, 16, 8, 12), (8, 70, 700, 300, 260),
                                          (64, 600, 256, 260, 132), (128, 4096, 128, 128, 128), (3, 65, 64, 64, 64)])
@pytest.mark.parametrize("kind", ["one", "first", "last", "even"])
def test_backward_of_rows_on_one_expert(E, rows, K, F, N, kind):
    """All rows on one expert, or nearly all on the first or the last: the gradients,
    their bits in each wanted one alone and on every run; experts without rows get
    zeros."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("hot", E, rows, kind)
    counts = np.zeros(E, np.int64)
    if kind == "even":
        counts[:] = rows // E
        counts[:rows % E] += 1
    elif kind == "one":
        counts[E // 3] = rows
    else:
        counts = skewed(E, rows, 0 if kind == "first" else E - 1, rng)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    x, dy = f32(rng, rows, K), f32(rng, rows, N)
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    plan = emu.ExpertPlan(None, None, None, ints(offsets))
    X, DY, WI, WO = dev(x), dev(dy), dev(wi), dev(wo)
    y, d, h = emu.expert_ffn_fwd(X, WI, WO, plan, save=True)
    got = emu.expert_ffn_bwd(DY, X, WI, WO, d, h, plan)
    again = emu.expert_ffn_bwd(DY, X, WI, WO, d, h, plan)
    alone = [emu.expert_ffn_bwd(DY, X, WI, WO, d, h, plan, need=[j == i for j in range(3)])[i] for i in range(3)]
    done()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(got, again, alone))
    assert not bool(got[1][dev(counts == 0)].any()) and not bool(got[2][dev(counts == 0)].any())
    for e in np.flatnonzero(counts)[np.argsort(-counts[counts > 0])][:12]:
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        want = expert_reference(x[r], wi[e], wo[e], "silu", "bf16x9", dy[r])
        for g, w, name in zip((y[r], h[r], got[0][r], got[1][e], got[2][e]), want, ("Y", "H", "dX", "dW_in", "dW_out")):
            w.check(host(g), f"expert {e} {name}")


@pytest.mark.parametrize("E,rows,width", [(64, 2500, 64), (256, 12000, 64)])
def test_backward_time_of_rows_on_one_expert(E, rows, width):
    """The same rows, spread evenly and all on one expert: the pass's time does not
    grow with an expert's rows.  (It was 27 and 48 times the even one's where one
    block went through all of an expert's rows in order, which is far from the six
    that are allowed here.)"""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("hottime", E, rows)
    K = F = N = width
    x, dy, wi, wo = (dev(f32(rng, *s)) for s in ((rows, K), (rows, N), (E, 2 * F, K), (E, N, F)))
    even = ints(rows * np.arange(E + 1) // E)
    one = ints(np.where(np.arange(E + 1) > E // 3, rows, 0))
    best = []
    for offsets in (even, one):
        plan = emu.ExpertPlan(None, None, None, offsets)
        y, d, h = emu.expert_ffn_fwd(x, wi, wo, plan, save=True)
        run = lambda: emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
        times = []
        for _ in range(8):
            run()
            a, b = torch.cuda.Event(True), torch.cuda.Event(True)
            a.record()
            for _ in range(10):
                run()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    done()
    assert best[1] <= 6 * best[0], best


@pytest.mark.parametrize("N", [20000, 40003, 100000])
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_of_wide_rows_adds_its_squares_in_two_words(N, residual):
    """A large value and many whose squares are each below half of its last bit: sums
    in one word drop them wherever they meet it.  Each quad of squares is off by three
    roundings at most, their sum in two words by its last one; the mean and the
    addition of eps add three, the root halves those seven, and rounds, and so does
    the reciprocal: 5.5 in all."""
    import fp32_emulated_gemm_gb300 as emu
    small = np.float32(2.0 ** -12.25)
    x = np.full((3, N), small, np.float32)
    x[0, 0], x[1, N - 1], x[2, N // 2] = 1, 1, 1
    q = None
    if residual:                              # (the sums are exact: a half and a half)
        q = (x / 2).astype(np.float32)
        x = q.copy()
    y, s, rstd = emu.rms_norm_fwd(dev(x), residual=dev(q), eps=EPS)
    Q, scales, *_ = emu.rms_norm_quant(dev(x), residual=dev(q), eps=EPS)
    done()
    s64 = (x if q is None else x + q).astype(np.float64)
    want = 1 / np.sqrt((s64 ** 2).mean(1) + float(np.float32(EPS)))
    V(want, 5.6 * U * want).check(host(rstd), "rstd")
    y64 = s64 * want[:, None]
    V(y64, 6.7 * U * np.abs(y64)).check(host(y), "Y")
    wide = np.repeat(host(scales).astype(np.float64), 128, 1)[:, :N]
    assert np.all(np.abs(host(Q.float()) * wide - y64) <= 2.0 ** -4 * y64 * (1 + 8 * U) + 8 * U * y64 + 2.0 ** -10 * wide)


@pytest.mark.parametrize("counts,K,F,N,act", [
    ([3, 0, 5], 36, 100, 60, "silu"), ([1, 0, 0, 2], 700, 1540, 129, "gelu"), ([40, 17, 5, 33], 36, 2052, 1030, "gelu_tanh"),
    ([200, 0, 7, 120], 256, 512, 260, "silu"), ([1500, 0, 257, 900], 260, 387, 72, "silu"), ([5000, 0, 257, 3300], 64, 100, 60, "none")])
def test_saved_derivatives_and_outputs(counts, K, F, N, act):
    """D = [u a'(g) | a(g)], H and Y of each form of the forward pass against the
    definition."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("saved", sum(counts), K)
    E, offsets = len(counts), np.concatenate([[0], np.cumsum(counts)])
    x = f32(rng, sum(counts), K)
    wi, wo = f32(rng, E, 2 * F, K, std=K ** -0.5), f32(rng, E, N, F, std=F ** -0.5)
    y, d, h = emu.expert_ffn_fwd(dev(x), dev(wi), dev(wo), emu.ExpertPlan(None, None, None, ints(offsets)), act=act, save=True)
    done()
    assert d.shape == (sum(counts), 2 * F)
    for e in range(E):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        z = R.product(x[r], wi[e].T, "bf16x9")
        g, u = z.cols(0, F), z.cols(F, 2 * F)
        a = R.act_value(act, g) if act != "none" else g
        slope = R.act_grad(act, g) if act != "none" else V(np.ones_like(g.val))
        (u * slope).check(host(d[r, :F]), f"expert {e} u a'(g)")
        a.check(host(d[r, F:]), f"expert {e} a(g)")
        (a * u).check(host(h[r]), f"expert {e} H")
        R.product(a * u, wo[e].T, "bf16x9").check(host(y[r]), f"expert {e} Y")


@pytest.mark.parametrize("mode", ["bf16x9", "tf32x3"])
@pytest.mark.parametrize("M", [7, 100, 2048])
def test_one_expert_and_the_dense_block(M, mode):
    """One expert with every row and the gated block agree in D, H and Y within both
    calls' bounds (their sums are cut differently, so not bit for bit)."""
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("dense", M)
    K, F, N = 256, 512, 132
    x, wi, wo = f32(rng, M, K), f32(rng, 1, 2 * F, K, std=0.06), f32(rng, 1, N, F, std=0.04)
    y, d, h = emu.expert_ffn_fwd(dev(x), dev(wi), dev(wo), emu.ExpertPlan(None, None, None, ints([0, M])), mode=mode, save=True)
    h2, d2 = emu.gated_fwd(dev(x), dev(wi[0]), mode=mode, save=True)
    y2 = emu.linear_fwd(h2, dev(wo[0]), mode=mode)
    done()
    z = R.product(x, wi[0].T, mode)
    g, u = z.cols(0, F), z.cols(F, 2 * F)
    a, slope = R.act_value("silu", g), R.act_grad("silu", g)
    ud = u * slope
    for one, dense, want, name in ((d[:, :F], d2[:, :F], ud, "u a'(g)"), (d[:, F:], d2[:, F:], a, "a(g)"), (h, h2, a * u, "H"),
                                   (y, y2, R.product(a * u, wo[0].T, mode), "Y")):
        want.check(host(one), name)
        want.check(host(dense), name + " of the dense block")
        assert np.all(np.abs(host(one).astype(np.float64) - host(dense)) <= 2 * want.err + 2 * U * np.abs(want.val) + 1e-37), name


def test_chunks_of_rows_in_a_graph():
    """A captured backward pass whose replays meet other offsets than the capture did:
    even ones, all rows on one expert, none at all."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = rng_of("chunkgraph")
    E, rows, K, F, N = 64, 2500, 64, 65, 60
    x, dy, wi, wo = (dev(f32(rng, *s)) for s in ((rows, K), (rows, N), (E, 2 * F, K), (E, N, F)))
    kinds = [ints(rows * np.arange(E + 1) // E), ints(np.where(np.arange(E + 1) > 7, rows, 0)), ints([0] * (E + 1)),
             ints(np.concatenate([[5], np.full(E, 9)]))]
    offsets = kinds[0].clone()
    plan = emu.ExpertPlan(None, None, None, offsets)
    d, h = dev(f32(rng, rows, 2 * F)), dev(f32(rng, rows, F))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = emu.expert_ffn_bwd(dy, x, wi, wo, d, h, plan)
    for i in (0, 1, 2, 3, 1, 0):
        offsets.copy_(kinds[i])
        graph.replay()
        torch.cuda.synchronize()
        want = emu.expert_ffn_bwd(dy, x, wi, wo, d, h, emu.ExpertPlan(None, None, None, kinds[i]))
        torch.cuda.synchronize()
        r = slice(int(kinds[i][0]), int(kinds[i][-1]))
        assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2]), i
    done()
