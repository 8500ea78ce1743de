"""The operators of a layer of experts where calls meet limits or one another."""
import threading

import numpy as np
import pytest

from tests.test_gpu_experts import check_plan, ints, route_oracle
from tests.test_gpu_feed_forward import dev, done, f32, rng_of

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
