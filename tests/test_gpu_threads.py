"""Several host threads on one stream: the calls' launches share the stream's
buffers, and each call's results are its own."""
import threading

import numpy as np
import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu


def rand(rng, *shape):
    return _gpu.to_dev(rng.standard_normal(shape).astype(np.float32))


def calls(emu, seed):
    """Calls of different sizes that use every buffer: sums over rows, copies of
    odd operands, products split along k, split ahead and side by side."""
    rng = np.random.default_rng(seed)
    M, N, K = 1100 + 37 * seed, 299, 501 + 10 * seed
    x, w, dy, d = rand(rng, M, K), rand(rng, N, K), rand(rng, M, N), rand(rng, M, N)
    mean, rstd = rand(rng, M), rand(rng, M)
    a, b = rand(rng, 300, 3000), rand(rng, 260, 3000)
    big = rand(rng, 1400, 301 + seed)
    w2 = rand(rng, 450, 301 + seed)

    def sgemm():
        return [emu.sgemm(a, b, transB=True), emu.sgemm(a, b, transB=True, mode="tf32x3")]

    return [lambda: emu.linear_act_bwd(dy, x, w, d, act="gelu", mode="tf32x3"),
            lambda: emu.layer_norm_bwd(x, x, None, mean, rstd),
            lambda: emu.linear_act_bwd(dy, x, w),
            lambda: [emu.gated_fwd(big, w2, mode="tf32x3")],
            sgemm]


@pytest.mark.parametrize("own_stream", [False, True])
def test_threads_on_one_stream(own_stream):
    import contextlib
    import torch
    import fp32_emulated_gemm_gb300 as emu
    sets = [calls(emu, seed) for seed in range(3)]
    want = [[[t.clone() for t in call()] for call in s] for s in sets]
    torch.cuda.synchronize()
    emu.emu_shutdown()                       # the buffers grow again while the threads run
    stream = torch.cuda.Stream()
    wrong, start = [], threading.Barrier(len(sets))

    def worker(i):
        try:
            with torch.cuda.stream(stream) if own_stream else contextlib.nullcontext():
                start.wait(60)
                for rep in range(60):
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
