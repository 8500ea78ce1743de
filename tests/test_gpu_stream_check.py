"""emu_stream_check on an idle stream: one read of one error word, whatever
kernels the library has."""
import statistics
import time

import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu


def test_the_check_costs_one_read():
    """At most two and a half times a synchronising 4-byte read by PyTorch (it is
    a synchronisation and such a read; a read for each of the library's four
    kernel files took 3.8 times)."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    word = torch.zeros(1, device=_gpu.device())

    def median(f):
        times = []
        for _ in range(100):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return statistics.median(times)

    assert emu.emu_stream_check() == 0
    check, read = (min(median(f) for _ in range(5)) for f in (emu.emu_stream_check, word.item))
    assert check <= 2.5 * read, (check, read)


def test_a_timeout_is_reported_once():
    import fp32_emulated_gemm_gb300 as emu
    emu.emu_selftest_wait_timeout(1_000_000)
    assert emu.emu_stream_check() == 6
    assert emu.emu_stream_check() == 0
