"""More of the feed-forward operators' host checks, without a GPU."""
import ctypes

import pytest

from fp32_emulated_gemm_gb300 import build as emu_build

INVALID, NOT_SUPPORTED = 1, 2


@pytest.fixture(scope="module")
def ff():
    emu_build.build()
    from fp32_emulated_gemm_gb300 import feed_forward
    return feed_forward


@pytest.fixture(scope="module")
def p():
    buf = (ctypes.c_float * 64)()
    yield (ctypes.cast(buf, ctypes.c_void_p).value + 15) & ~15


def test_the_blocks_backward_needs_what_it_uses(ff, p):
    """Without dX, dW_in and db_in neither D nor dZ, without dW_out no H.  (The
    call that has all it needs is stopped by dW_out's leading dimension.)"""
    def bwd(D=p, H=p, dZ=p, inner=None, dWo=p, lddwo=6):
        return ff._fn("emu_gated_ffn_bwd")(0, 8, 4, 4, 4, p, 4, p, 4, p, 4, p, 4, D, 8, H, 4, dZ, 8, inner, 4, None, 4, None,
                                           dWo, lddwo, p, None)
    assert bwd(D=None, dZ=None) == NOT_SUPPORTED
    assert bwd(D=None, dZ=None, H=None) == INVALID
    assert bwd(D=None, inner=p) == INVALID and bwd(dZ=None, inner=p) == INVALID
    assert bwd(dZ=p + 4, inner=p) == NOT_SUPPORTED
