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


def test_checks_come_before_the_copies_of_odd_operands(ff, p):
    """Operands off the 16-byte boundaries, which need a buffer and so the
    device, do not keep a wrong argument from being answered first."""
    odd = p + 4
    fn = lambda name, *a: ff._fn(name)(*a, None)
    la = lambda mode=0, Y=p, ldw=5: fn("emu_linear_act_fwd", mode, 1, 1040, 4, 5, odd, 5, odd, ldw, odd, odd, 7, None, 0, Y, 4)
    assert la(mode=9) == INVALID and la(ldw=4) == INVALID and la(Y=odd) == NOT_SUPPORTED
    lb = lambda mode=0, lddx=8: fn("emu_linear_act_bwd", mode, 1040, 4, 5, odd, 5, odd, 5, odd, 5, None, 0, None, 0, p, lddx, p, 8, p)
    assert lb(mode=9) == INVALID and lb(lddx=4) == INVALID and lb(lddx=6) == NOT_SUPPORTED
    gf = lambda mode=0, ldh=4: fn("emu_gated_fwd", mode, 4, 1040, 4, 5, odd, 5, odd, 5, odd, p, 8, p, ldh)
    assert gf(mode=9) == INVALID and gf(ldh=6) == NOT_SUPPORTED
    gb = lambda lddw=8: fn("emu_gated_bwd", 0, 1040, 4, 5, odd, 5, odd, 5, odd, 5, odd, 9, p, 8, p, 8, p, lddw, p)
    assert gb(lddw=4) == INVALID and gb(lddw=6) == NOT_SUPPORTED
    ff_ = lambda ldy=4: fn("emu_gated_ffn_fwd", 0, 4, 1040, 5, 4, 4, odd, 5, odd, 5, odd, odd, 5, odd, odd, 5, None, 0, p, 4, p, ldy)
    assert ff_(ldy=6) == NOT_SUPPORTED
    fb = lambda lddwi=8: fn("emu_gated_ffn_bwd", 0, 1040, 5, 4, 4, odd, 5, odd, 5, odd, 5, odd, 5, odd, 9, odd, 5, p, 8, p, 8,
                            p, lddwi, p, p, 4, p)
    assert fb(lddwi=4) == INVALID and fb(lddwi=6) == NOT_SUPPORTED
