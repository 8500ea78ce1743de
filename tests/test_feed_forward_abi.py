"""The feed-forward operators' host side, without a GPU: the binding matches
the header, and argument errors are answered before any device work."""
import ctypes
import os
import re

import pytest

import fp32_emulated_gemm_gb300 as emu
from fp32_emulated_gemm_gb300 import build as emu_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    emu_build.build()
    from fp32_emulated_gemm_gb300 import feed_forward
    return feed_forward


def _header():
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "emu_gemm.h")).read(), flags=re.S)


def test_binding_signatures_match_the_header(ff):
    for name, kinds in ff._SIGNATURES.items():
        args = re.search(name + r"\((.*?)\)", _header(), re.S).group(1).split(",")
        assert args[-1].split()[0] == "emu_stream_t"
        want = "".join("p" if "*" in a else "n" if "int64_t" in a else "f" if "float" in a else "e" for a in args[:-1])
        assert kinds == want, name


def test_activation_enum_matches_the_binding(ff):
    enum = {m.group(1): int(m.group(2)) for m in re.finditer(r"(EMU_ACT_\w+)\s*=\s*(\d+)", _header())}
    assert enum == {"EMU_ACT_" + k.upper(): v for k, v in emu.ACTS.items()}
    for name, value in enum.items():
        assert getattr(emu, name) == value


def test_host_checks_answer_without_a_device(ff):
    buf = (ctypes.c_float * 64)()
    p = (ctypes.cast(buf, ctypes.c_void_p).value + 15) & ~15
    fn = lambda name, *a: ff._fn(name)(*a, None)
    INVALID, NOT_SUPPORTED = 1, 2
    ln = lambda M=4, N=4, X=p, ldx=4, eps=1e-5, Y=p, ldy=4: fn("emu_layer_norm_fwd", M, N, X, ldx, p, p, eps, Y, ldy, p, p)
    assert ln(M=-1) == INVALID and ln(ldx=3) == INVALID and ln(eps=-1.0) == INVALID and ln(X=None) == INVALID
    assert ln(N=2 ** 31) == NOT_SUPPORTED and ln(M=0) == 0 and ln(eps=float("nan")) == INVALID
    lb = lambda N=4, dX=p, lddx=4, add=None: fn("emu_layer_norm_bwd", 4, N, p, 4, p, 4, p, p, p, add, 4, dX, lddx, p, p)
    assert lb(lddx=3) == INVALID and lb(N=-1) == INVALID and lb(dX=None, add=p) == INVALID and lb(N=0) == 0
    la = lambda mode=0, act=1, M=1040, X=p, ldx=4, Y=p, ldy=4, r=None, ldr=0: fn(
        "emu_linear_act_fwd", mode, act, M, 4, 4, X, ldx, p, 4, p, r, ldr, None, 0, Y, ldy)
    assert la(mode=9) == INVALID and la(act=5) == INVALID and la(act=-1) == INVALID and la(ldy=3) == INVALID
    assert la(r=p, ldr=2) == INVALID and la(X=None) == INVALID and la(M=0) == 0
    assert la(Y=p + 4) == NOT_SUPPORTED and la(ldy=6) == NOT_SUPPORTED
    bw = lambda D=p, dZ=p, dX=p, lddx=4: fn("emu_linear_act_bwd", 0, 1040, 4, 4, p, 4, p, 4, p, 4, D, 4, dZ, 4, dX, lddx, p, 4, p)
    assert bw(dZ=None) == INVALID and bw(lddx=2) == INVALID and bw(lddx=6) == NOT_SUPPORTED
    gf = lambda F=4, H=p, ldh=4, ldw=4: fn("emu_gated_fwd", 0, 4, 1040, F, 4, p, 4, p, ldw, p, p, 8, H, ldh)
    assert fn("emu_gated_fwd", 4, 4, 40, 4, 4, p, 4, p, 4, p, None, 0, p, 4) == INVALID    # fp32 works by way of D
    assert gf(H=None) == INVALID and gf(ldh=3) == INVALID and gf(ldw=3) == INVALID and gf(F=2 ** 30) == NOT_SUPPORTED
    assert gf(F=0) == 0


def test_few_row_rule(ff):
    """At most 1,024 rows with (M - 8) N K <= 50 million."""
    q = emu.load().emu_few_rows_query
    q.argtypes = [ctypes.c_int64] * 3
    for M, N, K in ((1, 1, 1), (1024, 1, 1), (1025, 1, 1), (0, 4, 4), (1024, 128, 384), (1024, 128, 385), (9, 50_000_000, 1),
                    (9, 50_000_001, 1), (8, 2 ** 30, 2 ** 20), (64, 1024, 871), (64, 1024, 872),
                    (1024, 2 ** 31 - 257, 2 ** 31 - 257)):
        assert q(M, N, K) == int(M <= 1024 and (M - 8) * N * K <= 50_000_000), (M, N, K)


def test_exports_and_lazy_names():
    for name in emu._FEED_FORWARD:
        assert name in emu.__all__ and getattr(emu, name) is not None
