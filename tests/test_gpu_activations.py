"""The activations alone against 64 bits: through a product with the unit matrix,
which leaves its operand as it is, in the tiles' epilogue, the few-row form and
the row-wise kernel.

Bounds as the header states them: 8 u |z| for the value and 8 u (1 + |z|) for the
derivative, u = 2^-24.  (Phi by its approximation 1.3 u, the exponential and the
reciprocal 2 units in the last place each of at most a half, the roundings
between them one u each.)"""
import numpy as np
import pytest

from tests import _gpu
from tests import _running as R

pytestmark = pytest.mark.gpu
U = R.U


@pytest.mark.parametrize("rows,mode", [(1 << 18, "bf16x9"), (1 << 18, "tf32x3"), (1000, "bf16x9"), (1 << 18, "fp32")])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_values_and_derivatives(act, rows, mode):
    import torch
    import fp32_emulated_gemm_gb300 as emu
    rng = np.random.default_rng(5)
    # (the last 12 bits of the mantissa cleared: every mode multiplies these by one exactly)
    z = np.concatenate([rng.uniform(-a, a, (rows // 4, 4)) for a in (0.1, 2, 8, 40)]).astype(np.float32)
    z = (z.view(np.uint32) & np.uint32(0xFFFFF000)).view(np.float32)
    one = torch.eye(4, device=_gpu.device())
    y, d = emu.linear_act_fwd(_gpu.to_dev(z), one, act=act, mode=mode, save=True)
    assert emu.emu_stream_check() == 0
    a64, d64 = R.act64(act, z.astype(np.float64))
    a, g = y.cpu().numpy().astype(np.float64), None if d is None else d.cpu().numpy().astype(np.float64)
    if act in ("none", "relu"):
        assert np.array_equal(a, a64) and (g is None or np.array_equal(g, d64))
        return
    assert np.all(np.abs(a - a64) <= 8 * U * np.abs(z))
    assert np.all(np.abs(g - d64) <= 8 * U * (1 + np.abs(z)))
