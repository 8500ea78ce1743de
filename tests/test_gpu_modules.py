"""The feed-forward modules as inference runs them."""
import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu


def peak(call):
    import torch
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    call()
    torch.cuda.synchronize()
    return torch.cuda.max_memory_allocated() - before


def test_inference_through_a_module_holds_what_the_call_holds():
    """Under no_grad the block's module takes no more memory than the functional
    call without `save`: no M x 2F factors for a backward pass."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(0)
    M, K, F = 20000, 64, 512
    m = emu.EmuGatedFFN(K, F).to(_gpu.device())
    x = torch.randn(M, K, device=_gpu.device())
    p = (m.weight_in.detach(), m.bias_in.detach(), m.weight_out.detach(), m.bias_out.detach())
    call = lambda: emu.gated_ffn_fwd(x, *p)
    with torch.no_grad():
        assert torch.equal(m(x), call())
        assert peak(lambda: m(x)) == peak(call) < 4 * M * (F + K) + (1 << 20)
    y = m(x)
    assert y.requires_grad and torch.equal(y.detach(), call())
    assert emu.emu_stream_check() == 0


def test_inference_and_training_of_every_module_agree():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(1)
    for m in (emu.EmuLayerNorm(48), emu.EmuLinearAct(48, 100), emu.EmuGatedFFN(48, 100, mode="tf32x3"),
              emu.EmuFeedForward(48, 100), emu.EmuFeedForward(48, 100, mode="fp32")):
        m = m.to(_gpu.device())
        for rows in (1, 7, 1300):
            x = torch.randn(rows, 48, device=_gpu.device())
            y = m(x)
            assert y.requires_grad
            for off in (torch.no_grad, torch.inference_mode):
                with off():
                    z = m(x)
                assert not z.requires_grad and torch.equal(z, y.detach())
    assert emu.emu_stream_check() == 0


def test_layer_norm_without_statistics():
    import torch
    import fp32_emulated_gemm_gb300 as emu
    for M, N in ((192, 256), (5, 31), (3, 20000), (0, 8)):
        x, w, b = (torch.randn(*s, device=_gpu.device()) for s in ((M, N), (N,), (N,)))
        y = emu.layer_norm_fwd(x, w, b, save=False)
        assert torch.equal(y, emu.layer_norm_fwd(x, w, b)[0])
        out = torch.empty(M, N, device=_gpu.device())
        assert emu.layer_norm_fwd(x, w, b, save=False, out=out) is out and torch.equal(out, y)
    assert emu.emu_stream_check() == 0


def test_output_projection_gradients_alone():
    """dW_out and db_out without the others: the same values, no M x 2F buffer,
    and D is not asked for; db_out alone does not ask for H either."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    torch.manual_seed(2)
    M, K, F, N = 20000, 32, 512, 64
    x, wi, wo, dy = (torch.randn(*s, device=_gpu.device()) for s in ((M, K), (2 * F, K), (N, F), (M, N)))
    _, d, h = emu.gated_ffn_fwd(x, wi, None, wo, None, save=True)
    full = emu.gated_ffn_bwd(dy, x, wi, wo, d, h)
    only = lambda: emu.gated_ffn_bwd(dy, x, wi, wo, None, h, need=(False, False, False, True, True))
    some = only()
    assert some[:3] == (None, None, None) and peak(only) <= 4 * (N * F + N) + (1 << 20)
    bound = 2 * (2 * M + 8) * 2.0 ** -24 * (dy.abs().T @ h.abs())        # two plans of the same product
    assert bool(((some[3] - full[3]).abs() <= bound).all()) and torch.equal(some[4], full[4])
    bias = emu.gated_ffn_bwd(dy, x, wi, wo, None, None, need=(False, False, False, False, True))
    assert torch.equal(bias[4], full[4])
    assert emu.emu_stream_check() == 0
