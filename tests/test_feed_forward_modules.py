"""The feed-forward modules' host side, without a GPU: the functional calls are
replaced by plain ones that record how they were called."""
import pytest
import torch
import torch.nn.functional as F

import fp32_emulated_gemm_gb300 as emu


@pytest.fixture
def calls(monkeypatch):
    from fp32_emulated_gemm_gb300 import feed_forward as ff
    made = []

    def layer_norm_fwd(X, weight=None, bias=None, *, eps=1e-5, save=True, out=None):
        made.append(("layer_norm", None))
        y = F.layer_norm(X, X.shape[1:], weight, bias, eps)
        return (y, X.new_zeros(len(X)), X.new_zeros(len(X))) if save else y

    def linear_act_fwd(X, W, bias=None, *, act="none", residual=None, mode="bf16x9", save=False, out=None):
        made.append(("linear_act", save))
        y = F.gelu(F.linear(X, W, bias))
        y = y if residual is None else y + residual
        return (y, X.new_zeros(len(X), len(W))) if save else y

    def gated_ffn_fwd(X, W_in, b_in, W_out, b_out, *, act="silu", residual=None, mode="bf16x9", save=False, out=None):
        made.append(("gated_ffn", save))
        g, u = F.linear(X, W_in, b_in).chunk(2, -1)
        y = F.linear(F.silu(g) * u, W_out, b_out)
        y = y if residual is None else y + residual
        return (y, X.new_zeros(len(X), len(W_in)), g * u) if save else y

    for f in (layer_norm_fwd, linear_act_fwd, gated_ffn_fwd):
        monkeypatch.setattr(ff, f.__name__, f)
    return made


MODULES = {
    "linear_act": lambda: emu.EmuLinearAct(6, 10),
    "gated_ffn": lambda: emu.EmuGatedFFN(6, 8),
    "feed_forward": lambda: emu.EmuFeedForward(6, 8),
}


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("name", MODULES)
def test_nothing_is_saved_with_gradients_off(calls, name, off):
    """Parameters that require gradients do not make an inference call store
    what only a backward pass reads."""
    torch.manual_seed(0)
    m, x = MODULES[name](), torch.randn(5, 6)
    trained = m(x)
    assert trained.requires_grad and [s for _, s in calls if s is not None] == [True]
    calls.clear()
    with off():
        y = m(x)
    assert not y.requires_grad and torch.equal(y, trained.detach())
    assert [s for _, s in calls if s is not None] == [False]


@pytest.mark.parametrize("name", MODULES)
def test_nothing_is_saved_when_no_input_needs_a_gradient(calls, name):
    m = MODULES[name]().requires_grad_(False)
    assert not m(torch.randn(5, 6)).requires_grad
    assert [s for _, s in calls if s is not None] == [False]


def test_layer_norm_with_gradients_off(calls):
    m, x = emu.EmuLayerNorm(6), torch.randn(5, 6)
    with torch.no_grad():
        y = m(x)
    assert not y.requires_grad and torch.allclose(y, F.layer_norm(x, (6,)), atol=1e-6)


def test_the_norms_statistics_are_kept_for_gradients_alone(monkeypatch):
    from fp32_emulated_gemm_gb300 import feed_forward as ff
    saves = []

    def layer_norm_fwd(X, weight=None, bias=None, *, eps=1e-5, save=True, out=None):
        saves.append(save)
        y = F.layer_norm(X, X.shape[1:], weight, bias, eps)
        return (y, X.new_zeros(len(X)), X.new_zeros(len(X))) if save else y

    def gated_ffn_fwd(X, *args, residual=None, save=False, **kw):
        return (X + residual, X, X) if save else X + residual

    monkeypatch.setattr(ff, "layer_norm_fwd", layer_norm_fwd)
    monkeypatch.setattr(ff, "gated_ffn_fwd", gated_ffn_fwd)
    x = torch.randn(5, 6)
    for m in (emu.EmuLayerNorm(6), emu.EmuFeedForward(6, 8)):
        m(x)
        with torch.no_grad():
            m(x)
        m.requires_grad_(False)(x)
    assert saves == [True, False, False] * 2


@pytest.mark.parametrize("name", MODULES)
def test_inputs_of_another_width_are_refused(calls, name):
    """An input whose elements make a whole number of rows of the right width
    is no input of that width."""
    m = MODULES[name]()
    for shape in ((5, 12), (2, 3, 3), (12,), (4, 18), ()):
        with pytest.raises(ValueError):
            m(torch.randn(shape))
    assert calls == []
    out = 10 if name == "linear_act" else 6
    for shape in ((6,), (0, 6), (2, 3, 6), (2, 0, 6)):
        assert m(torch.randn(shape)).shape == (*shape[:-1], out)


@pytest.mark.parametrize("name", ["linear_act", "gated_ffn"])
def test_residuals_of_another_shape_are_refused(calls, name):
    """The residual's rows are the result's: another shape of as many elements
    is refused, as a sum of the two would be; the flat matrix is taken."""
    m, out = MODULES[name](), 10 if name == "linear_act" else 6
    x = torch.randn(2, 3, 6)
    for shape in ((3, 2, out), (6 * out,), (2, 3 * out), (1, 3, out), (2, out, 3)):
        with pytest.raises(ValueError):
            m(x, torch.randn(shape))
    assert calls == []
    r = torch.randn(2, 3, out)
    y = m(x, r)
    assert torch.allclose(y - r, m(x), atol=1e-6) and torch.equal(y, m(x, r.reshape(6, out)))
