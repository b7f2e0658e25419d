"""A 4-bit weight's scales have no gradients: a graph over them is refused, not left out."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def test_scales_that_want_gradients(lm):
    w4 = lm.quantize_weight(torch.randn((32, 128), device="cuda").half())
    x = torch.randn((4, 128), device="cuda").half()
    want, values = lm.linear(x, w4), w4.values()
    w4.scale.requires_grad_()
    for call in (lambda: lm.linear(x, w4), w4.values):
        with pytest.raises(RuntimeError, match="inference-only"):
            call()
    with torch.no_grad():
        assert torch.equal(lm.linear(x, w4), want) and torch.equal(w4.values(), values)


def test_scales_with_a_tangent(lm):
    w4 = lm.quantize_weight(torch.randn((32, 128), device="cuda").half())
    x = torch.randn((4, 128), device="cuda").half()
    with fwd.dual_level():
        w4.scale = fwd.make_dual(w4.scale, w4.scale)
        for call in (lambda: lm.linear(x, w4), w4.values):
            with pytest.raises(RuntimeError, match="inference-only"):
                call()
