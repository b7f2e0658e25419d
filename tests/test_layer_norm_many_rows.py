"""Sums over rows where a warp's teams have unequal numbers of them.

Rows of one value, a power of two, have a mean without rounding, no deviations and n = 0 in every place: dweight is 0
and dbias the gradients' sum, however large the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [7, 12769, 12771, 26001])
def test_large_rows_of_one_value(lm, dtype, width, rows):
    x = torch.full((rows, width), 2.0 ** 120, device="cuda", dtype=dtype).requires_grad_()
    w, b = (torch.ones(width, device="cuda", requires_grad=True) for _ in range(2))
    g = torch.ones((rows, width), device="cuda", dtype=dtype)
    y = lm.layer_norm(x, w, b)
    assert torch.equal(y, torch.ones_like(y))
    dx, dw, db = torch.autograd.grad(y, (x, w, b), g)
    assert not dw.any() and (db == rows).all() and not dx.any()
