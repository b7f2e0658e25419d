"""A block's scale, for every finite value that can be its largest: max |x| * c with c the float32 nearest to 1 / 127, as
include/logmel.h defines it.  c rounds 1 / 127 down to 24 bits and the product rounds once more, so that it is within one
unit in the last place of the division and the largest value becomes 127."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.mark.parametrize("dtype,codes", [(torch.float16, 0x7c00), (torch.bfloat16, 0x7f80)])
def test_every_largest_value(lm, dtype, codes):
    top = torch.arange(codes, dtype=torch.int16, device="cuda").view(dtype)
    rows = codes
    c = lm.KvCache(rows, 16, 1, 32, block=16, dtype=dtype)
    k = torch.zeros((rows, 1, 1, 32), dtype=dtype, device="cuda")
    k[:, 0, 0, 7] = top
    k[:, 0, 0, 20] = -top
    values, _ = c.append(0, k, k, values=True)
    want = top.float() * (torch.ones((), device="cuda") / 127)
    want = torch.where(want > 0, want, 1.0)
    scale = c.k_scale[0, c.table[:, 0].long(), 0]
    assert torch.equal(scale, want) and torch.equal(c.v_scale[0, c.table[:, 0].long(), 0], want)
    ulp = (scale.view(torch.int32) - (top.float() / 127).view(torch.int32)).abs()
    assert int(ulp[1:].max()) <= 1
    held = c.k8[0, c.table[:, 0].long(), 0, 0]
    full = (top > 0).int() * 127
    assert torch.equal(held[:, 7].int(), full) and torch.equal(held[:, 20].int(), -full)
    assert torch.equal(values[:, 0, 0, 7], (full * scale).to(dtype)) and not values[:, 1:].any()
