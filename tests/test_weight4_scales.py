"""Scales of 4-bit weights above the largest value of x's type.

A value is q times its scale, rounded to x's type: 0 where q is 0, infinite past the type's largest value.  That holds
for every number of rows (the forms below 17 rows, and of up to 64 onto few outputs, keep the scale in 32 bits).
"""
import pytest
import torch

from test_weight4 import check, numbers, value64

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]
LARGE = {torch.float16: (65519.0, 65520.0, 70000.0, -140000.0, 1e30, torch.finfo(torch.float32).max),
         torch.bfloat16: (3.3895e38, -3.39e38, 3.3962e38, torch.finfo(torch.float32).max)}
ROWS = [5, 16, 40, 100, 300, 768, 1000]


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_stay_zeros(lm, dtype, group, rows):
    """Groups of zeros with such a scale add nothing; the others give what they give alone."""
    n, k = 150, 300
    q, s = numbers(n, k, group, seed=rows)
    for i, large in enumerate(LARGE[dtype]):
        q[5 * i, group:2 * group] = 0
        s[5 * i, 1] = large
    x = torch.randn((rows, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    w4 = lm.Weight4.pack(q, s, group=group, dtype=dtype)
    assert w4.values().isfinite().all()
    check(lm.linear(x, w4, out_dtype=torch.float32), x, value64(q, s, group))


@pytest.mark.parametrize("rows", ROWS[3:])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_are_rounded_to_the_types_of_x(lm, dtype, rows):
    """One value that is not zero in an output: x times what values() says, also where that is infinite."""
    n, k = 2 * len(LARGE[dtype]) + 120, 300
    q, s = numbers(n, k, 32)
    q.zero_()
    for i, large in enumerate(LARGE[dtype]):
        s[2 * i:2 * i + 2, 1] = large
        q[2 * i, 40], q[2 * i + 1, 40] = 1, -1
    w4 = lm.Weight4.pack(q, s, group=32, dtype=dtype)
    x = torch.full((rows, k), 0.5, device="cuda", dtype=dtype)
    want = (0.5 * w4.values()[:, 40].float()).expand(rows, -1)
    assert want.isinf().any() and (dtype == torch.bfloat16 or want[0, 0] == 32752)
    assert torch.equal(lm.linear(x, w4, out_dtype=torch.float32), want)


@pytest.mark.parametrize("rows", ROWS[2:])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("odd", [0.0, 1e-6, 1e30, float("inf"), float("nan")])
def test_other_outputs_keep_their_bits(lm, dtype, rows, odd):
    """What a scale is like, and how its values are formed, is not felt beside it."""
    q, s = numbers(150, 300, 32, seed=3)
    x = torch.randn((rows, 300), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    want = lm.linear(x, lm.Weight4.pack(q, s, group=32, dtype=dtype))
    s[7, 2], s[100, 5] = odd, odd
    got = lm.linear(x, lm.Weight4.pack(q, s, group=32, dtype=dtype))
    keep = [i for i in range(150) if i not in (7, 100)]
    assert torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dtype", TYPES)
def test_scales_that_are_not_finite(lm, dtype, rows):
    """As values() says: q times infinity is infinite, or NaN where q is 0, and so is what x adds up to."""
    q, s = numbers(150, 300, 32, seed=5)
    q[7], q[9] = 1, -1  # no zeros: the sums are infinite
    q[11, 70] = 0
    s[7, 2], s[9, 5], s[11, 2], s[13, 1] = float("inf"), float("inf"), float("inf"), float("nan")
    w4 = lm.Weight4.pack(q, s, group=32, dtype=dtype)
    v = w4.values()
    assert (v[7, 64:96] == float("inf")).all() and (v[9, 160:192] == -float("inf")).all()
    assert v[11, 70].isnan() and v[13, 32:64].isnan().all()
    x = torch.rand((rows, 300), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype) + 0.25
    y = lm.linear(x, w4)
    assert (y[:, 7] == float("inf")).all() and (y[:, 9] == -float("inf")).all()
    assert not y[:, 11].isfinite().any() and y[:, 13].isnan().all()
    keep = [i for i in range(150) if i not in (7, 9, 11, 13)]
    assert y[:, keep].isfinite().all()
