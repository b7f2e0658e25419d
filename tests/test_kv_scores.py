"""Scores of the cache's attention where one element of the head sets a block's scale.

The tolerance is that of test_kv_cache.py: a score is a 32-bit sum of exact products, off by at most
(head_dim + 8) * 2^-23 * scale * sum |q k|.  Here the large keys meet queries of zero (or small ones), so that sum |q k|
is far below what the block's scale allows, and nothing of the size of the outlier may enter the sums.
"""
import pytest
import torch

import test_kv_cache as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,rows,heads,tokens,t", [(64, 2, 2, 300, 1), (128, 2, 2, 300, 5), (64, 48, 10, 160, 64),
                                                     (128, 30, 12, 150, 130), (128, 130, 7, 100, 1), (32, 2, 2, 300, 20),
                                                     (64, 1, 2, 9000, 1)])
@pytest.mark.parametrize("small,at", [(0, 0.0), (1, 0.0), (3, 2.0 ** -9)])
def test_an_outlier_sets_the_scale(lm, dtype, dim, rows, heads, tokens, t, small, at):
    """Keys within +-small but for element 5, which is 127; queries all of one sign but for that element."""
    c = kv.filled(lm, rows, tokens, heads, dim, 32, dtype, seed=dim)
    c.k8.clamp_(-small, small)
    c.k8[..., 5] = 127
    c.k_scale.fill_(64.0)
    c.lens.fill_(tokens - t)
    q = kv.gen(3)(rows, t, heads, dim).abs() + 0.5
    q[..., 5] = at
    q = q.to(dtype)
    kv.check_attend(c.attend(0, q), c, 0, q, [t] * rows, True)


def test_every_byte(lm):
    """Keys and values of every 8-bit value, -128 included, each in every place of a 4-byte word."""
    c = lm.KvCache(1, 256, 1, 32, block=16, dtype=torch.float16)
    b = (torch.arange(256, device="cuda")[:, None] + 67 * torch.arange(32, device="cuda")) % 256 - 128
    c.k8.view(-1, 32)[:256] = b.to(torch.int8)
    c.v8.view(-1, 32)[:256] = b.flip(0).to(torch.int8)
    c.k_scale.fill_(2.0 ** -9)
    c.v_scale.fill_(2.0 ** -6)
    c.lens.fill_(256)
    for e in range(32):
        q = torch.zeros((1, 1, 1, 32), device="cuda", dtype=torch.float16)
        q[..., e] = 5.0
        kv.check_attend(c.attend(0, q, causal=False), c, 0, q, [0], False)
