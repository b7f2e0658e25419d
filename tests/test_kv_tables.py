"""Block tables of the key/value cache that are not one block of its own per column."""
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


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("rows,heads,dim,tokens,t", [(3, 2, 64, 90, 1), (2, 1, 128, 75, 3), (1, 2, 32, 9000, 1),
                                                     (160, 5, 64, 70, 1), (48, 10, 64, 160, 64)])
def test_a_row_names_a_block_twice(lm, block, rows, heads, dim, tokens, t):
    """Place t of a row is table[t / block][t % block], whatever else names the block.  The last block of
    the cache is one of them: nothing may be read past it."""
    c = kv.filled(lm, rows, tokens, heads, dim, block, torch.float16, seed=rows + block)
    width = c.table.shape[1]
    c.table.copy_(c.table[:, :(width + 1) // 2].repeat_interleave(2, 1)[:, :width])
    c.table[0].fill_(c.blocks - 1)
    c.table[-1, 1:].copy_(c.table[-1, :-1].clone())  # pairs that start at an odd column
    c.lens.copy_(tokens - t - torch.arange(rows) * 3 % (tokens // 2))
    q = kv.gen(t)(rows, t, heads, dim).half()
    kv.check_attend(c.attend(0, q), c, 0, q, [t] * rows, True)
    kv.check_attend(c.attend(0, q, causal=False), c, 0, q, [0] * rows, False)
