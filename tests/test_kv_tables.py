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


def search(lm, c, seed, steps, clips, beams):
    """Steps of append, attend, advance and reorder; the attentions' outputs."""
    r, outs = kv.gen(seed), []
    g = torch.Generator(device="cuda").manual_seed(seed)
    for _ in range(steps):
        q, k, v = (r(c.rows, 1, c.heads, c.head_dim).to(c.dtype) for _ in range(3))
        c.append(0, k, v)
        outs.append(c.attend(0, q))
        c.advance(1)
        c.reorder(torch.randint(0, beams, (clips, beams), generator=g, device="cuda", dtype=torch.int32))
    return torch.stack(outs)


@pytest.mark.parametrize("block,steps", [(16, 40), (32, 33), (16, 7)])
def test_a_cache_is_used_again(lm, block, steps):
    clips, beams = 2, 3
    c = lm.KvCache(clips * beams, 48, 2, 64, block=block, dtype=torch.float16)
    first = search(lm, c, 1, steps, clips, beams)
    if steps > block:
        assert c.table[:, 0].unique().numel() < c.rows  # rows share blocks that the next search writes
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.reset(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    names = torch.cat([c.table.flatten(), c.spare])
    assert torch.equal(names.sort().values, torch.arange(c.blocks, device="cuda", dtype=torch.int32))
    assert not c.lens.any()
    again = search(lm, c, 2, steps, clips, beams)
    fresh = lm.KvCache(clips * beams, 48, 2, 64, block=block, dtype=torch.float16)
    assert torch.equal(again, search(lm, fresh, 2, steps, clips, beams))
    c.reset()
    assert torch.equal(first, search(lm, c, 1, steps, clips, beams))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.reset()
    g.replay()
    assert torch.equal(again, search(lm, c, 2, steps, clips, beams))


def test_reset_of_empty_caches(lm):
    for rows, tokens in ((0, 64), (3, 0)):
        c = lm.KvCache(rows, tokens, 2, 64)
        c.reset()
        assert c.table.shape == (rows, -(-tokens // 32)) and c.spare.tolist() == list(range(rows * c.width, c.blocks))


@pytest.mark.parametrize("absent", [-1, 2 ** 31 - 1])
@pytest.mark.parametrize("beams", [2, 5])
def test_an_absent_open_block_stays_absent(lm, absent, beams):
    """Rows that continue a row without its open block have the tokens that it has, and keep their spare block."""
    c = kv.filled(lm, beams, 64, 1, 64, 32, torch.float16, seed=3)
    c.lens.fill_(40)
    c.table[0, 1] = absent
    spare = c.spare.clone()
    q = kv.gen(3)(1, 1, 1, 64).half().expand(beams, -1, -1, -1)
    want = c.attend(0, q, causal=False)[0].clone()
    c.reorder(torch.zeros((1, beams), dtype=torch.int32, device="cuda"))
    assert torch.equal(c.attend(0, q, causal=False), want.expand(beams, -1, -1, -1))
    assert (c.table[:, 1] == absent).all() and torch.equal(c.spare, spare)
    assert not c.read(0, 32, 8)[0].any()


def test_a_row_without_its_open_block_takes_another(lm):
    c = kv.filled(lm, 2, 64, 2, 64, 32, torch.float16, seed=4)
    c.lens.fill_(40)
    c.table[1, 1] = -1
    mine = int(c.spare[1])
    c.reorder(torch.zeros((1, 2), dtype=torch.int32, device="cuda"))
    k, v = c.read(0, 0, 40)
    assert torch.equal(k[0], k[1]) and torch.equal(v[0], v[1]) and k.any()
    assert int(c.table[1, 1]) == mine and int(c.spare[1]) == -1


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
