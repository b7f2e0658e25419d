"""The 8-bit key/value cache against its definition.

append: scales, 8-bit values and read-back are compared exactly with the same
IEEE operations in torch (amax, * 1/127, /, round half to even).

attend: against softmax attention in 64 bits over the cache's own contents.
Tolerance, from the arithmetic: a score is a 32-bit sum of exact products, off
by d <= (head_dim + 8) * 2^-23 * scale * sum |q k|, and 2^-22 of itself for the
change of base; weights are rounded to 16 bits once at most (2^-11, or 2^-24 of
the largest where that is more), and exponentials are good to 2^-20; so a
result is off by (2^-11 + 2 d + 2^-18) of the weighted mean of |v| and 2^-24 of
the largest |v|, plus one rounding to the output's type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -7.99, torch.float16: 2.0 ** -10.99}


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def filled(lm, rows, tokens, heads, dim, block, dtype, seed=0, layers=1, shuffle=True):
    """A cache whose blocks hold random values with scales of their own, in random order."""
    c = lm.KvCache(rows, tokens, heads, dim, layers=layers, block=block, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k8, c.v8):
        t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda", dtype=torch.int8))
    for t in (c.k_scale, c.v_scale):
        t.copy_((torch.rand(t.shape, generator=g, device="cuda") * 2 + 0.1) / 127)
    if shuffle:
        order = torch.randperm(c.blocks, generator=g, device="cuda").int()
        c.table.copy_(order[:c.table.numel()].view_as(c.table))
        c.spare.copy_(order[c.table.numel():])
    return c


def row64(c, which, layer, r, n):
    x8, sc = (c.k8, c.k_scale) if which == "k" else (c.v8, c.v_scale)
    pages = c.table[r].long()[:-(-n // c.block)]
    x = x8[layer, pages].double() * sc[layer, pages].double()[..., None, None]
    return x.transpose(1, 2).flatten(0, 1)[:n]


def check_attend(out, c, layer, q, new, causal, scale=None):
    rows, t, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    group = hq // c.heads
    cap = c.table.shape[1] * c.block
    for r in range(rows):
        held = max(0, int(c.lens[r]))
        n = min(max(int(new[r]), 0), t) if causal else int(new[r])
        total = min(held + n, cap)
        ref = torch.zeros((t, hq, d), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(ref)
        if total:
            k, v = row64(c, "k", layer, r, total), row64(c, "v", layer, r, total)
            k, v = (x.repeat_interleave(group, 1) for x in (k, v))
            qd = q[r].double()
            s = torch.einsum("ihd,lhd->ihl", qd, k) * scale
            mag = torch.einsum("ihd,lhd->ihl", qd.abs(), k.abs()) * abs(scale)
            err = (d + 8) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -22 * s.abs().amax(-1)
            if causal:
                i = torch.arange(t, device="cuda")
                seen = (torch.arange(total, device="cuda")[None] <= held + i[:, None]) & (i < n)[:, None]
                s = torch.where(seen[:, None], s, -math.inf)
            p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
            z = p.sum(-1, keepdim=True)
            p = torch.where(z > 0, p / z, 0.0)
            ref = torch.einsum("ihl,lhd->ihd", p, v)
            mean = torch.einsum("ihl,lhd->ihd", p, v.abs())
            tol = (2.0 ** -11 + 2 * err[..., None] + 2.0 ** -18) * mean + 2.0 ** -24 * v.abs().amax()
            dead = z[..., 0] == 0
            assert not out[r][dead].any()
        tol = tol + UNIT[out.dtype] * (ref.abs() + 2.0 ** -14)
        off = (out[r].double() - ref).abs()
        assert (off <= tol).all(), (r, held, n, float((off - tol).max()), float(off.max()))


# ---- append ---------------------------------------------------------------

def append_ref(c, layer, k, v, new):
    """The definition, token by token block by block, on copies of the cache's tensors."""
    out = {}
    for name, x, x8, sc in (("k", k, c.k8, c.k_scale), ("v", v, c.v8, c.v_scale)):
        x8, sc = x8.clone(), sc.clone()
        rows, t, h, d = x.shape
        bs = c.block
        for r in range(rows):
            held = min(max(0, int(c.lens[r])), c.max_tokens)
            n = min(max(int(new[r]), 0), t)
            end = min(held + n, c.max_tokens)
            at = held
            while at < end:
                j = at // bs
                stop = min(end, (j + 1) * bs)
                blk = int(c.table[r, j])
                y = x[r, at - held:stop - held].float().transpose(0, 1)  # [h, n, d]
                top = torch.where(y.isfinite(), y.abs(), math.inf).amax((1, 2))
                before = sc[layer, blk] if at % bs else torch.zeros(h, device="cuda")
                now = torch.maximum(before, top * (torch.ones((), device="cuda") / 127))
                now = torch.where(now > 0, now, 1.0)
                old = x8[layer, blk, :, :at % bs].float()
                re = torch.round(old * (before / now)[:, None, None])
                x8[layer, blk, :, :at % bs] = re.nan_to_num(0, 0, 0).to(torch.int8)
                q = torch.round(y / now[:, None, None]).nan_to_num(0, 0, 0)
                x8[layer, blk, :, at % bs:stop - j * bs] = q.to(torch.int8)
                sc[layer, blk] = now
                at = stop
        out[name] = (x8, sc)
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,block", [(32, 16), (64, 16), (64, 32), (128, 32), (32, 128), (64, 128), (128, 128), (128, 64)])
@pytest.mark.parametrize("t", [1, 7, 150])
def test_append_is_its_definition(lm, dtype, dim, block, t):
    rows, heads, layers = 6, 3, 2
    c = filled(lm, rows, 300, heads, dim, block, dtype, seed=t + dim, layers=layers)
    c.lens.copy_(torch.tensor([0, 5, block, 2 * block - 1, 130, c.max_tokens - 3]))
    r = gen(t)
    mag = torch.tensor([1.0, 3.0, 0.01, 30.0, 1e-3, 1.0], device="cuda")[:, None, None, None]
    k, v = ((r(rows, t, heads, dim) * mag).to(dtype) for _ in range(2))
    new = torch.tensor([t, t, max(1, t - 1), t, t // 2, t], dtype=torch.int32, device="cuda")
    k[4, t // 2:] = math.nan  # past the row's count
    was = [x.clone() for x in (c.table, c.lens)]
    ref = append_ref(c, 1, k, v, new)
    kv, vv = c.append(1, k, v, new, values=True)
    for name, x8, sc, val in (("k", c.k8, c.k_scale, kv), ("v", c.v8, c.v_scale, vv)):
        assert torch.equal(x8, ref[name][0])
        assert torch.equal(sc, ref[name][1])
        for i in range(rows):
            held = int(c.lens[i])
            base = held // block * block
            end = min(held + int(new[i]), c.max_tokens)
            want = torch.zeros_like(val[i])
            if end > base and new[i] > 0:
                want[:end - base] = (row32(c, name, 1, i, end)[base:end]).to(dtype)
            elif end > base:
                want[:end - base] = val[i, :end - base]  # nothing new: the open block as it was
                assert torch.equal(want[:end - base], row32(c, name, 1, i, end)[base:end].to(dtype))
            assert torch.equal(val[i], want), (name, i)
    assert torch.equal(was[0], c.table) and torch.equal(was[1], c.lens)


def row32(c, which, layer, r, n):
    x8, sc = (c.k8, c.k_scale) if which == "k" else (c.v8, c.v_scale)
    pages = c.table[r].long()[:-(-n // c.block)]
    x = x8[layer, pages].float() * sc[layer, pages][..., None, None]
    return x.transpose(1, 2).flatten(0, 1)[:n]


def test_append_of_views_and_odd_strides(lm):
    rows, t, heads, dim = 3, 40, 4, 64
    a, b = (lm.KvCache(rows, 100, heads, dim, dtype=torch.float16) for _ in range(2))
    r = gen(2)
    for shift in (0, 1):  # a fused projection's halves, and one that 16-byte loads do not fit
        qkv = r(rows, t, 3 * heads * dim + 9).half()
        k, v = (qkv[..., i * heads * dim + shift:(i + 1) * heads * dim + shift].unflatten(-1, (heads, dim)) for i in (1, 2))
        a.append(0, k, v)
        b.append(0, k.contiguous(), v.contiguous())
        a.advance(t)
        b.advance(t)
        for x, y in zip(a.read(0, 0, 100), b.read(0, 0, 100)):
            assert torch.equal(x, y)


def test_append_poisons_a_block_with_nan_or_infinity(lm):
    c = lm.KvCache(2, 64, 2, 32, block=16, dtype=torch.float16)
    k = gen(1)(2, 40, 2, 32).half()
    v = k.clone()
    k[0, 20, 1, 3] = math.nan
    v[1, 2, 0, 0] = -math.inf
    kv, vv = c.append(0, k, v, values=True)
    assert kv[0, 16:32, 1].isnan().all() and kv[0, :16].isfinite().all() and kv[0, 32:40].isfinite().all()
    assert kv[0, 16:32, 0].isfinite().all() and vv[1, :16, 0].isnan().all() and vv[1, 16:].isfinite().all()
    c.advance(40)
    out = c.attend(0, gen(3)(2, 1, 2, 32).half(), causal=False)
    assert out[0, 0, 1].isnan().all() and out[0, 0, 0].isfinite().all()
    assert out[1, 0, 0].isnan().all() and out[1, 0, 1].isfinite().all()


def test_zero_tokens_and_zero_rows(lm):
    c = lm.KvCache(2, 64, 2, 32, dtype=torch.float16)
    z = torch.zeros((2, 5, 2, 32), device="cuda", dtype=torch.float16)
    k, v = c.append(0, z, z, values=True)
    assert not k.any() and (c.k_scale[0, c.table[:, 0].long()] == 1).all()
    c.append(0, z[:, :0], z[:, :0])
    none = lm.KvCache(0, 64, 2, 32, dtype=torch.float16)
    none.append(0, z[:0], z[:0])
    assert none.attend(0, z[:0]).shape == (0, 5, 2, 32)
    assert c.attend(0, z[:, :0]).shape == (2, 0, 2, 32)


# ---- attend ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,block", [(32, 16), (64, 16), (64, 32), (64, 128), (128, 16), (128, 64), (128, 32), (32, 128)])
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("causal", [True, False])
def test_single_tokens_over_ragged_rows(lm, dtype, dim, block, group, causal):
    lens = [0, 1, 2, block - 1, block, block + 1, 100, 31, 32, 33, 64, 65, 299, 511, 640, 7]
    c = filled(lm, len(lens), 641, 3, dim, block, dtype, seed=dim + group)
    c.lens.copy_(torch.tensor(lens))
    q = (gen(group)(len(lens), 1, 3 * group, dim) * 2).to(dtype)
    out = c.attend(0, q, causal=causal)
    check_attend(out, c, 0, q, [1] * len(lens) if causal else [0] * len(lens), causal)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,group", [(2, 1), (5, 1), (3, 5), (16, 1), (17, 2), (33, 1), (70, 8), (223, 1)])
@pytest.mark.parametrize("dim", [32, 64, 128])
def test_many_queries(lm, dtype, t, group, dim):
    c = filled(lm, 4, 400, 2, dim, 32, dtype, seed=t)
    c.lens.copy_(torch.tensor([0, 130, 17, 400 - t]))
    q = (gen(t)(4, t, 2 * group, dim) * 2).to(dtype)
    new = torch.tensor([t, t, t // 2, t], dtype=torch.int32, device="cuda")
    check_attend(c.attend(0, q, new), c, 0, q, new.tolist(), True)
    extra = torch.tensor([0, 9, 0, 0], dtype=torch.int32, device="cuda")
    check_attend(c.attend(0, q, extra, causal=False), c, 0, q, extra.tolist(), False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_long_rows(lm, dtype):
    c = filled(lm, 2, 40000, 2, 64, 64, dtype, seed=4)
    c.lens.copy_(torch.tensor([39990, 20011]))
    q = (gen(8)(2, 2, 8, 64) * 3).to(dtype)
    check_attend(c.attend(0, q), c, 0, q, [2, 2], True)


def test_an_offset_past_32_bits(lm):
    # A layer that starts past 2^32 elements, and a block past 2^31 within it.
    c = lm.KvCache(2, 17 * 1024, 1, 128, layers=1, block=128, dtype=torch.float16)
    blocks = (5 << 30) // (128 * 128 * 8)
    big = lm.KvCache(8, blocks * 16, 8, 128, layers=2, block=128, dtype=torch.float16)
    assert big.k8[0].numel() > 2 ** 31
    r = gen(1)
    k, v = (r(8, 300, 8, 128).half() for _ in range(2))
    big.table.copy_(big.blocks - 1 - torch.arange(big.table.numel(), device="cuda").view_as(big.table))
    big.append(1, k, v)
    big.advance(300)
    q = r(8, 1, 8, 128).half()
    check_attend(big.attend(1, q, causal=False), big, 1, q, [0] * 8, False)
    del c


@pytest.mark.parametrize("dim", [32, 64, 128])
@pytest.mark.parametrize("block", [16, 64])
def test_a_prompt_over_a_long_row(lm, dim, block):
    """Many queries and many tokens: tiles beyond the first 32, parts, ragged ends."""
    c = filled(lm, 2, 3000, 1, dim, block, torch.float16, seed=dim)
    c.lens.copy_(torch.tensor([2800, 1203]))
    q = gen(dim)(2, 130, 2, dim).half()
    new = torch.tensor([130, 77], dtype=torch.int32, device="cuda")
    check_attend(c.attend(0, q, new), c, 0, q, new.tolist(), True)
    check_attend(c.attend(0, q, new, causal=False), c, 0, q, new.tolist(), False)


def test_results_repeat(lm):
    """Parts are joined in order, whichever finishes last."""
    c = filled(lm, 2, 30000, 2, 64, 32, torch.bfloat16, seed=3)
    c.lens.copy_(torch.tensor([29000, 17001]))
    q = gen(3)(2, 3, 4, 64).bfloat16()
    first = c.attend(0, q, causal=False)
    for _ in range(20):
        assert torch.equal(first, c.attend(0, q, causal=False))


def test_garbage_past_the_rows_does_not_matter(lm):
    c = filled(lm, 3, 200, 2, 64, 16, torch.float16, seed=7)
    c.lens.copy_(torch.tensor([50, 0, 97]))
    q = gen(3)(3, 2, 2, 64).half()
    new = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    want = c.attend(0, q, new).clone()
    # A poisoned block in the last open tile, absent and wild table entries, masked tokens' bytes.
    for r, n in ((0, 52), (1, 0), (2, 98)):
        used = -(-n // 16)
        wild = c.table[r, used:].long().clone()
        c.k_scale[0, wild] = math.nan
        c.v_scale[0, wild] = math.inf
        c.k8[0, wild] = -128
        c.table[r, used + 1:] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31], device="cuda",
                                             dtype=torch.int32).repeat(10)[:c.table.shape[1] - used - 1]
        if n % 16:
            c.k8[0, c.table[r, used - 1].long(), :, n % 16:] = -128
            c.v8[0, c.table[r, used - 1].long(), :, n % 16:] = -128
    assert torch.equal(c.attend(0, q, new), want)


def test_absent_blocks_count_as_absent_tokens(lm):
    c = filled(lm, 1, 128, 1, 64, 32, torch.bfloat16, seed=5)
    d = filled(lm, 1, 128, 1, 64, 32, torch.bfloat16, seed=5)
    c.lens.fill_(128)
    d.lens.fill_(96)
    c.table[0, 1] = -1
    d.table[0, 1:3] = c.table[0, 2:4]
    q = gen(5)(1, 1, 1, 64).bfloat16()
    torch.testing.assert_close(c.attend(0, q, causal=False), d.attend(0, q, causal=False), rtol=2 ** -7, atol=2 ** -9)
    c.table.fill_(-1)
    assert not c.attend(0, q, causal=False).any()


def test_scales_of_very_different_blocks(lm):
    # Blocks whose values differ by 2^40: small ones count where their weights do.
    c = filled(lm, 2, 128, 1, 64, 32, torch.float16, seed=6)
    for j, s in enumerate((2.0 ** -30, 8.0, 2.0 ** -12, 0.0)):
        c.v_scale[0, c.table[:, j].long()] = s / 127
    c.k_scale.fill_(2.0 ** -9)
    c.lens.copy_(torch.tensor([32, 128]))
    q = gen(6)(2, 1, 1, 64).half()
    check_attend(c.attend(0, q, causal=False), c, 0, q, [0, 0], False)


def test_scores_of_any_size(lm):
    c = filled(lm, 2, 300, 2, 64, 32, torch.bfloat16, seed=8)
    c.lens.fill_(290)
    for mag in (0.0, 1e-30, 40.0, 3000.0):
        q = (gen(4)(2, 1, 2, 64) * mag).bfloat16()
        check_attend(c.attend(0, q), c, 0, q, [1, 1], True)
        check_attend(c.attend(0, q, scale=-0.3), c, 0, q, [1, 1], True, scale=-0.3)


def test_lengths_past_the_table_and_below_zero(lm):
    c = filled(lm, 3, 96, 1, 64, 32, torch.float16, seed=9)
    c.lens.copy_(torch.tensor([96, -5, 95], dtype=torch.int32))
    q = gen(9)(3, 4, 1, 64).half()
    check_attend(c.attend(0, q), c, 0, q, [4, 4, 4], True)
    k = gen(10)(3, 4, 1, 64).half()
    before = c.k8.clone()
    c.append(0, k, k)
    changed = (c.k8 != before).flatten(2).any(-1)[0].nonzero().flatten().tolist()
    assert set(changed) <= {int(c.table[1, 0]), int(c.table[2, 2])}


def test_strided_queries_streams_and_graphs(lm):
    c = filled(lm, 5, 700, 4, 64, 32, torch.bfloat16, seed=10)
    c.lens.copy_(torch.tensor([3, 650, 200, 0, 64]))
    fused = gen(11)(5, 2, 3 * 4 * 64 + 4).bfloat16()
    q = fused[..., 2:2 + 4 * 64].unflatten(-1, (4, 64))
    want = c.attend(0, q.contiguous())
    assert torch.equal(c.attend(0, q), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a, b = c.attend(0, q), c.attend(0, q, stream=s)
        s.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(0, q, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)


def test_calls_of_many_shapes_share_their_scratch(lm):
    """Rows long enough to be split, and row counts that change from call to call."""
    shapes = [(1, 1, 9000, 1), (3, 2, 5000, 1), (1, 8, 4000, 4), (30, 4, 2000, 1), (2, 1, 20000, 2), (6, 6, 1500, 20)]
    made = []
    for i, (rows, heads, tokens, t) in enumerate(shapes):
        c = filled(lm, rows, tokens, heads, 64, 32, torch.float16, seed=i)
        c.lens.fill_(tokens - t)
        made.append((c, gen(i)(rows, t, heads, 64).half()))
    first = [c.attend(0, q) for c, q in made]
    for c, q in made:
        check_attend(c.attend(0, q), c, 0, q, [q.shape[1]] * c.rows, True)
    for _ in range(3):
        for (c, q), want in zip(reversed(made), reversed(first)):
            assert torch.equal(c.attend(0, q), want)
        for (c, q), want in zip(made, first):
            assert torch.equal(c.attend(0, q), want)


# ---- reorder --------------------------------------------------------------

@pytest.mark.parametrize("block,layers", [(16, 1), (32, 3), (128, 2)])
def test_beams_follow_their_parents(lm, block, layers):
    """Many steps of append and reorder against rows that are copied whole."""
    clips, beams, heads, dim = 3, 4, 2, 32
    rows, steps = clips * beams, 75
    c = lm.KvCache(rows, steps, heads, dim, layers=layers, block=block, dtype=torch.float16)
    g = torch.Generator(device="cuda").manual_seed(block)
    mine = [torch.zeros((rows, steps, heads, dim), dtype=torch.int32, device="cuda") for _ in range(2 * layers)]
    for step in range(steps):
        for layer in range(layers):
            # Scales that never grow after the first token of a block: each block is exact on its own grid.
            k, v = (torch.randint(-127, 128, (rows, 1, heads, dim), generator=g, device="cuda") for _ in range(2))
            k[..., 0], v[..., 0] = 127, -127
            c.append(layer, k.half(), v.half())
            mine[2 * layer][:, step], mine[2 * layer + 1][:, step] = k[:, 0].int(), v[:, 0].int()
        c.advance(1)
        parents = torch.randint(0, beams, (clips, beams), generator=g, device="cuda", dtype=torch.int32)
        c.reorder(parents)
        whole = (torch.arange(clips, device="cuda")[:, None] * beams + parents).flatten()
        mine = [m[whole] for m in mine]
        names = torch.cat([c.table.flatten(), c.spare])
        assert 0 <= int(names.min()) and int(names.max()) < c.blocks
        own = torch.cat([c.table[:, (step + 1) // block:].flatten(), c.spare])
        assert own.unique().numel() == own.numel()  # blocks yet to be written belong to one row
    k, v = c.read(None, 0, steps)
    for layer in range(layers):
        assert torch.equal(k[layer].int(), mine[2 * layer]) and torch.equal(v[layer].int(), mine[2 * layer + 1])


def test_a_step_of_every_operation_in_turn(lm):
    """Operations that use scratch, one after another on one stream, do not disturb each other's."""
    clips, beams = 2, 3
    c = filled(lm, 6, 900, 2, 64, 16, torch.float16, seed=3)
    c.lens.fill_(700)
    r = gen(5)
    logits, scores, w = r(clips, beams, 5000), r(clips, beams), r(64, 128).half()
    q = r(6, 1, 2, 64).half()
    table, spare, first = c.table.clone(), c.spare.clone(), None
    for _ in range(4):
        c.table.copy_(table)
        c.spare.copy_(spare)
        step = lm.beam_step(logits, scores)
        c.reorder(step.parents)
        got = [*step[:3], c.attend(0, q, causal=False), lm.linear(q.view(6, 128), w), c.table.clone(), c.spare.clone()]
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b)
    whole = (torch.arange(clips, device="cuda")[:, None] * beams + step.parents).flatten().long()
    assert torch.equal(c.table[:, :43], table[whole][:, :43])


def test_parents_out_of_range_leave_their_rows(lm):
    c = filled(lm, 4, 64, 1, 32, 16, torch.float16, seed=1)
    c.lens.fill_(20)
    was = c.table.clone(), c.spare.clone(), c.k8.clone()
    c.reorder(torch.tensor([[0, 1], [-1, 7]], dtype=torch.int32, device="cuda"))
    assert torch.equal(was[0], c.table) and torch.equal(was[1], c.spare) and torch.equal(was[2], c.k8)


def test_read_of_parts(lm):
    c = filled(lm, 2, 90, 2, 64, 16, torch.bfloat16, seed=2, layers=2)
    c.lens.copy_(torch.tensor([50, 90]))
    k, v = c.read(1, 13, 60)
    assert k.shape == (2, 60, 2, 64)
    assert torch.equal(k[0, :37], row32(c, "k", 1, 0, 50)[13:].bfloat16()) and not k[0, 37:].any()
    assert torch.equal(v[1], row32(c, "v", 1, 1, 73)[13:].bfloat16())
    k2, v2 = c.read(None, 13, 60)
    assert torch.equal(k2[1], k) and torch.equal(v2[1], v) and k2.shape == (2, 2, 60, 2, 64)
    assert c.read(0, 5, 0)[0].shape == (2, 0, 2, 64)
    past = c.read(0, 1000, 3)[0]
    assert not past.any()


def test_refusals(lm):
    for bad in (dict(head_dim=48), dict(block=24), dict(dtype=torch.float32), dict(device="cpu"), dict(heads=0),
                dict(layers=0), dict(rows=-1)):
        with pytest.raises(ValueError):
            lm.KvCache(**{**dict(rows=2, max_tokens=64, heads=2, head_dim=64), **bad})
    c = lm.KvCache(2, 64, 2, 64, dtype=torch.float16)
    k = torch.zeros((2, 3, 2, 64), device="cuda", dtype=torch.float16)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: c.append(1, k, k), lambda: c.append(0, k, k[:, :2]), lambda: c.append(0, k.float(), k),
                lambda: c.append(0, k, k.cpu()), lambda: c.append(0, k[:1], k[:1]), lambda: c.append(0, k, k, n.long()),
                lambda: c.append(0, k, k, n[:1]), lambda: c.append(0, k.transpose(2, 3), k),
                lambda: c.attend(0, k[:, :, :1]), lambda: c.attend(-1, k), lambda: c.attend(0, k.bfloat16()),
                lambda: c.attend(0, k, out=k.float()), lambda: c.read(0, -1, 2), lambda: c.read(2, 0, 2),
                lambda: c.reorder(n), lambda: c.reorder(n.view(1, 2).long()), lambda: c.reorder(n.view(2, 1)[:1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError, match="inference-only"):
        c.attend(0, k.requires_grad_())


def test_outputs_that_overlap_queries(lm):
    c = lm.KvCache(2, 64, 2, 64, dtype=torch.float16)
    k = torch.randn((2, 3, 2, 64), device="cuda").half()
    c.append(0, k, k)
    q = k.clone()
    with pytest.raises(lm.LogmelError, match="INVALID_ARG"):
        c.attend(0, q, out=q)
    both = torch.randn((2, 2, 3, 2, 64), device="cuda").half()
    got = c.attend(0, both[0], out=both[1])
    assert torch.equal(got, c.attend(0, both[0].clone()))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,heads,dim,tokens,t,group,causal", [
    (160, 5, 64, 70, 1, 1, True), (200, 6, 32, 40, 1, 2, False), (130, 7, 128, 100, 1, 1, True),
    (120, 9, 64, 33, 5, 4, False), (90, 13, 128, 17, 5, 8, False), (321, 3, 64, 200, 1, 1, True), (150, 6, 32, 64, 17, 1, True)])
def test_many_rows_of_few_tokens(lm, dtype, rows, heads, dim, tokens, t, group, causal):
    """More rows and heads than the device has room for: heads need not fill a CTA's four warps."""
    c = filled(lm, rows, tokens, heads, dim, 16, dtype, seed=rows)
    c.lens.copy_(torch.arange(rows) * 7 % (tokens - t + 1))
    q = gen(heads)(rows, t, heads * group, dim).to(dtype)
    out = c.attend(0, q, causal=causal)
    check_attend(out, c, 0, q, [t] * rows if causal else [0] * rows, causal)
    assert torch.equal(out, c.attend(0, q, causal=causal))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,heads,dim,tokens,t,group,causal", [
    (48, 10, 64, 160, 64, 1, True), (50, 12, 32, 100, 50, 1, False), (30, 12, 128, 150, 130, 1, True),
    (60, 8, 64, 90, 16, 4, True), (40, 11, 128, 40, 7, 8, False), (20, 16, 64, 448, 223, 1, True)])
def test_many_queries_of_many_rows(lm, dtype, rows, heads, dim, tokens, t, group, causal):
    """Tiles of 64 queries that fill the device, and their ragged ends."""
    c = filled(lm, rows, tokens, heads, dim, 32, dtype, seed=rows)
    c.lens.copy_(torch.arange(rows) * 5 % (tokens - t + 1))
    counts = torch.tensor([t if r % 7 else r % 3 for r in range(rows)], dtype=torch.int32, device="cuda")
    q = gen(heads)(rows, t, heads * group, dim).to(dtype)
    out = c.attend(0, q, counts if causal else None, causal=causal)
    check_attend(out, c, 0, q, counts.tolist() if causal else [0] * rows, causal)


@pytest.mark.parametrize("rows,heads,group,dim,t", [(1, 1, 1, 64, 1), (1, 1, 4, 32, 1), (2, 1, 8, 128, 2), (1, 2, 3, 64, 11)])
def test_rows_of_many_parts(lm, rows, heads, group, dim, t):
    """One or two units over the whole device: more parts than a warp has lanes."""
    c = filled(lm, rows, 90000, heads, dim, 64, torch.float16, seed=dim)
    c.lens.copy_(torch.tensor([89000, 40001][:rows]))
    q = gen(t)(rows, t, heads * group, dim).half()
    out = c.attend(0, q)
    check_attend(out, c, 0, q, [t] * rows, True)
    assert torch.equal(out, c.attend(0, q))
