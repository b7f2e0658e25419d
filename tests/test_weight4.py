"""Weights in 4 bits: their rounding, and linear() with them, against the definitions in 64 bits.

Tolerance of linear: that of tests/test_linear.py with w = q s; the scale enters after a group's sum, which is
one more rounding of 2^-24 of each group.  For more than 16 rows each value is first rounded to
x's type: half a step, 2^-8 (bf16) or 2^-11 (f16, 2^-25 where subnormal), of every |x w|, and up to a sixteenth of
that for a scale in two parts: q * high + (q * low rounded), high and low of x's type.  In bf16 low's rounding and
its product's take 2^-17 of the value, 2^-9 of 2^-8; in f16 with scales from 2^-10 on low is off by at most 2^-25 (half
the least step), times |q| <= 8, against half a step of 2^-21 |q| at the least.
"""
import copy
import math
import pickle

import pytest
import torch
import torch.autograd.forward_ad as fwd

from test_linear import UNIT, act64

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def numbers(n, k, group, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-8, 8, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    s = torch.rand((n, -(-k // group)), generator=gen, device="cuda") + 0.25
    return q, s * (0.25 / math.sqrt(max(k, 1)))


def value64(q, s, group):
    return q.double() * s.double().repeat_interleave(group, 1)[:, :q.shape[1]]


def check(y, x, w, bias=None, act=None, residual=None, scale=1.0):
    xd = x.double()
    k, rows = x.shape[-1], x.numel() // max(1, x.shape[-1])
    z, mag = xd @ w.t(), xd.abs() @ w.t().abs()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ref = scale * act64(z, act)
    if residual is not None:
        ref = ref + residual.double()
    off = 1.13 * (k + 16) * 2.0 ** -23 * mag
    if rows > 16:
        off = off + 1.13 * (17 / 16 * UNIT[x.dtype] * mag + 2.0 ** -25 * xd.abs().sum(-1, keepdim=True))
    tol = abs(scale) * (off + 2.0 ** -20 * (z.abs() + 1)) + UNIT[y.dtype] * (ref.abs() + 2.0 ** -14)
    assert y.shape == ref.shape
    gap = (y.double() - ref).abs() - tol
    assert bool((gap <= 0).all()), float(gap.max())


SIZES = [(1, 16, 8, 32), (1, 1, 1, 32), (5, 64, 64, 64), (5, 512, 512, 128), (3, 201, 80, 64), (8, 1024, 1000, 32),
         (9, 72, 129, 32), (16, 130, 16, 128), (17, 2048, 100, 64), (31, 80, 384, 32), (33, 256, 257, 64), (5, 4096, 40, 128),
         (64, 333, 31, 32), (65, 96, 1024, 32), (100, 320, 500, 64), (129, 640, 130, 128), (320, 256, 300, 64),
         (700, 520, 250, 32), (2, 5000, 50, 64), (48, 64, 5001, 64), (1, 33, 17, 128)]


@pytest.mark.parametrize("m,k,n,group", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_sizes(lm, m, k, n, group, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m + k + n)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, s = numbers(n, k, group, seed=m)
    w4, w = lm.Weight4.pack(q, s, group=group, dtype=dtype), value64(q, s, group)
    x, b, res = r(m, k).to(dtype), r(n), r(m, n).to(dtype)
    check(lm.linear(x, w4), x, w)
    check(lm.linear(x, w4, b, activation="gelu", residual=res, scale=0.5), x, w, b, "gelu", res, 0.5)


@pytest.mark.parametrize("m", [16, 17, 40, 64, 70, 96, 128, 200, 300])
@pytest.mark.parametrize("group", [32, 128])
def test_more_tiles_than_multiprocessors(lm, m, group):
    """CTAs that go through several tiles, and come round in their rings more than once."""
    q, s = numbers(20001, 700, group, seed=m)
    x = torch.randn((m, 700), device="cuda", generator=torch.Generator(device="cuda").manual_seed(m)).half()
    check(lm.linear(x, lm.Weight4.pack(q, s, group=group, dtype=torch.float16)), x, value64(q, s, group))


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [7, 20, 300])
def test_epilogues(lm, act, out_dtype, m):
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, s = numbers(200, 128, 64)
    x, b, res = (r(m, 128) * 3).bfloat16(), r(200).bfloat16(), r(m, 200).bfloat16()
    y = lm.linear(x, lm.Weight4.pack(q, s), b, activation=act, residual=res, scale=-1.5, out_dtype=out_dtype)
    assert y.dtype == out_dtype
    check(y, x, value64(q, s, 64), b, act, res, -1.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [5, 12, 40, 150])
def test_strides_windows_and_alignment(lm, dtype, rows):
    gen = torch.Generator(device="cuda").manual_seed(7)
    frames = torch.randn((3, rows + 2, 81), generator=gen, device="cuda").to(dtype)
    for m, taps in ((80, 3), (81, 3), (64, 1)):
        f = frames[..., :m].contiguous()
        x = f.as_strided((3, rows, taps * m), ((rows + 2) * m, m, 1))
        q, s = numbers(100, taps * m, 32, seed=m)
        y = lm.linear(x, lm.Weight4.pack(q, s, group=32, dtype=dtype), activation="gelu")
        check(y.view(-1, 100), x.reshape(-1, taps * m), value64(q, s, 32), act="gelu")
    big = torch.randn((rows, 200), generator=gen, device="cuda").to(dtype)
    q, s = numbers(50, 128, 64)
    w4, w = lm.Weight4.pack(q, s, dtype=dtype), value64(q, s, 64)
    for x in (big[:, :128], big[:, 8:136], big[:, 3:131], big[:1, 1:129].expand(rows, -1), big[0, :128], big[::2, 2:130]):
        check(lm.linear(x, w4), x, w)
    wide = torch.zeros((rows, 80), device="cuda", dtype=dtype)
    lm.linear(big[:, :128], w4, out=wide[:, 7:57])
    check(wide[:, 7:57], big[:, :128], w)
    assert not wide[:, :7].any() and not wide[:, 57:].any()
    keep = wide.clone()
    lm.linear(big[:, :128], w4, residual=wide[:, 7:57], out=wide[:, 7:57])
    check(wide[:, 7:57], big[:, :128], w, residual=keep[:, 7:57])


@pytest.mark.parametrize("rows", [1, 200])
def test_what_is_not_finite(lm, rows):
    """A scale or x that is not finite reaches its own outputs only (q = 0 times infinity is NaN)."""
    q, s = numbers(40, 256, 64)
    x = torch.randn((rows, 256), device="cuda").half()
    ref = lm.linear(x, lm.Weight4.pack(q, s, dtype=torch.float16))
    s2 = s.clone()
    s2[3, 1], s2[17, 3] = float("nan"), float("inf")
    y = lm.linear(x, lm.Weight4.pack(q, s2, dtype=torch.float16))
    keep = [i for i in range(40) if i not in (3, 17)]
    assert y[:, 3].isnan().all() and not y[:, 17].isfinite().any() and torch.equal(y[:, keep], ref[:, keep])
    x[0, 100] = float("inf")
    y = lm.linear(x, lm.Weight4.pack(q, s, dtype=torch.float16))
    assert not y[0].isfinite().any() and torch.equal(y[1:], ref[1:])


@pytest.mark.parametrize("rows", [5, 16, 100, 1000])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [2.0 ** -18, 2.0 ** -12, -1.0, 2.0 ** 10])
def test_scales_of_any_size(lm, rows, dtype, size):
    q, s = numbers(150, 200, 32, seed=rows)
    x = torch.randn((rows, 200), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(dtype)
    w4 = lm.Weight4.pack(q, s * size, group=32, dtype=dtype)
    check(lm.linear(x, w4, out_dtype=torch.float32), x, value64(q, s * size, 32))


@pytest.mark.parametrize("rows", [16, 500])
def test_repeats_its_bits(lm, rows):
    q, s = numbers(300, 1000, 32)
    w4 = lm.Weight4.pack(q, s, group=32, dtype=torch.float16)
    x = torch.randn((rows, 1000), device="cuda").half()
    assert torch.equal(lm.linear(x, w4), lm.linear(x, w4))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 64), (17, 100), (33, 128), (40, 333), (5, 2048), (50, 32)])
def test_pack_and_values(lm, group, n, k):
    q, s = numbers(n, k, group, seed=n)
    for dtype in TYPES:
        w4 = lm.Weight4.pack(q, s, group=group, dtype=dtype)
        assert torch.equal(w4.values(torch.float32), q.float() * s.repeat_interleave(group, 1)[:, :k])
        assert torch.equal(w4.values(), (q.float() * s.repeat_interleave(group, 1)[:, :k]).to(dtype))
        assert w4.shape == (n, k) and w4.group == group and w4.device == q.device
    wild = q.clone()
    wild[0, 0] = 100
    assert lm.Weight4.pack(wild, s, group=group).values(torch.float32)[0, 0] == 7 * s[0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("n,k", [(1, 1), (17, 100), (33, 300), (100, 1024)])
def test_quantize(lm, dtype, group, n, k):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    w = torch.randn((n, k + 3), generator=gen, device="cuda").to(dtype)[:, 3:]
    w[n // 2, :min(k, 40)] = 0
    w4 = lm.quantize_weight(w, group)
    assert w4.dtype == (torch.bfloat16 if dtype == torch.float32 else dtype)
    pad = torch.nn.functional.pad(w.float(), (0, -k % group)).view(n, -1, group)
    m = pad.abs().amax(-1)
    s = torch.where(m > 0, (m.double() / 7).float(), 1.0)  # (torch divides by a number through its reciprocal)
    q = torch.round(pad / s[..., None])
    want = (q * s[..., None]).view(n, -1)[:, :k]
    assert torch.equal(w4.values(torch.float32), want)
    gap = (want - w.float()).abs() - 0.5001 * s.repeat_interleave(group, 1)[:, :k]
    assert bool((gap <= 0).all())


def test_quantize_what_is_not_finite(lm):
    w = torch.randn((4, 128), device="cuda")
    w[1, 5], w[2, 70] = float("nan"), float("inf")
    v = lm.quantize_weight(w, 64).values(torch.float32)
    assert v[1, :64].isnan().all() and v[2, 64:].isnan().all()
    assert v[0].isfinite().all() and v[3].isfinite().all() and v[1, 64:].isfinite().all() and v[2, :64].isfinite().all()


def test_copies(lm):
    q, s = numbers(20, 100, 64)
    w4 = lm.Weight4.pack(q, s, group=64, dtype=torch.float16)
    x = torch.randn((3, 100), device="cuda").half()
    ref = lm.linear(x, w4)
    deep, pickled = copy.deepcopy(w4), pickle.loads(pickle.dumps(w4))
    w4.packed.zero_()
    assert torch.equal(lm.linear(x, deep), ref) and torch.equal(lm.linear(x, pickled), ref)


def test_empty(lm):
    for m, k, n in ((0, 64, 8), (4, 64, 0), (4, 0, 8)):
        q, s = numbers(n, k, 64)
        w4 = lm.Weight4.pack(q, s, group=64, dtype=torch.float16)
        b = torch.randn(n, device="cuda")
        x = torch.randn((m, k), device="cuda").half()
        y = lm.linear(x, w4, b, activation="relu")
        assert y.shape == (m, n)
        if k == 0:
            assert torch.equal(y, b.clamp(min=0).half().expand(m, n))


def test_refusals(lm):
    q, s = numbers(32, 128, 64)
    w4 = lm.Weight4.pack(q, s, dtype=torch.float16)
    x = torch.randn((4, 128), device="cuda").half()
    for bad in (lambda: lm.linear(x.bfloat16(), w4), lambda: lm.linear(x[:, :64], w4), lambda: lm.linear(x.cpu(), w4),
                lambda: lm.Weight4.pack(q.cpu(), s), lambda: lm.Weight4.pack(q.int(), s), lambda: lm.Weight4.pack(q, s.half()),
                lambda: lm.Weight4.pack(q, s[:, :1]), lambda: lm.Weight4.pack(q, s[:31]), lambda: lm.Weight4.pack(q.t(), s),
                lambda: lm.Weight4.pack(q, s, group=48), lambda: lm.Weight4.pack(q, s, group=32),
                lambda: lm.Weight4.pack(q, s, dtype=torch.float32), lambda: lm.quantize_weight(x, 16),
                lambda: lm.quantize_weight(x.t()), lambda: lm.quantize_weight(x.double()), lambda: w4.values(torch.int8),
                lambda: lm.linear(x, lm.Weight4(w4.packed[:, :1], w4.scale, w4.shape, 64, torch.float16)),
                lambda: lm.linear(x, lm.Weight4(w4.packed, w4.scale, (1 << 20, 128), 64, torch.float16))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError, match="inference-only"):
        lm.linear(x.clone().requires_grad_(), w4)
    with fwd.dual_level(), pytest.raises(RuntimeError, match="inference-only"):
        lm.linear(fwd.make_dual(x, x), w4)
    with pytest.raises(lm.LogmelError):
        lm.linear(x, w4, out=x[:, :32])


@pytest.mark.parametrize("rows", [5, 300])
def test_streams_and_graphs(lm, rows):
    q, s = numbers(130, 256, 64)
    w4 = lm.Weight4.pack(q, s, dtype=torch.bfloat16)
    x = torch.randn((rows, 256), device="cuda").bfloat16()
    ref = lm.linear(x, w4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(lm.linear(x, w4, stream=side).clone(), ref)
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, lm.linear(x, w4)))
    for _ in range(3):
        for graph, y in graphs:
            y.zero_()
            graph.replay()
        assert all(torch.equal(y, ref) for _, y in graphs)
