"""linear() against its definition in 64 bits.

Tolerance, from the arithmetic: products of 16-bit values are exact in 32
bits; a sum of k of them (in any order, rounded or truncated to 32 bits) is off
by at most (k + 8) * 2^-23 * sum |x w|, plus as much of the bias; activations
are at most 1.13-Lipschitz and evaluated to 2^-20 of |z| + 2^-20; one rounding
to the output's type adds 2^-8 (bf16), 2^-11 (f16, or 2^-25 where subnormal)
or 2^-24 (f32) of the result.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -7.99, torch.float16: 2.0 ** -10.99, torch.float32: 2.0 ** -23.9}


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def act64(z, a):
    if a == "relu":
        return z.clamp(min=0)
    if a == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if a == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if a == "silu":
        return z * torch.sigmoid(z)
    return z


def check(y, x, w, bias=None, act=None, residual=None, scale=1.0):
    xd, wd = x.double(), w.double()
    k = x.shape[-1]
    z = torch.einsum("...k,nk->...n", xd, wd)
    mag = torch.einsum("...k,nk->...n", xd.abs(), wd.abs())
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ref = scale * act64(z, act)
    if residual is not None:
        ref = ref + residual.double()
    tol = abs(scale) * (1.13 * (k + 8) * 2.0 ** -23 * mag + 2.0 ** -20 * (z.abs() + 1)) + \
        UNIT[y.dtype] * (ref.abs() + 2.0 ** -14)
    assert y.shape == ref.shape
    bad = (y.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((y.double() - ref).abs() - tol).max()))


def make(shape, n, dtype, seed=0, bias=True, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    k = shape[-1]
    return (r(*shape).to(dtype), (r(n, k) / math.sqrt(max(k, 1))).to(dtype), r(n) if bias else None,
            r(*shape[:-1], n).to(dtype) if residual else None)


SIZES = [(1, 16, 8), (1, 1, 1), (5, 64, 64), (5, 512, 512), (3, 201, 80), (16, 1024, 1000), (17, 72, 129), (64, 80, 384),
         (65, 256, 257), (127, 333, 31), (128, 128, 128), (129, 64, 256), (200, 520, 500), (257, 1000, 513), (300, 4096, 40),
         (640, 96, 1024), (1500, 240, 512), (2, 5000, 50), (48, 640, 5001)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_sizes(lm, m, k, n, dtype):
    x, w, b, r = make((m, k), n, dtype, seed=m * 7 + k + n)
    check(lm.linear(x, w), x, w)
    check(lm.linear(x, w, b, activation="gelu", residual=r, scale=0.5), x, w, b, "gelu", r, 0.5)


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [7, 300])
def test_epilogues(lm, act, out_dtype, m):
    x, w, b, r = make((m, 128), 200, torch.bfloat16, seed=3)
    x = x * 3
    y = lm.linear(x, w, b.bfloat16(), activation=act, residual=r, scale=-1.5, out_dtype=out_dtype)
    assert y.dtype == out_dtype
    check(y, x, w, b.bfloat16(), act, r, -1.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bands,taps,hop", [(80, 3, 1), (128, 3, 2), (81, 3, 1), (16, 5, 3)])
def test_windows_of_frames_are_read_in_place(lm, dtype, bands, taps, hop):
    g = torch.Generator(device="cuda").manual_seed(5)
    frames = torch.rand((3, 211, bands), generator=g, device="cuda").to(dtype)
    rows = (211 - taps) // hop + 1
    x = frames.as_strided((3, rows, taps * bands), (211 * bands, hop * bands, 1))
    w = (torch.randn((100, taps * bands), generator=g, device="cuda") / math.sqrt(taps * bands)).to(dtype)
    y = lm.linear(x, w, activation="gelu")
    check(y, x, w, act="gelu")


def test_strides_and_leading_dimensions(lm):
    g = torch.Generator(device="cuda").manual_seed(6)
    big = torch.randn((4, 6, 2, 5, 136), generator=g, device="cuda").bfloat16()
    w = torch.randn((50, 200), generator=g, device="cuda").bfloat16()[:, 8:72]
    for x in (big[..., :64], big[..., 3:67], big[:, :, 0, :, :64], big[:, :, 1, 2, 8:72], big[0, 0, 0, :, :64],
              big[0, 0, 0, 0, :64], big[:, :1, :1, :, :64], big[2:3, 1, 0, :1, :64],
              big[:, 0, 0, :1, :64].expand(-1, 3, -1), big[:1, 0, 0, 0, :64].expand(9, -1)):
        try:
            y = lm.linear(x, w)
        except ValueError:
            assert x.dim() == 4 and x.shape[2] == 5  # [4, 6, 5, K] of every second 5: not evenly spaced
            continue
        check(y, x, w)
    x = big[0, 0, 0, :, :64]
    wide = torch.zeros((5, 80), device="cuda", dtype=torch.bfloat16)
    out = wide[:, 7:57]
    res = torch.randn((5, 2, 50), device="cuda", dtype=torch.bfloat16)[:, 1]
    assert lm.linear(x, w, residual=res, out=out) is out
    check(out, x, w, residual=res)
    assert not wide[:, :7].any() and not wide[:, 57:].any()
    both = res.clone()
    lm.linear(x, w, residual=both, out=both)
    check(both, x, w, residual=res)


def test_empty_and_degenerate(lm):
    x, w, b, r = make((4, 64), 32, torch.float16)
    assert lm.linear(x[:0], w).shape == (0, 32)
    assert lm.linear(x, w[:0]).shape == (4, 0)
    assert lm.linear(x.expand(0, 4, 64), w).shape == (0, 4, 32)
    check(lm.linear(x[:, :0], w[:, :0], b, activation="silu", residual=r), x[:, :0], w[:, :0], b, "silu", r)
    y = lm.linear(x, w, b)
    assert y.shape == (4, 32)


def test_infinities_and_nans_stay_in_their_rows(lm):
    for m in (6, 140):
        x, w, b, _ = make((m, 100), 70, torch.float16, seed=9)
        clean = lm.linear(x, w, b)
        x[2, 5] = math.nan
        x[4, 99] = math.inf
        y = lm.linear(x, w, b, activation="relu")
        assert y[2].isnan().sum() + (y[2] == 0).sum() == 70
        keep = [i for i in range(m) if i not in (2, 4)]
        assert torch.equal(y[keep], clean[keep].clamp(min=0))
        z = lm.linear(x, w, b)
        assert z[2].isnan().all() and not z[4].isfinite().any()


def test_calls_in_a_row_another_stream_and_a_graph(lm):
    a = [make((m, 768), n, torch.bfloat16, seed=m) for m, n in ((5, 700), (40, 256), (200, 333))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for x, w, b, r in a * 3:
        y = lm.linear(x, w, b, residual=r)
        z = lm.linear(x, w, b, residual=r, stream=s)
        s.synchronize()
        assert torch.equal(y, z)
        check(y, x, w, b, residual=r)
    outs = [torch.empty_like(t[3]) for t in a]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for (x, w, b, r), o in zip(a, outs):
            lm.linear(x, w, b, residual=r, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        for (x, w, b, r), o in zip(a, outs):
            assert torch.equal(o, lm.linear(x, w, b, residual=r))


def test_refusals(lm):
    x, w, b, r = make((4, 64), 32, torch.float16)
    for bad in (lambda: lm.linear(x.float(), w), lambda: lm.linear(x, w.bfloat16()), lambda: lm.linear(x.cpu(), w),
                lambda: lm.linear(x, w.cpu()), lambda: lm.linear(x, w[:, :60]), lambda: lm.linear(x[:, ::2], w[:, ::2]),
                lambda: lm.linear(x, w, b[:30]), lambda: lm.linear(x, w, b.double()),
                lambda: lm.linear(x, w, activation="tanh"), lambda: lm.linear(x, w, residual=r[:2]),
                lambda: lm.linear(x, w, residual=r.float()), lambda: lm.linear(x, w, out_dtype=torch.int32),
                lambda: lm.linear(x, w, out=torch.empty((4, 31), device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            bad()
    w.requires_grad_()
    with pytest.raises(RuntimeError, match="inference-only"):
        lm.linear(x, w)
    with torch.no_grad():
        lm.linear(x, w)


@pytest.mark.parametrize("m,k,n", [(3000, 1024, 4001), (1100, 4096, 2050), (6000, 130, 1000), (513, 2000, 9999),
                                   (20, 4096, 300), (33, 4095, 520), (7, 2049, 130), (130, 5000, 260), (3000, 3000, 80),
                                   (1, 8192, 64), (64, 640, 128)])
def test_every_way_of_cutting(lm, m, k, n):
    """Pairs of CTAs, several rounds of tiles, k split over clusters of 2, 4 and 8."""
    x, w, b, r = make((m, k), n, torch.bfloat16, seed=m + n)
    check(lm.linear(x, w, b, activation="silu", residual=r), x, w, b, "silu", r)
    check(lm.linear(x, w, out_dtype=torch.float32), x, w)


@pytest.mark.parametrize("bands", [80, 81])
def test_windows_of_many_frames(lm, bands):
    g = torch.Generator(device="cuda").manual_seed(8)
    frames = torch.rand((5, 1502, bands), generator=g, device="cuda").half()
    x = frames.as_strided((5, 1500, 3 * bands), (1502 * bands, bands, 1))
    w = (torch.randn((512, 3 * bands), generator=g, device="cuda") / 16).half()
    b = torch.randn(512, generator=g, device="cuda")
    check(lm.linear(x, w, b, activation="gelu"), x, w, b, "gelu")


def test_results_repeat(lm):
    for m, k, n in ((5, 1024, 1024), (200, 4096, 512), (3000, 1024, 1024)):
        x, w, b, r = make((m, k), n, torch.float16, seed=1)
        first = lm.linear(x, w, b, activation="gelu", residual=r)
        for _ in range(5):
            assert torch.equal(first, lm.linear(x, w, b, activation="gelu", residual=r))


def test_outputs_that_overlap_inputs(lm):
    """Refused where a byte is shared; columns of one buffer, and out = residual, are not."""
    for dtype in (torch.float16, torch.bfloat16):
        buf = torch.randn((40, 200), device="cuda").to(dtype)
        w = torch.randn((64, 64), device="cuda").to(dtype)
        x = buf[:, :64]
        for bad in (lambda: lm.linear(x, w, out=x), lambda: lm.linear(x, w, out=buf[:, 63:127]),
                    lambda: lm.linear(buf[:, 8:72], w, out=buf[:, 64:128]),
                    lambda: lm.linear(w, w, out=w), lambda: lm.linear(x, w, residual=buf[:, 100:164], out=buf[:, 104:168]),
                    lambda: lm.linear(x, w, out=torch.empty((1, 64), device="cuda", dtype=dtype).expand(40, 64)),
                    lambda: lm.linear(x, w, buf[3, 64:128], out=buf[:, 64:128])):
            with pytest.raises(lm.LogmelError, match="INVALID_ARG"):
                bad()
        want = lm.linear(x.clone(), w, residual=buf[:, 136:].clone())
        lm.linear(x, w, residual=buf[:, 136:], out=buf[:, 136:])
        assert torch.equal(buf[:, 136:], want)
        lm.linear(x, w, out=buf[:, 64:128])
        assert torch.equal(buf[:, 64:128], lm.linear(x.clone(), w))
        rows = torch.randn((16, 64), device="cuda").to(dtype)
        got = lm.linear(rows[8:], w, out=rows[:8])
        assert torch.equal(got, lm.linear(rows[8:].clone(), w))
