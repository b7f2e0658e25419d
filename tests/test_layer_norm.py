"""layer_norm() and its gradients against the definition in 64 bits.

Tolerances, from the arithmetic.  A sum of C terms in 32 bits whose parts are summed by 128 threads or more and
joined is off by at most E = (C / 128 + 64) 2^-24 of the sum of magnitudes.  The deviations d are taken about a
mean that is off by E |mean| and put right by their own average, which is off by E avg|d|; the variance is off by
2 E of itself and its root by E.  So n = (x - mean) / sqrt(var + eps) is off by
    N = 4 E (|n| + 1 + E |mean| / sqrt(var + eps)).
y takes N |w| and 2^-23 of |n w| + |b|; dx, with h = g w, takes
    r (2^-22 |h| + E avg|h| + |n| (E avg|h n| + avg(|h| N)) + N |avg(h n)|) and (E + 2^-21) of itself;
sums over R rows take N and (R / 64 + 512) 2^-24 of the sum of magnitudes.  Each result is then rounded once: half a
step is 2^-24 (f32), 2^-11 (f16) or 2^-8 (bf16) of it, and 2^-25 where f16 is subnormal.
"""
import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def rounding(ref, dtype):
    return 1.001 * HALF_STEP[dtype] * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 1e-44)


def within(got, ref, tol, dtype):
    assert got.dtype == dtype and got.shape == ref.shape
    gap = (got.double() - ref).abs() - tol - rounding(ref, dtype)
    assert bool((gap <= 0).all()), float(gap.max())


class Definition:
    def __init__(self, x, w, b, eps):
        x = x.double().reshape(-1, x.shape[-1])
        c = x.shape[1]
        self.e = (c / 128 + 64) * 2.0 ** -24
        var, mean = torch.var_mean(x, -1, keepdim=True, correction=0)
        self.r = 1 / torch.sqrt(var + eps)
        self.n = (x - mean) * self.r
        self.w = torch.ones(c, dtype=torch.float64, device=x.device) if w is None else w.double()
        self.b = torch.zeros(c, dtype=torch.float64, device=x.device) if b is None else b.double()
        self.off = 4 * self.e * (self.n.abs() + 1 + self.e * mean.abs() * self.r)

    def check(self, y):
        ref = self.n * self.w + self.b
        tol = self.off * self.w.abs() + 2.0 ** -23 * ((self.n * self.w).abs() + self.b.abs())
        within(y.reshape(ref.shape), ref, tol, y.dtype)

    def check_dx(self, dx, g):
        g = g.double().reshape(self.n.shape)
        h, n, r, off, e = g * self.w, self.n, self.r, self.off, self.e
        avg = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
        ref = r * (h - avg(h) - n * avg(h * n))
        tol = r * (2.0 ** -22 * h.abs() + e * avg(h.abs()) + n.abs() * (e * avg((h * n).abs()) + avg(h.abs() * off))
                   + off * avg(h * n).abs()) + (e + 2.0 ** -21) * ref.abs()
        within(dx.reshape(ref.shape), ref, tol, dx.dtype)

    def check_sums(self, dw, db, g):
        g = g.double().reshape(self.n.shape)
        rows = (g.shape[0] / 64 + 512) * 2.0 ** -24
        if dw is not None:
            within(dw, (g * self.n).sum(0), (g.abs() * self.off).sum(0) + rows * (g * self.n).abs().sum(0), dw.dtype)
        if db is not None:
            within(db, g.sum(0), rows * g.abs().sum(0), db.dtype)


def inputs(rows, width, dtype, wtype, seed=0, offset=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = r(rows, width) * (r(rows, 1).abs() + 0.1) + offset * r(rows, 1)
    return x.to(dtype), (1 + 0.3 * r(width)).to(wtype), r(width).to(wtype), r(rows, width).to(dtype)


def both(lm, x, w, b, g, eps=1e-5):
    d = Definition(x, w, b, eps)
    leaves = [t.detach().requires_grad_() if t is not None else None for t in (x, w, b)]
    y = lm.layer_norm(*leaves, eps=eps)
    d.check(y.detach())
    with torch.no_grad():
        assert torch.equal(lm.layer_norm(x, w, b, eps=eps), y) or y.isnan().any()
    grads = torch.autograd.grad(y, [t for t in leaves if t is not None], g)
    d.check_dx(grads[0], g)
    rest = list(grads[1:])
    d.check_sums(rest.pop(0) if w is not None else None, rest.pop(0) if b is not None else None, g)
    return y, grads


SIZES = [(1, 1), (1, 2), (3, 7), (5, 32), (2, 33), (7, 64), (1, 255), (4, 256), (33, 257), (9, 511), (300, 768), (65, 771),
         (5, 1024), (1300, 1024), (17, 1025), (40, 1280), (3, 2047), (6, 2048), (19, 3000), (11, 4096), (2, 4099),
         (50, 8192), (3, 8200), (2, 16384), (3, 16392), (2, 20001), (1, 70000), (3000, 24), (5000, 3)]


@pytest.mark.parametrize("rows,width", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_sizes(lm, rows, width, dtype):
    x, w, b, g = inputs(rows, width, dtype, torch.float32, seed=rows + width)
    both(lm, x, w, b, g)


MANY = [(700, 1025), (1300, 1280), (650, 1536), (700, 2047), (1301, 2048), (620, 2560), (620, 3001), (650, 4096), (610, 4104),
        (620, 5120), (609, 6150), (650, 8192), (640, 8200), (620, 9001)]


@pytest.mark.parametrize("rows,width", MANY)
@pytest.mark.parametrize("dtype", TYPES)
def test_many_wide_rows(lm, rows, width, dtype):
    """Teams of fewer threads than few rows have."""
    x, w, b, g = inputs(rows, width, dtype, torch.float32, seed=rows + width)
    both(lm, x, w, b, g)


@pytest.mark.parametrize("dtype", TYPES[1:])
@pytest.mark.parametrize("width", [1, 100, 1024, 5000])
def test_parameters_of_the_inputs_type_or_none(lm, dtype, width):
    x, w, b, g = inputs(21, width, dtype, dtype, seed=width)
    both(lm, x, w, b, g)
    both(lm, x, w.float(), b, g)
    both(lm, x, None, None, g)
    both(lm, x, w, None, g, eps=0.1)
    both(lm, x, None, b.float(), g)


def test_rows_far_from_zero(lm):
    """The mean is 10^4 deviations: an average that is rounded to 32 bits alone would be felt."""
    x, w, b, g = inputs(30, 1000, torch.float32, torch.float32, seed=5)
    both(lm, x + 1e4 * x.std(), w, b, g)


@pytest.mark.parametrize("width", [1, 640, 1024, 9000, 17000])
def test_constant_rows_and_rows_that_are_not_finite(lm, width):
    x = torch.full((5, width), 0.1, device="cuda")
    x[1] = 0
    y = lm.layer_norm(x, eps=1e-5)
    assert (y.abs() <= 1e-2).all()  # 0.1 rounds off by 2^-27 at most, times 1 / sqrt(1e-5)
    x[2, -1], x[3, 0] = float("nan"), float("inf")
    y = lm.layer_norm(x)
    assert y[2:4].isnan().all() and y[[0, 1, 4]].isfinite().all()
    assert lm.layer_norm(x[:1] * 0, eps=0.0).isnan().all()  # 0 / 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [64, 1024, 1023, 4096])
def test_strides_and_alignment(lm, dtype, width):
    x, w, b, g = inputs(4 * 6, width + 40, dtype, torch.float32, seed=3)
    for view, grad in ((x[:, 8:8 + width], g[:, 3:3 + width]), (x[:, 1:1 + width], g[:, 8:8 + width]),
                       (x[::2, :width], g[::2, 40:]), (x.view(4, 6, -1)[..., 16:16 + width], g.view(4, 6, -1)[..., :width]),
                       (x[0, :width], g[0, :width]), (x[3:4, 5:5 + width], g[0, :width].expand(1, -1))):
        both(lm, view, w[:width], b[1:1 + width], grad)
    flat = x.view(-1)
    windows = flat.as_strided((5, width), (8, 1))  # rows that overlap
    both(lm, windows, w[3:3 + width], b[:width], g[:5, :width])
    y, _ = both(lm, windows.expand(3, 5, width)[:1], None, None, g[:5, :width][None])
    lone = x[:1, :width].detach().requires_grad_()  # one row for all: its gradient is the rows' sum
    y = lm.layer_norm(lone.expand(6, -1), w[:width])
    got, = torch.autograd.grad(y, lone, g[:6, :width])
    each = torch.autograd.grad(lm.layer_norm(lone, w[:width]), lone, g[:6, :width].double().sum(0)[None].to(dtype))[0]
    assert got.shape == each.shape
    with pytest.raises(ValueError, match="evenly spaced"):
        lm.layer_norm(x.view(4, 6, -1)[:, :5, :width])


def test_gradients_that_are_expanded_or_strided(lm):
    x, w, b, g = inputs(12, 256, torch.float32, torch.float32)
    x3 = x.view(3, 4, 256).requires_grad_()
    d = Definition(x.detach(), w, b, 1e-5)
    for grad in (torch.ones((), device="cuda").expand(3, 4, 256), g.view(3, 4, 256).transpose(0, 1).contiguous().transpose(0, 1),
                 g.t().contiguous().t().view(3, 4, 256), g[:1].expand(12, 256).view(3, 4, 256)):
        dx, = torch.autograd.grad(lm.layer_norm(x3, w, b), x3, grad)
        d.check_dx(dx, grad)


def test_out(lm):
    x, w, b, _ = inputs(20, 300, torch.bfloat16, torch.float32)
    ref = lm.layer_norm(x, w, b)
    wide = torch.zeros((20, 320), device="cuda", dtype=torch.bfloat16)
    assert lm.layer_norm(x, w, b, out=wide[:, 7:307]).data_ptr() == wide.data_ptr() + 14
    assert torch.equal(wide[:, 7:307], ref) and not wide[:, :7].any() and not wide[:, 307:].any()
    same = x.clone()
    assert lm.layer_norm(same, w, b, out=same) is same and torch.equal(same, ref) and same._version == 1
    with pytest.raises(lm.LogmelError):
        lm.layer_norm(x, w, b, out=torch.empty(300, device="cuda", dtype=torch.bfloat16).expand(20, 300))
    buf = torch.zeros(20 * 300 + 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(lm.LogmelError):
        lm.layer_norm(buf[:6000].view(20, 300), out=buf[8:].view(20, 300))
    with pytest.raises(RuntimeError, match="out goes without gradients"):
        lm.layer_norm(x.detach().requires_grad_(), out=torch.empty_like(x))


def test_empty(lm):
    for shape in ((0, 5), (5, 0), (0, 0), (2, 0, 3), (0,)):
        x = torch.zeros(shape, device="cuda", requires_grad=True)
        w = torch.ones(shape[-1], device="cuda", requires_grad=True)
        b = torch.ones(shape[-1], device="cuda", requires_grad=True)
        y = lm.layer_norm(x, w, b)
        assert y.shape == x.shape
        dx, dw, db = torch.autograd.grad(y.sum(), (x, w, b))
        assert dx.shape == x.shape and not dw.any() and not db.any() and dw.shape == w.shape


def test_which_gradients_are_taken(lm):
    x, w, b, g = inputs(50, 200, torch.float16, torch.float32)
    full = torch.autograd.grad(lm.layer_norm(*(t.requires_grad_() for t in (x, w, b))), (x, w, b), g)
    for i in range(3):
        ts = [t.detach().requires_grad_(j == i) for j, t in enumerate((x, w, b))]
        got, = torch.autograd.grad(lm.layer_norm(*ts), ts[i], g)
        assert torch.equal(got, full[i])
    y = lm.layer_norm(x, w, b)
    y.backward(g)
    assert torch.equal(x.grad, full[0]) and torch.equal(w.grad, full[1]) and torch.equal(b.grad, full[2])


def test_gradients_against_differences(lm):
    """<gradient, v> is the slope of sum(g y) along v.  A central difference with step t takes 2^-24 of each
    rounded y on either side, the tolerance of the values, and what the definition's own difference is off by."""
    x, w, b, g = inputs(6, 90, torch.float32, torch.float32, seed=9)
    _, v, u, _ = inputs(6, 90, torch.float32, torch.float32, seed=10)
    vx = torch.randn_like(x)
    leaves = [t.detach().requires_grad_() for t in (x, w, b)]
    grads = torch.autograd.grad(lm.layer_norm(*leaves), leaves, g)
    slope = sum((a.double() * c.double()).sum() for a, c in zip(grads, (vx, v, u)))
    t = 2.0 ** -7
    ends, ends64, noise = [], [], 0.0
    for s in (t, -t):
        p = [a + s * c for a, c in zip((x, w, b), (vx, v, u))]
        d = Definition(*p, 1e-5)
        ref = d.n * d.w + d.b
        ends64.append((g.double() * ref).sum())
        ends.append((g.double() * lm.layer_norm(*p).double()).sum())
        # (x + s v rounds to 32 bits as well)
        noise += float((g.double().abs() * (d.off * d.w.abs() + 2.0 ** -22 * (ref.abs() + d.b.abs() + 8 * d.r))).sum())
    exact = [a.double().requires_grad_() for a in (x, w, b)]
    var, mean = torch.var_mean(exact[0], -1, keepdim=True, correction=0)
    want = torch.autograd.grad((exact[0] - mean) / torch.sqrt(var + 1e-5) * exact[1] + exact[2], exact, g.double())
    want = sum((a * c.double()).sum() for a, c in zip(want, (vx, v, u)))
    bend = abs((ends64[0] - ends64[1]) / (2 * t) - want)
    assert abs((ends[0] - ends[1]) / (2 * t) - slope) <= bend + noise / (2 * t) + 1e-4 * slope.abs()


def test_refusals(lm):
    x, w, b, _ = inputs(4, 64, torch.float16, torch.float32)
    for bad in (lambda: lm.layer_norm(x.cpu()), lambda: lm.layer_norm(x.double()), lambda: lm.layer_norm(x, w[:63]),
                lambda: lm.layer_norm(x, w.cpu()), lambda: lm.layer_norm(x, w.bfloat16()),
                lambda: lm.layer_norm(x, w, b.double()), lambda: lm.layer_norm(x.t()), lambda: lm.layer_norm(x, eps=-1.0),
                lambda: lm.layer_norm(x, eps=float("nan")), lambda: lm.layer_norm(x, w.repeat(2)[::2]),
                lambda: lm.layer_norm(x, out=torch.empty_like(x).float()), lambda: lm.layer_norm(x, out=x[:3]),
                lambda: lm.layer_norm(x[0, 0])):
        with pytest.raises(ValueError):
            bad()
    with fwd.dual_level(), pytest.raises(RuntimeError, match="tangent"):
        lm.layer_norm(fwd.make_dual(x.float(), x.float()))
    x = x.detach().requires_grad_()
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(lm.layer_norm(x).sum(), x, create_graph=True)
    y = lm.layer_norm(x)
    with torch.no_grad():
        x.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_repeats_its_bits(lm):
    x, w, b, g = inputs(4001, 1024, torch.bfloat16, torch.float32)
    first = both(lm, x, w, b, g)
    again = both(lm, x, w, b, g)
    assert torch.equal(first[0], again[0]) and all(torch.equal(p, q) for p, q in zip(first[1], again[1]))


def test_streams_and_graphs(lm):
    x, w, b, g = inputs(700, 520, torch.bfloat16, torch.float32)
    ref = lm.layer_norm(x, w, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(lm.layer_norm(x, w, b, stream=side).clone(), ref)
    side.synchronize()
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    want = torch.autograd.grad(lm.layer_norm(*leaves), leaves, g)
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(lm.layer_norm(*leaves), leaves, g)
    side.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that are replayed in turn: scratch of their own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = lm.layer_norm(*leaves)
            grads = torch.autograd.grad(y, leaves, g)
            y = y.detach()
        graphs.append((graph, y, grads))
    for _ in range(3):
        for graph, y, grads in graphs:
            y.zero_()
            for t in grads:
                t.zero_()
            graph.replay()
        for graph, y, grads in graphs:
            assert torch.equal(y, ref) and all(torch.equal(p, q) for p, q in zip(grads, want))
    with torch.no_grad():
        leaves[0].copy_(x * 2)
    graphs[0][0].replay()
    assert torch.equal(graphs[0][1], lm.layer_norm(x * 2, w, b))


def test_no_capture_beside_an_eager_graph_of_the_same_leaf(lm):
    x, w, b, g = inputs(8, 64, torch.float32, torch.float32)
    x.requires_grad_()
    alive = lm.layer_norm(x, w, b)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="default stream over the same leaf"):
        with torch.cuda.graph(graph):
            lm.layer_norm(x, w, b)
    del alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lm.layer_norm(x, w, b)
        dx, = torch.autograd.grad(y, x, g)
    graph.replay()
    Definition(x.detach(), w, b, 1e-5).check_dx(dx, g)
