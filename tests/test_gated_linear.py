"""gated_linear() and its gradients against the definition in 64 bits.

Tolerances, from the arithmetic.  A projection's sum of k exact products in 32 bits is off by at most
(k + 8) 2^-23 of the sum of magnitudes (and as much of the bias); call these A and B for a = x Wg^T + bg and
b = x Wu^T + bu.  Activations are at most 1.13-Lipschitz with derivatives that are at most 1.2-Lipschitz (relu's jumps
by 1 where |a| <= A), both evaluated to S = 2^-20 (1 + |a|).  So act(a) is off by 1.13 A + S, its derivative by 1.2 A + S,
and y = act(a) b, da = g b act'(a) and db = g act(a) by the products' rule.  da and db are rounded to x's type for the
products with the weights and x, whose sums of t terms take (t + 8) 2^-23 of the sum of magnitudes; the biases'
gradients are sums of what was not rounded.  Each result is rounded once: half a step is 2^-11 (f16; 2^-25 where
subnormal), 2^-8 (bf16) or 2^-24 (f32).
"""
import math

import pytest
import torch
import torch.autograd.forward_ad as fwd

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TYPES = [torch.float16, torch.bfloat16]
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid", None]


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def act64(z, act):
    """The value and the derivative."""
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    p = torch.sigmoid(z)
    if act == "silu":
        return z * p, p * (1 + z * (1 - p))
    if act == "sigmoid":
        return p, p * (1 - p)
    return z, torch.ones_like(z)


def rounding(ref, dtype):
    return 1.001 * HALF_STEP[dtype] * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 1e-38)


def within(got, ref, tol, what):
    assert got.shape == ref.shape, what
    gap = (got.double() - ref).abs() - tol - rounding(ref, got.dtype)
    assert bool((gap <= 0).all()), (what, float(gap.max()), float(ref.abs().max()))


class Definition:
    def __init__(self, x, wg, wu, bg, bu, act):
        self.dtype = x.dtype
        k = x.shape[-1]
        self.x, self.wg, self.wu = x.double().reshape(math.prod(x.shape[:-1]), k), wg.double(), wu.double()
        each = []
        for w, b in ((self.wg, bg), (self.wu, bu)):
            z, mag = self.x @ w.t(), self.x.abs() @ w.t().abs()
            if b is not None:
                z, mag = z + b.double(), mag + b.double().abs()
            each.append((z, (k + 8) * 2.0 ** -23 * mag))
        (a, self.ea), (self.b, self.eb) = each
        self.h, self.s = act64(a, act)
        s = 2.0 ** -20 * (1 + a.abs())
        self.eh, self.es = 1.13 * self.ea + s, 1.2 * self.ea + s
        if act == "relu":
            self.es = torch.where(a.abs() <= self.ea, 1.0, 0.0)

    def check(self, y):
        ref = self.h * self.b
        within(y.reshape(ref.shape), ref, self.eh * self.b.abs() + self.h.abs() * self.eb + self.eh * self.eb
               + 2.0 ** -23 * ref.abs(), "y")

    def check_grads(self, g, dx=None, dwg=None, dwu=None, dbg=None, dbu=None):
        g = g.double().reshape(self.h.shape)
        rows, n = g.shape
        da, db = g * self.b * self.s, g * self.h
        ta = g.abs() * (self.eb * (self.s.abs() + self.es) + self.b.abs() * self.es) + 2.0 ** -22 * da.abs()
        tb = g.abs() * self.eh + 2.0 ** -23 * db.abs()
        ra, rb = ta + rounding(da.abs() + ta, self.dtype), tb + rounding(db.abs() + tb, self.dtype)
        if dx is not None:
            tol = ra @ self.wg.abs() + rb @ self.wu.abs()
            tol = tol + (2 * n + 8) * 2.0 ** -23 * ((da.abs() + ra) @ self.wg.abs() + (db.abs() + rb) @ self.wu.abs())
            within(dx.reshape(rows, dx.shape[-1]), da @ self.wg + db @ self.wu, tol, "dx")
        for got, d, t, what in ((dwg, da, ra, "dWg"), (dwu, db, rb, "dWu")):
            if got is not None:
                mag = (d.abs() + t).t() @ self.x.abs()
                within(got, d.t() @ self.x, t.t() @ self.x.abs() + (rows + 8) * 2.0 ** -23 * mag, what)
        for got, d, t, what in ((dbg, da, ta, "dbg"), (dbu, db, tb, "dbu")):
            if got is not None:
                within(got, d.sum(0), t.sum(0) + (rows / 64 + 512) * 2.0 ** -24 * d.abs().sum(0), what)


def inputs(rows, k, n, dtype, seed=0, bias=True, btype=torch.float32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, wg, wu = r(rows, k).to(dtype), *((r(n, k) * (1.5 / math.sqrt(max(k, 1)))).to(dtype) for _ in range(2))
    bg, bu = ((0.5 * r(n)).to(btype) if bias else None for _ in range(2))
    return x, wg, wu, bg, bu, r(rows, n).to(dtype)


def both(lm, x, wg, wu, bg, bu, g, act="silu"):
    d = Definition(x, wg, wu, bg, bu, act)
    leaves = [t.detach().requires_grad_() if t is not None else None for t in (x, wg, wu, bg, bu)]
    y = lm.gated_linear(*leaves, activation=act)
    d.check(y.detach())
    with torch.no_grad():
        assert torch.equal(lm.gated_linear(x, wg, wu, bg, bu, activation=act), y)
    grads = iter(torch.autograd.grad(y, [t for t in leaves if t is not None], g))
    got = [next(grads) if t is not None else None for t in leaves]
    for t, leaf in zip(got, leaves):
        assert t is None or (t.dtype == leaf.dtype and t.shape == leaf.shape)
    d.check_grads(g, *got)
    return y.detach(), got


SIZES = [(1, 1, 1), (1, 16, 8), (5, 64, 64), (5, 512, 1000), (3, 201, 80), (16, 256, 500), (17, 72, 129), (64, 80, 384),
         (65, 256, 257), (127, 333, 31), (128, 128, 128), (129, 64, 256), (200, 520, 500), (257, 1000, 513), (300, 64, 40),
         (700, 96, 1024), (1500, 240, 520), (2, 3000, 50), (48, 640, 2001), (2100, 128, 64), (5000, 32, 24), (5000, 64, 2001),
         (9000, 72, 520)]


@pytest.mark.parametrize("rows,k,n", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_sizes(lm, rows, k, n, dtype):
    both(lm, *inputs(rows, k, n, dtype, seed=rows + k + n, bias=rows % 2 == 1), act=ACTS[(rows + k) % 3])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [3, 300])
def test_activations(lm, act, rows):
    x, *rest = inputs(rows, 128, 200, torch.bfloat16, seed=2)
    both(lm, x * 3, *rest, act=act)


@pytest.mark.parametrize("dtype", TYPES)
def test_biases(lm, dtype):
    x, wg, wu, bg, bu, g = inputs(33, 100, 72, dtype, btype=dtype)
    both(lm, x, wg, wu, bg, bu, g)
    both(lm, x, wg, wu, bg, None, g)
    both(lm, x, wg, wu, None, bu.float(), g)


@pytest.mark.parametrize("act", ACTS)
def test_large_values(lm, act):
    """|a| up to a few thousand: activations saturate, and nothing becomes NaN."""
    x, wg, wu, bg, bu, g = inputs(40, 64, 96, torch.bfloat16, seed=4)
    y, grads = both(lm, x * 1000, wg, wu, bg, bu, g, act=act)
    big = lm.gated_linear(x.float().mul(2.0 ** 60).bfloat16().requires_grad_(), wg, wu, activation=act)
    assert act in ("relu", None) or not big.isnan().any()


def test_what_is_not_finite_stays_in_its_row(lm):
    x, wg, wu, bg, bu, g = inputs(20, 64, 96, torch.bfloat16)
    ref = lm.gated_linear(x, wg, wu, bg, bu)
    x2 = x.clone()
    x2[3, 5], x2[7, 0] = float("nan"), float("inf")
    y = lm.gated_linear(x2, wg, wu, bg, bu)
    keep = [i for i in range(20) if i not in (3, 7)]
    assert y[3].isnan().all() and torch.equal(y[keep], ref[keep])
    leaf = x2.clone().requires_grad_()
    dx, = torch.autograd.grad(lm.gated_linear(leaf, wg, wu, bg, bu), leaf, g)
    want, = torch.autograd.grad(lm.gated_linear(x.requires_grad_(), wg, wu, bg, bu), x, g)
    assert dx[3].isnan().all() and torch.equal(dx[keep], want[keep])


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_leading_dimensions(lm, dtype):
    x, wg, wu, bg, bu, g = inputs(24, 136, 150, dtype, seed=6)
    k, n = 64, 50
    wg, wu, bg, bu = wg[:n, 8:72], wu[100:100 + n, 3:67], bg[:n], bu[9:9 + n]
    for v, gr in ((x[:, :k], g[:, :n]), (x[:, 3:67], g[:, 50:100]), (x[::2, 8:72], g[::2, 1:51]),
                  (x.view(4, 6, -1)[..., :k], g.view(4, 6, -1)[..., :n]), (x[0, :k], g[0, :n]),
                  (x[:1, 1:65], g[:1, :n]), (x[:1, :k].expand(5, -1), g[:5, :n]),
                  (x.view(-1).as_strided((7, k), (8, 1)), g[:7, :n])):
        both(lm, v, wg, wu, bg, bu, gr)
    both(lm, x[:, :k], wg, wg, bg, bg, g[:, :n])  # one weight for both
    one = wg[:1].detach().requires_grad_()  # shared rows: the gradient is their sum
    y = lm.gated_linear(x[:, :k].contiguous(), one.expand(n, -1).contiguous(), wu)
    torch.autograd.grad(y, one, g[:, :n])
    with pytest.raises(ValueError, match="evenly spaced"):
        lm.gated_linear(x.view(4, 6, -1)[:, :5, :k], wg, wu)


def test_gradients_that_are_expanded_or_strided(lm):
    x, wg, wu, bg, bu, g = inputs(12, 40, 48, torch.bfloat16)
    d = Definition(x, wg, wu, bg, bu, "silu")
    x3 = x.view(3, 4, 40).requires_grad_()
    for grad in (torch.ones((), device="cuda", dtype=torch.bfloat16).expand(3, 4, 48),
                 g.view(3, 4, 48).transpose(0, 1).contiguous().transpose(0, 1), g.t().contiguous().t().view(3, 4, 48),
                 g[:1].expand(12, 48).view(3, 4, 48)):
        dx, = torch.autograd.grad(lm.gated_linear(x3, wg, wu, bg, bu), x3, grad)
        d.check_grads(grad, dx)


def test_out(lm):
    x, wg, wu, bg, bu, _ = inputs(20, 64, 300, torch.bfloat16)
    ref = lm.gated_linear(x, wg, wu, bg, bu)
    wide = torch.zeros((20, 320), device="cuda", dtype=torch.bfloat16)
    lm.gated_linear(x, wg, wu, bg, bu, out=wide[:, 7:307])
    assert torch.equal(wide[:, 7:307], ref) and not wide[:, :7].any() and not wide[:, 307:].any()
    with pytest.raises(lm.LogmelError):
        lm.gated_linear(x, wg[:64], wu[:64], out=x)
    with pytest.raises(RuntimeError, match="out goes without gradients"):
        lm.gated_linear(x.detach().requires_grad_(), wg, wu, out=torch.empty_like(ref))


def test_empty(lm):
    for rows, k, n in ((0, 16, 8), (4, 0, 8), (4, 16, 0), (0, 0, 0)):
        x, wg, wu, bg, bu, g = inputs(rows, k, n, torch.float16)
        leaves = [t.requires_grad_() for t in (x, wg, wu, bg, bu)]
        y = lm.gated_linear(*leaves)
        grads = torch.autograd.grad(y, leaves, g)
        Definition(*(t.detach() for t in leaves), "silu").check(y.detach())
        for t, leaf in zip(grads, leaves):
            assert t.shape == leaf.shape
        if rows == 0 or n == 0:
            assert not any(t.any() for t in grads)
        elif k == 0:
            Definition(*(t.detach() for t in leaves), "silu").check_grads(g, None, None, None, grads[3], grads[4])


def test_which_gradients_are_taken(lm):
    ts = inputs(50, 72, 90, torch.float16)
    g = ts[5]
    leaves = [t.requires_grad_() for t in ts[:5]]
    full = torch.autograd.grad(lm.gated_linear(*leaves), leaves, g)
    for i in range(5):
        one = [t.detach().requires_grad_(j == i) for j, t in enumerate(ts[:5])]
        got, = torch.autograd.grad(lm.gated_linear(*one), one[i], g)
        assert torch.equal(got, full[i])
    lm.gated_linear(*leaves).backward(g)
    assert all(torch.equal(t.grad, f) for t, f in zip(leaves, full))


def test_gradients_against_differences(lm):
    """<gradient, v> is the slope of sum(g y) along v: a central difference takes the tolerance of the values on
    either side, and what the definition's own difference is off by."""
    x, wg, wu, bg, bu, g = inputs(6, 40, 30, torch.float16, seed=9)
    vs = [t / 16 for t in inputs(6, 40, 30, torch.float16, seed=10)[:5]]
    leaves = [t.detach().requires_grad_() for t in (x, wg, wu, bg, bu)]
    grads = torch.autograd.grad(lm.gated_linear(*leaves), leaves, g)
    slope = sum((a.double() * v.double()).sum() for a, v in zip(grads, vs))
    ends, ends64, noise, steps = [], [], 0.0, []
    for s in (1, -1):
        p = [t + s * v for t, v in zip((x, wg, wu, bg, bu), vs)]
        steps.append(p)
        d = Definition(*p, "silu")
        ref = d.h * d.b
        ends64.append((g.double() * ref).sum())
        ends.append((g.double() * lm.gated_linear(*p).double()).sum())
        noise += float((g.double().abs() * (d.eh * d.b.abs() + d.h.abs() * d.eb + rounding(ref, torch.float16))).sum())
    moved = [(a.double() - b.double()) / 2 for a, b in zip(*steps)]  # the steps that were taken, rounded
    slope = sum((a.double() * v).sum() for a, v in zip(grads, moved))
    exact = [t.double().requires_grad_() for t in (x, wg, wu, bg, bu)]
    a, b = exact[0] @ exact[1].t() + exact[3], exact[0] @ exact[2].t() + exact[4]
    want = torch.autograd.grad(a * torch.sigmoid(a) * b, exact, g.double())
    off = sum((1.01 * rounding(t, torch.float16) * 8 * v.abs()).sum() for t, v in zip(want, moved))
    want = sum((t * v).sum() for t, v in zip(want, moved))
    bend = abs((ends64[0] - ends64[1]) / 2 - want)
    assert abs((ends[0] - ends[1]) / 2 - slope) <= bend + noise / 2 + off


def test_refusals(lm):
    x, wg, wu, bg, bu, _ = inputs(4, 64, 32, torch.float16)
    for bad in (lambda: lm.gated_linear(x.cpu(), wg, wu), lambda: lm.gated_linear(x.float(), wg, wu),
                lambda: lm.gated_linear(x, wg.bfloat16(), wu), lambda: lm.gated_linear(x, wg, wu[:31]),
                lambda: lm.gated_linear(x, wg[:, :63], wu), lambda: lm.gated_linear(x, wg, None),
                lambda: lm.gated_linear(x, wg, wu, bg[:31]), lambda: lm.gated_linear(x, wg, wu, bg, bu.half()),
                lambda: lm.gated_linear(x, wg, wu, bg.double()), lambda: lm.gated_linear(x, wg, wu, activation="swish"),
                lambda: lm.gated_linear(x, wg, wu.cpu()), lambda: lm.gated_linear(x, wg, wu, out=x),
                lambda: lm.gated_linear(x.t(), wg, wu), lambda: lm.gated_linear(x[0, 0], wg, wu)):
        with pytest.raises(ValueError):
            bad()
    with fwd.dual_level(), pytest.raises(RuntimeError, match="tangent"):
        lm.gated_linear(x, fwd.make_dual(wg, wg), wu)
    x = x.detach().requires_grad_()
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(lm.gated_linear(x, wg, wu).sum(), x, create_graph=True)


def test_repeats_its_bits(lm):
    ts = inputs(1100, 256, 384, torch.bfloat16)
    first, again = both(lm, *ts), both(lm, *ts)
    assert torch.equal(first[0], again[0]) and all(torch.equal(p, q) for p, q in zip(first[1], again[1]))


def test_streams_and_graphs(lm):
    ts = inputs(300, 130, 200, torch.bfloat16)
    g = ts[5]
    leaves = [t.requires_grad_() for t in ts[:5]]
    y = lm.gated_linear(*leaves)
    want = (y.detach(), *torch.autograd.grad(y, leaves, g))
    del y
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.no_grad():
        assert torch.equal(lm.gated_linear(*leaves, stream=side).clone(), want[0])
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = lm.gated_linear(*leaves)
            grads = torch.autograd.grad(y, leaves, g)
            y = y.detach()
        graphs.append((graph, (y, *grads)))
    for _ in range(3):
        for graph, outs in graphs:
            for t in outs:
                t.zero_()
            graph.replay()
        for graph, outs in graphs:
            assert all(torch.equal(p, q) for p, q in zip(outs, want))


def test_no_capture_beside_an_eager_graph_of_the_same_leaf(lm):
    x, wg, wu, *_ = inputs(8, 64, 32, torch.float16)
    wu.requires_grad_()
    alive = lm.gated_linear(x, wg, wu)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="default stream over the same leaf"):
        with torch.cuda.graph(graph):
            lm.gated_linear(x, wg, wu)
    del alive
