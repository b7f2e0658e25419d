"""Tensors of more than 2^31 elements: offsets past 32 bits, checked in the last rows."""
import pytest
import torch

import test_gated_linear as gated
import test_layer_norm as norm
import test_weight4 as weight4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def half(*shape):
    return torch.empty(shape, device="cuda", dtype=torch.float16).normal_()


@pytest.mark.parametrize("rows,width", [(2 ** 21 + 3, 1032), (2 ** 21 + 3, 1031), (2 ** 27 + 5, 24), (131100, 16400)])
def test_layer_norm(lm, rows, width):
    x, g = half(rows, width).requires_grad_(), half(rows, width)
    w, b = (torch.randn(width, device="cuda", requires_grad=True) for _ in range(2))
    y = lm.layer_norm(x, w, b)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), g)
    end = slice(rows - 9, rows)
    d = norm.Definition(x.detach()[end], w.detach(), b.detach(), 1e-5)
    d.check(y.detach()[end])
    d.check_dx(dx[end], g[end])
    sums = [torch.zeros(width, dtype=torch.float64, device="cuda") for _ in range(4)]
    for at in range(0, rows, 2 ** 28 // width):  # of g and of g n, and their magnitudes
        xs, gs = x.detach()[at:at + 2 ** 28 // width].double(), g[at:at + 2 ** 28 // width].double()
        var, mean = torch.var_mean(xs, -1, keepdim=True, correction=0)
        n = gs * (xs - mean) / torch.sqrt(var + 1e-5)
        for s, t in zip(sums, (gs, n, gs.abs(), n.abs())):
            s += t.sum(0)
    # (the bound of a sum over rows, and 2^-17 of a deviation's part in each: see test_layer_norm)
    part = (rows / 64 + 512) * 2.0 ** -24
    assert bool(((db.double() - sums[0]).abs() <= part * sums[2]).all())
    assert bool(((dw.double() - sums[1]).abs() <= part * sums[3] + 2.0 ** -17 * (sums[3] + sums[2])).all())


def test_gated_linear(lm):
    rows, k, n = 270001, 40, 8192
    x, wg, wu, g = half(rows, k), half(n, k) / 6, half(n, k) / 6, half(rows, n)
    bg, bu = (torch.randn(n, device="cuda") for _ in range(2))
    leaves = [t.requires_grad_() for t in (x, wg, wu, bg, bu)]
    y = lm.gated_linear(*leaves)
    grads = [t.detach() for t in torch.autograd.grad(y, leaves, g)]
    leaves, y = [t.detach() for t in leaves], y.detach()
    x, wg, wu, bg, bu = leaves
    end = slice(rows - 33, rows)
    d = gated.Definition(x[end], wg, wu, bg, bu, "silu")
    d.check(y[end])
    d.check_grads(g[end], grads[0][end])
    at = torch.tensor([0, 1, 4095, 8190, 8191], device="cuda")
    d = gated.Definition(x, wg[at], wu[at], bg[at], bu[at], "silu")
    d.check(y[:, at])
    d.check_grads(g[:, at], None, *(t[at] for t in grads[1:]))


@pytest.mark.parametrize("rows,k,n", [(16, 32, 2 ** 27 + 77), (64, 64, 2 ** 25 + 77), (270001, 64, 8200)])
def test_four_bits(lm, rows, k, n):
    q = torch.randint(-8, 8, (n, k), device="cuda", dtype=torch.int8)
    s = torch.rand((n, -(-k // 32)), device="cuda") * 0.05 + 0.01
    w4 = lm.Weight4.pack(q, s, group=32, dtype=torch.float16)
    x = half(rows, k)
    y = lm.linear(x, w4)
    end = slice(n - 301, n)
    some = slice(max(0, rows - 50), rows)
    weight4.check(y[some, end], x[some], weight4.value64(q[end], s[end], 32))
    assert torch.equal(w4.values()[end], (q[end].float() * s[end].repeat_interleave(32, 1)[:, :k]).half())
