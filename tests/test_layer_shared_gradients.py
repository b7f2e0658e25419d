"""Gradients of one row that serves for all: the sum of the rows' gradients.

The rows' own gradients are the operators' (checked here against the definition in 64 bits, with the bounds of their
tests); torch adds them up in 32 bits, off by at most (rows + 8) 2^-24 of the sum of magnitudes, and rounds once.
"""
import pytest
import torch

import test_gated_linear as gated
import test_layer_norm as norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def is_sum_of(got, rows):
    ref, mag = rows.double().sum(0), rows.double().abs().sum(0)
    gap = (got.double().reshape(ref.shape) - ref).abs()
    tol = (rows.shape[0] + 8) * 2.0 ** -24 * mag
    assert bool((gap <= tol + norm.rounding(ref.abs() + tol, got.dtype)).all())
    assert bool((ref.abs() > 4 * norm.HALF_STEP[got.dtype] * mag).any())  # (something is left to be seen)


@pytest.mark.parametrize("dtype", norm.TYPES)
@pytest.mark.parametrize("rows,width", [(6, 64), (6, 1023), (40, 1024), (3, 9000)])
def test_norm_of_one_row(lm, dtype, rows, width):
    x, w, b, g = norm.inputs(rows, width, dtype, torch.float32, seed=width)
    one = x[:1].detach().requires_grad_()
    each = x[:1].detach().expand(rows, -1).requires_grad_()
    got, = torch.autograd.grad(lm.layer_norm(one.expand(rows, -1), w, b), one, g)
    dx, = torch.autograd.grad(lm.layer_norm(each, w, b), each, g)
    norm.Definition(each.detach(), w, b, 1e-5).check_dx(dx, g)
    is_sum_of(got, dx)


@pytest.mark.parametrize("dtype", gated.TYPES)
@pytest.mark.parametrize("rows,k,n", [(12, 64, 50), (70, 72, 129), (5, 33, 16)])
def test_gated_layer_of_one_row(lm, dtype, rows, k, n):
    x, wg, wu, bg, bu, g = gated.inputs(rows, k, n, dtype, seed=n)
    for which in range(3):  # x, w_gate, w_up
        leaves = [t.detach().clone() for t in (x, wg, wu, bg, bu)]
        count = (rows, n, n)[which]
        one = leaves[which][:1].clone().requires_grad_()
        each = one.detach().expand(count, -1).contiguous().requires_grad_()
        leaves[which] = one.expand(count, -1).contiguous()
        got, = torch.autograd.grad(lm.gated_linear(*leaves), one, g)
        leaves[which] = each
        d, = torch.autograd.grad(lm.gated_linear(*leaves), each, g)
        ref = gated.Definition(*(t.detach() for t in leaves), "silu")
        ref.check_grads(g, **{("dx", "dwg", "dwu")[which]: d})
        is_sum_of(got, d)
    # Rows that are one by their stride alone are read in place.
    one = x[:1].detach().requires_grad_()
    each = one.detach().expand(rows, -1).requires_grad_()
    got, = torch.autograd.grad(lm.gated_linear(one.expand(rows, -1), wg, wu, bg, bu), one, g)
    d, = torch.autograd.grad(lm.gated_linear(each, wg, wu, bg, bu), each, g)
    is_sum_of(got, d)
