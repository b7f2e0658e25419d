"""The operators of a layer in a run, each result held against the definition of its own step.

Every operator gets what the one before gave, called or captured, and its result is bounded as in its own tests, from
the inputs that it had: a second rounding or a wrong tail shows, where a bound on the whole run would hide it.
"""
import math

import pytest
import torch

import test_gated_linear as gated
import test_layer_norm as norm
import test_linear as linear
import test_weight4 as weight4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def make(dtype, width, inner, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dense = lambda n, k: (r(n, k) / math.sqrt(k)).to(dtype)  # noqa: E731
    return r, 1 + 0.1 * r(width), 0.1 * r(width), dense(inner, width), dense(inner, width), dense(width, inner)


def run(step, captured):
    """The step's results: of a call, or of a graph's second replay."""
    if not captured:
        return step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    for t in got:
        t.detach().zero_()
    graph.replay()
    return got


@pytest.mark.parametrize("dtype", gated.TYPES)
@pytest.mark.parametrize("rows", [1, 5, 16, 17, 160, 900])
@pytest.mark.parametrize("captured", [False, True])
def test_serving(lm, dtype, rows, captured):
    """norm -> 4-bit projection -> norm -> gated block -> 4-bit projection with a residual."""
    r, w, b, gate, up, down = make(dtype, 192, 520)
    x = r(rows, 192).to(dtype)
    out, down = lm.quantize_weight((r(192, 192) / 14).to(dtype), 32), lm.quantize_weight(down, 64)

    def step():
        n1 = lm.layer_norm(x, w, b)
        y = lm.linear(n1, out, residual=x)
        n2 = lm.layer_norm(y, w, b)
        h = lm.gated_linear(n2, gate, up)
        return n1, y, n2, h, lm.linear(h, down, residual=y)
    with torch.no_grad():
        n1, y, n2, h, z = run(step, captured)
    norm.Definition(x, w, b, 1e-5).check(n1)
    weight4.check(y, n1, out.values(torch.float32).double(), residual=x)
    norm.Definition(y, w, b, 1e-5).check(n2)
    gated.Definition(n2, gate, up, None, None, "silu").check(h)
    weight4.check(z, h, down.values(torch.float32).double(), residual=y)


@pytest.mark.parametrize("dtype", gated.TYPES)
@pytest.mark.parametrize("rows", [3, 210, 1300])
@pytest.mark.parametrize("captured", [False, True])
def test_training(lm, dtype, rows, captured):
    """norm -> gated block with biases, and all gradients of both."""
    width, inner = 192, 520
    r, w, b, gate, up, _ = make(dtype, width, inner, seed=1)
    x, g = r(rows, width).to(dtype), r(rows, inner).to(dtype)
    biases = [0.2 * r(inner), 0.2 * r(inner)]
    leaves = [t.detach().clone().requires_grad_() for t in (x, w, b, gate, up, *biases)]

    def step():
        x, w, b, gate, up, bg, bu = leaves
        n = lm.layer_norm(x, w, b)
        h = lm.gated_linear(n, gate, up, bg, bu)
        return (n.detach(), h.detach(), *torch.autograd.grad(h, [n, *leaves], g))
    n, h, dn, dx, dw, db, dgate, dup, dbg, dbu = run(step, captured)
    first = norm.Definition(x, w, b, 1e-5)
    first.check(n)
    second = gated.Definition(n, gate, up, *biases, "silu")
    second.check(h)
    second.check_grads(g, dn, dgate, dup, dbg, dbu)
    first.check_dx(dx, dn)
    first.check_sums(dw, db, dn)


@pytest.mark.parametrize("rows", [5, 300])
def test_other_layers_between(lm, rows):
    """linear and the 4-bit one in turn with the norm, on one stream and its kept scratch; operands off 16-byte boundaries."""
    dtype, width = torch.float16, 131
    r, w, b, *_ = make(dtype, width, 40, seed=2)
    x, dense = r(rows, width).to(dtype), (r(width, width) / 11).to(dtype)
    four = lm.quantize_weight(dense, 32)
    for _ in range(3):
        n = lm.layer_norm(x, w, b)
        y = lm.linear(n, dense)
        z = lm.linear(y, four, residual=x)
        norm.Definition(x, w, b, 1e-5).check(n)
        linear.check(y, n, dense)
        weight4.check(z, y, four.values(torch.float32).double(), residual=x)
        x = z
