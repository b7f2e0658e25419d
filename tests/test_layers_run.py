"""The operators of a layer together, as a model calls them, against the same steps in 64 bits.

Each operator's own error is bounded in its tests.  Here every intermediate result is rounded to bf16 by at most
2^-8 of itself on both sides' way, so that runs of them are compared in the norm: each of the five or six roundings
adds at most 2^-8 of its operand, and a layer's steps amplify none by more than about 2 (weights have unit rows):
an error of 16 * 2^-8 of the result's norm would take all of them at their bound and in one direction.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def close(got, ref):
    assert got.shape == ref.shape
    assert float((got.double() - ref).norm()) <= 16 * 2.0 ** -8 * float(ref.norm())


def norm64(x, w, b):
    var, mean = torch.var_mean(x, -1, keepdim=True, correction=0)
    return (x - mean) / torch.sqrt(var + 1e-5) * w + b


def weights(width, inner, dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    dense = lambda n, k: (r(n, k) / math.sqrt(k)).to(dtype)  # noqa: E731
    return r, dict(w=1 + 0.1 * r(width), b=0.1 * r(width), gate=dense(inner, width), up=dense(inner, width),
                   down=dense(width, inner), qkv=dense(3 * width, width), out=dense(width, width))


@pytest.mark.parametrize("rows", [5, 160])
@pytest.mark.parametrize("captured", [False, True])
def test_a_decoding_step(lm, rows, captured):
    """norm -> projections in 4 bits -> cache -> attention -> norm -> gated block -> projection in 4 bits."""
    width, heads, inner, dt = 256, 4, 640, torch.bfloat16
    r, p = weights(width, inner, dt)
    x = r(rows, 1, width).to(dt)
    qkv4, out4, down4 = (lm.quantize_weight(p[k]) for k in ("qkv", "out", "down"))
    cache = lm.KvCache(rows, 64, heads, width // heads, dtype=dt)

    def step():
        q, k, v = lm.linear(lm.layer_norm(x, p["w"], p["b"]), qkv4).unflatten(-1, (3, heads, -1)).unbind(2)
        cache.append(0, k, v)
        y = lm.linear(cache.attend(0, q).flatten(2), out4, residual=x)
        return lm.linear(lm.gated_linear(lm.layer_norm(y, p["w"], p["b"]), p["gate"], p["up"]), down4, residual=y)
    if captured:
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step()
        y.zero_()
        graph.replay()
    else:
        y = step()
    xd = x.double()
    v = (norm64(xd, p["w"].double(), p["b"].double()) @ qkv4.values(torch.float32).double().t())[..., 2 * width:]
    z = v @ out4.values(torch.float32).double().t() + xd  # one token: attention is its value
    n = norm64(z, p["w"].double(), p["b"].double())
    a = n @ p["gate"].double().t()
    h = a * torch.sigmoid(a) * (n @ p["up"].double().t())
    close(y, h @ down4.values(torch.float32).double().t() + z)


@pytest.mark.parametrize("captured", [False, True])
def test_a_training_step_of_a_feed_forward_layer(lm, captured):
    """norm -> gated block -> projection, and the gradients of all weights and of x."""
    width, inner, dt = 192, 520, torch.bfloat16
    r, p = weights(width, inner, dt, seed=1)
    x, g = r(3, 70, width).to(dt), r(3, 70, width).to(dt)
    names = ("w", "b", "gate", "up", "down")
    leaves = [t.clone().requires_grad_() for t in (x, *(p[k] for k in names))]

    def step():
        x, w, b, gate, up, down = leaves
        y = x + lm.gated_linear(lm.layer_norm(x, w, b), gate, up) @ down.t()
        return (y.detach(), *torch.autograd.grad(y, leaves, g))
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for t in got:
            t.zero_()
        graph.replay()
    else:
        got = step()
    exact = [t.detach().double().requires_grad_() for t in leaves]
    xd, w, b, gate, up, down = exact
    n = norm64(xd, w, b)
    a = n @ gate.t()
    y = xd + (a * torch.sigmoid(a) * (n @ up.t())) @ down.t()
    for t, ref in zip(got, (y.detach(), *torch.autograd.grad(y, exact, g.double()))):
        close(t, ref)
