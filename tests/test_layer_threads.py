"""Backward passes beside calls of another host thread on the same stream.

A backward pass runs on a thread of torch's engine, which does not hold the interpreter's lock: between its launches
another Python thread can launch whole calls on the stream.  Sums over rows, copies of operands and the projections'
gradients lie in scratch from one launch to the next, so that scratch has to be the pass's own.
"""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def rand(seed, *shapes):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=gen, device="cuda") for s in shapes]


def norm(lm, rows=5, width=1024):
    x, w, b, g = rand(1, (rows, width), (width,), (width,), (rows, width))
    leaves = [t.requires_grad_() for t in (x, w, b)]
    return lambda: (lm.layer_norm(*leaves), leaves, g)


def gated(lm, rows=6, k=67, n=70):
    """(k off 16-byte boundaries: the operands are copied, too)"""
    x, wg, wu, bg, bu, g = rand(2, (rows, k), (n, k), (n, k), (n,), (n,), (rows, n))
    leaves = [t.detach().requires_grad_() for t in (x.half(), wg.half() / 8, wu.half() / 8, bg, bu)]
    return lambda: (lm.gated_linear(*leaves), leaves, g.half())


def gradients(forward):
    y, leaves, g = forward()
    return [y.detach(), *torch.autograd.grad(y, leaves, g)]


OPERATORS = {"norm": norm, "gated": gated}


@pytest.mark.parametrize("name", OPERATORS)
def test_a_backward_pass_keeps_no_scratch(lm, name):
    forward = OPERATORS[name](lm)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):  # a stream that has no scratch yet
        y, leaves, g = forward()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        grads = torch.autograd.grad(y, leaves, g, retain_graph=True)
        torch.cuda.synchronize()
        del grads
        assert torch.cuda.memory_allocated() == before


@pytest.mark.parametrize("name", OPERATORS)
def test_beside_another_threads_calls(lm, name):
    forward = OPERATORS[name](lm)
    x, w, wg, wu = (t.half() for t in rand(3, (9, 65), (33, 65), (40, 65), (40, 65)))
    q = lm.quantize_weight(w)
    calls = (lambda: lm.linear(x, w), lambda: lm.linear(x, q), lambda: lm.gated_linear(x, wg, wu))
    want, others = gradients(forward), [c() for c in calls]
    torch.cuda.synchronize()
    stop, wrong = threading.Event(), []

    def other():
        try:
            i = 0
            while not stop.is_set():
                got = [calls[(i + j) % 3]() for j in range(3)]
                if i % 16 == 0 and not all(torch.equal(t, others[(i + j) % 3]) for j, t in enumerate(got)):
                    wrong.append(i)
                i += 1
        except Exception as e:  # noqa: BLE001 (a thread's own is not seen otherwise)
            wrong.append(e)

    thread = threading.Thread(target=other)
    thread.start()
    try:
        off = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(600):
            for got, ref in zip(gradients(forward), want):
                off += (got != ref).sum()
    finally:
        stop.set()
        thread.join()
    assert int(off) == 0 and not wrong
