"""A backward pass that is captured while a graph of the default stream lives behind its inputs.

torch's engine would make the default stream wait for the captured one, which ends the process: the calls refuse it
first.  Each case has a process of its own.
"""
import pathlib
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = pathlib.Path(__file__).resolve().parents[1]

START = """
import torch, log_mel_spectrogram_gb300 as lm
torch.manual_seed(0)
x = torch.randn((8, 64), device="cuda").half()
w = torch.randn((32, 64), device="cuda").requires_grad_()  # f32, cast by the layer
s = torch.ones(64, device="cuda").requires_grad_()
def layer():
    return lm.gated_linear(lm.layer_norm(x, s * 2), w.half(), w.half())
def refused(f):
    try:
        f()
    except RuntimeError as e:
        assert "default stream over the same leaf" in str(e), e
    else:
        raise AssertionError("not refused")
"""

# The leaves are cast, or come through another operation: no input is one.
BEHIND = """
alive = layer()
def captured():
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        torch.autograd.grad(layer().sum(), WANTED)
refused(captured)
del alive
"""
# Afterwards the same layer is captured, and gives what it gives eagerly.
AFTER = """
side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    want = torch.autograd.grad(layer().sum(), (w, s))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = torch.autograd.grad(layer().sum(), (w, s))
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.any() for a, b in zip(got, want))
"""
# An input that is not wanted may have come from such a graph.
UNWANTED = """
h = x.float().requires_grad_() * 2  # of the default stream, and not taken part in
with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
    got, = torch.autograd.grad(lm.layer_norm(h, s).sum(), s)
graph.replay()
torch.cuda.synchronize()
want, = torch.autograd.grad(lm.layer_norm(h, s).sum(), s)
assert torch.equal(got, want)
"""


@pytest.mark.parametrize("code", [BEHIND.replace("WANTED", "(w, s)") + AFTER, BEHIND.replace("WANTED", "w"),
                                  BEHIND.replace("WANTED", "s"), AFTER, UNWANTED],
                         ids=["all", "weight", "norm", "after", "unwanted"])
def test_captured(code):
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", START + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
