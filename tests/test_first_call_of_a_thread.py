"""Calls that are a host thread's first to CUDA.

Tensor maps are made by the CUDA driver, which wants the thread to have a context; CUDA's runtime, which the library uses
otherwise, gives a thread one at its first call.  The thread of torch's engine that runs backward passes is such a
thread, and a program's own threads are.  The operands here need no copies, which would be launches before the maps.
"""
import pathlib
import struct
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = pathlib.Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def in_a_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("m", [5, 200, 3000])
def test_c_calls(lm, m):
    from log_mel_spectrogram_gb300 import _native
    lib, n, k = _native.lib(), 256, 128
    x, w, wu = (torch.randn(s, device="cuda").half() / 8 for s in ((m, k), (n, k), (n, k)))
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    q = lm.quantize_weight(w)
    out, out4, outg = (torch.zeros((m, n), device="cuda", dtype=torch.float16) for _ in range(3))
    stream = torch.cuda.current_stream().cuda_stream

    def args(weight, to):
        return struct.pack("5P9q4ifi", x.data_ptr(), weight, 0, 0, to.data_ptr(), 1, m, k, n, 0, k, k, 0, n, 2, 2, 2, 0,
                           1.0, 0)
    w4 = struct.pack("2P2q2i", q.packed.data_ptr(), q.scale.data_ptr(), n, k, q.group, 0)
    gate = struct.pack("6P7q4i", x.data_ptr(), w.data_ptr(), wu.data_ptr(), 0, 0, outg.data_ptr(), m, k, n, k, k, k, n, 2,
                       0, 4, 0)
    linear, linear4, gated = args(w.data_ptr(), out), args(0, out4), gate
    torch.cuda.synchronize()
    assert in_a_thread(lambda: lib.lm_linear(linear, ws.data_ptr(), ws.numel(), stream)) == 0
    assert in_a_thread(lambda: lib.lm_linear4(linear4, w4, ws.data_ptr(), ws.numel(), stream)) == 0
    assert in_a_thread(lambda: lib.lm_gated_linear(gated, ws.data_ptr(), ws.numel(), stream)) == 0
    assert torch.equal(out, lm.linear(x, w)) and torch.equal(out4, lm.linear(x, q))
    assert torch.equal(outg, lm.gated_linear(x, w, wu))


BACKWARD = """
import torch, log_mel_spectrogram_gb300 as lm
x, wg, wu = (torch.randn(s, device="cuda").half().requires_grad_() for s in ((4, 64), (16, 64), (16, 64)))
g = torch.randn((4, 16), device="cuda").half()
y = lm.gated_linear(x, wg, wu)
del [torch.empty(1 << 10, device="cuda") for _ in range(32)][:]  # so that memory is at hand without a call to CUDA
grads = torch.autograd.grad(y, (x, wg, wu), g, retain_graph=True)
again = torch.autograd.grad(y, (x, wg, wu), g)
assert all(torch.equal(a, b) and a.any() for a, b in zip(grads, again))
"""


def test_a_backward_pass_that_comes_first(lm):
    r = subprocess.run([sys.executable, "-c", BACKWARD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
