"""The scratch memory that the torch side of the decoding operations keeps between calls."""
import ctypes

import pytest
import torch

import test_kv_cache as kv
import test_linear as lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def test_a_copied_operand_goes_with_its_call(lm):
    """Rows off 16-byte boundaries are copied first; the copy does not stay."""
    lm.linear(torch.ones((8, 64), device="cuda").half(), torch.ones((8, 64), device="cuda").half())
    x, w, _, _ = lin.make((8, 1023), 50001, torch.float16, bias=False, residual=False)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = lm.linear(x, w)
    kept = torch.cuda.memory_allocated() - before - y.numel() * 2
    lin.check(y, x, w)  # (this takes scratch of its own)
    assert kept < 1 << 20
    before = torch.cuda.memory_allocated()
    lm.linear(x, w)
    assert torch.cuda.memory_allocated() - before < 1 << 20


def test_copied_operands_in_a_graph(lm):
    a = [lin.make((m, 333), n, torch.bfloat16, seed=m) for m, n in ((7, 900), (300, 257))]
    want = [lm.linear(x, w, b, residual=r) for x, w, b, r in a]
    outs = [torch.empty_like(y) for y in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for (x, w, b, r), o in zip(a, outs):
            lm.linear(x, w, b, residual=r, out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        g.replay()
        for o, y in zip(outs, want):
            assert torch.equal(o, y)


def test_streams_that_come_and_go(lm):
    """Many short-lived streams, whose handles come back: results are right and the scratch does not pile up."""
    rt = ctypes.CDLL("libcudart.so.13")
    c = kv.filled(lm, 2, 3000, 2, 64, 32, torch.float16, seed=3)
    c.lens.fill_(2990)
    r = kv.gen(2)
    q, logits, scores = r(2, 1, 2, 64).half(), r(2, 4, 5000), r(2, 4)
    want, step = c.attend(0, q), lm.beam_step(logits, scores)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(200):
        h = ctypes.c_void_p()
        assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0
        s = torch.cuda.ExternalStream(h.value)
        got, other = c.attend(0, q, stream=s), lm.beam_step(logits, scores, stream=s)
        s.synchronize()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(other[:4], step[:4]))
        del got, other
        assert rt.cudaStreamDestroy(h) == 0
    assert torch.cuda.memory_allocated() - before < 160 << 18  # 128 workspaces of up to 256 KB
    assert torch.equal(c.attend(0, q), want)
