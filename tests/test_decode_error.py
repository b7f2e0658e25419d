"""What a wait that ran out inside linear or the cache's attention leaves behind: a bit that
decode_error() returns, whoever holds the workspace, and a workspace that the next call can use.

lm_debug_linear_withhold keeps one CTA's first tile of operands from counting as complete and gives waits
2 ms.  Nothing here faults, traps or hangs the GPU: the only failure is a wait that nothing completes.
"""
import ctypes
import struct
import time

import pytest
import torch

import test_kv_cache as kv
import test_kv_waits as waits

pytestmark = pytest.mark.gpu

MBAR_TIMEOUT_BIT = 1


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def linear(x, w, ws, withheld=None, wait_ns=2_000_000):
    (m, k), n = x.shape, w.shape[0]
    out = torch.full((m, n), 7.0, device="cuda", dtype=x.dtype)
    args = struct.pack("5P9q4ifi", x.data_ptr(), w.data_ptr(), 0, 0, out.data_ptr(), 1, m, k, n, 0, k, k, 0, n, 2, 2, 2, 0,
                       1.0, 0)
    stream = torch.cuda.current_stream().cuda_stream
    if withheld is None:
        assert waits.lib().lm_linear(args, ws.data_ptr(), ws.numel(), stream) == 0
    else:
        assert waits.lib().lm_debug_linear_withhold(args, ws.data_ptr(), ws.numel(), withheld, wait_ns, stream) == 0
    return out


@pytest.mark.parametrize("m,k,n,parts_of_k", [(3000, 1024, 1024, False), (8192, 512, 2048, False), (600, 200, 700, False),
                                              (5, 1024, 1024, True), (40, 4096, 256, True)])
@pytest.mark.parametrize("withheld", [0, 1, 7])
def test_linear_reports_and_recovers(lm, m, k, n, parts_of_k, withheld):
    g = torch.Generator(device="cuda").manual_seed(m)
    x, w = (torch.randn(s, generator=g, device="cuda").half() for s in ((m, k), (n, k)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want = linear(x, w, ws)
    assert lm.decode_error() == 0 and waits.error(ws) == 0
    t0 = time.perf_counter()
    got = linear(x, w, ws, withheld=withheld)
    ran_out = waits.error(ws)
    assert time.perf_counter() - t0 < 1.5  # gave up long before the regular limit
    assert lm.decode_error(clear=False) == lm.decode_error() == ran_out
    assert lm.decode_error() == 0
    if withheld == 0:
        assert ran_out & MBAR_TIMEOUT_BIT  # (of a pair, CTA 1's copies count on CTA 0's barriers)
    if not parts_of_k:
        assert ((got == want) | (got == 7)).all()  # right, or not written
    ws.zero_()
    assert torch.equal(linear(x, w, ws), want) and lm.decode_error() == 0 and waits.error(ws) == 0


@pytest.mark.parametrize("rows,heads,tokens,t", [(3, 2, 300, 1), (2, 2, 9000, 1), (160, 5, 70, 1), (48, 10, 160, 100)])
def test_attention_reports(lm, rows, heads, tokens, t):
    c = kv.filled(lm, rows, tokens, heads, 64, 32, torch.float16, seed=rows)
    c.lens.fill_(tokens - t)
    q = kv.gen(t)(rows, t, heads, 64).half()
    ws = waits.workspace(c, q)
    want = waits.attend(c, q, ws)
    assert lm.decode_error() == 0
    waits.attend(c, q, ws, withheld=0)
    assert lm.decode_error() & MBAR_TIMEOUT_BIT and lm.decode_error() == 0
    assert torch.equal(c.attend(0, q), want) and lm.decode_error() == 0


def test_a_wait_that_runs_out_is_waited_for_once(lm):
    """A CTA that gives up waits for all of its copies in flight, together no longer than one limit."""
    x, w = (torch.ones(s, device="cuda").half() for s in ((5, 8192), (256, 8192)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    linear(x, w, ws)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    linear(x, w, ws, withheld=0, wait_ns=100_000_000)
    b.record()
    torch.cuda.synchronize()
    assert lm.decode_error() & MBAR_TIMEOUT_BIT
    assert 100 <= a.elapsed_time(b) < 350  # the wait, the copies' and its neighbours'


def test_refusals(lm):
    v = ctypes.c_uint32()
    assert waits.lib().lm_decode_error(None, 0, None) == 1
    assert waits.lib().lm_decode_error(ctypes.byref(v), 0, None) == 0 and v.value == 0
    args = struct.pack("5P9q4ifi", *[1 << 20] * 2, 0, 0, 1 << 21, 1, 1, 8, 8, 0, 8, 8, 0, 8, 2, 2, 2, 0, 1.0, 0)
    for cta, ns in ((-1, 10 ** 6), (2 ** 31, 10 ** 6), (0, 10 ** 4), (0, 3 * 10 ** 9)):
        assert waits.lib().lm_debug_linear_withhold(args, 1 << 20, 256, cta, ns, None) == 1
