"""A wait of the cache's attention that runs out ends its CTA cleanly.

lm_debug_kv_attend_withhold keeps one CTA's first tile of tokens from counting as complete and gives
waits 2 ms.  The call completes, the workspace's error word says so, every output that the CTA does not
compute is what the regular call gives, and so is the next regular call.  Nothing here faults, traps or
hangs the GPU: the only failure is a wait that nothing completes.
"""
import ctypes
import struct
import time

import pytest
import torch

import test_kv_cache as kv

pytestmark = pytest.mark.gpu

MBAR_TIMEOUT_BIT = 1
LM_ERR_DEVICE_FAULT = 6


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def lib():
    from log_mel_spectrogram_gb300 import _native
    return _native.lib()


def attend(c, q, ws, withheld=None, wait_ns=2_000_000):
    """lm_kv_attend of layer 0, causal, through the C ABI."""
    rows, t, heads, dim = q.shape
    out = torch.full_like(q, 7.0)
    args = (c._args, 0, q.data_ptr(), struct.pack("3q", *q.stride()[:3]), t, heads, None, t, 1, dim ** -0.5,
            c._code, out.data_ptr(), ws.data_ptr(), ws.numel())
    stream = torch.cuda.current_stream().cuda_stream
    if withheld is None:
        assert lib().lm_kv_attend(*args, stream) == 0
    else:
        assert lib().lm_debug_kv_attend_withhold(*args, withheld, wait_ns, stream) == 0
    return out


def workspace(c, q):
    n = ctypes.c_size_t()
    assert lib().lm_kv_attend_workspace_size(c._args, q.shape[1], q.shape[2], ctypes.byref(n)) == 0
    return torch.zeros(n.value, dtype=torch.uint8, device="cuda")


def error(ws):
    v = ctypes.c_uint32()
    rc = lib().lm_workspace_error(ws.data_ptr(), ws.numel(), ctypes.byref(v), torch.cuda.current_stream().cuda_stream)
    assert rc == (LM_ERR_DEVICE_FAULT if v.value else 0)
    return v.value


# Of CTA 0's work: its row 0, heads, and queries (the last tile of them).
@pytest.mark.parametrize("rows,heads,dim,tokens,t,own_heads,own_queries", [
    (3, 2, 64, 300, 1, 1, 1), (3, 2, 128, 300, 12, 1, 12), (4, 3, 32, 200, 2, 1, 2),      # a head's tokens over the warps
    (160, 5, 64, 70, 1, 4, 1), (130, 7, 128, 100, 1, 4, 1),                                # a warp a head
    (48, 10, 64, 160, 100, 1, 36), (30, 12, 128, 150, 130, 1, 2), (60, 16, 32, 300, 64, 1, 64)])  # tiles of 64 queries
def test_a_withheld_tile_ends_its_cta(lm, rows, heads, dim, tokens, t, own_heads, own_queries):
    c = kv.filled(lm, rows, tokens, heads, dim, 32, torch.float16, seed=rows)
    c.lens.fill_(tokens - t)
    q = kv.gen(dim)(rows, t, heads, dim).half()
    ws = workspace(c, q)
    want = attend(c, q, ws)
    assert error(ws) == 0
    t0 = time.perf_counter()
    got = attend(c, q, ws, withheld=0)
    assert error(ws) & MBAR_TIMEOUT_BIT
    assert time.perf_counter() - t0 < 1.5  # gave up long before the regular limit
    assert torch.equal(got[1:], want[1:]) and torch.equal(got[0, :, own_heads:], want[0, :, own_heads:])
    assert torch.equal(got[0, :t - own_queries], want[0, :t - own_queries])
    assert (got[0, t - own_queries:, 0] == 7).all()  # not written
    ws[:4] = 0
    assert torch.equal(attend(c, q, ws), want) and error(ws) == 0


@pytest.mark.parametrize("withheld", [0, 1, 2, 5])
@pytest.mark.parametrize("rows,heads,dim,tokens,t", [(2, 2, 64, 9000, 1), (1, 2, 128, 20000, 3), (3, 2, 32, 5000, 16)])
def test_a_part_that_gave_up_leaves_no_count(lm, withheld, rows, heads, dim, tokens, t):
    """CTA x of a row is part x / heads of head x % heads.  The unit of the part that gave up is not joined, and the
    next call finds the workspace as the first one did."""
    c = kv.filled(lm, rows, tokens, heads, dim, 64, torch.float16, seed=rows)
    c.lens.fill_(tokens - t)
    q = kv.gen(dim)(rows, t, heads, dim).half()
    ws = workspace(c, q)
    want = attend(c, q, ws)
    for _ in range(2):
        got = attend(c, q, ws, withheld=withheld)
        assert error(ws) & MBAR_TIMEOUT_BIT
        head = withheld % heads
        assert torch.equal(got[1:], want[1:]) and torch.equal(got[0, :, 1 - head], want[0, :, 1 - head])
        assert (got[0, :, head] == 7).all()
        ws[:4] = 0
        assert torch.equal(attend(c, q, ws), want) and error(ws) == 0


def test_refusals(lm):
    c = kv.filled(lm, 1, 64, 1, 64, 32, torch.float16)
    q = torch.zeros((1, 1, 1, 64), device="cuda", dtype=torch.float16)
    ws = workspace(c, q)
    args = (c._args, 0, q.data_ptr(), struct.pack("3q", 64, 64, 64), 1, 1, None, 1, 1, 1.0, c._code, q.data_ptr(),
            ws.data_ptr(), ws.numel())
    for cta, ns in ((-1, 10 ** 6), (0, 10 ** 4), (0, 3 * 10 ** 9)):
        assert lib().lm_debug_kv_attend_withhold(*args, cta, ns, None) == 1
