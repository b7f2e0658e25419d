"""Waits that run out inside the gated layer's kernels and linear's with weights in 4 bits: a bit that
decode_error() returns and that the workspace holds, and a workspace that the next call can use.

lm_debug_*_withhold keeps one CTA's first tile of operands from counting as complete and gives waits 2 ms.  Nothing
here faults, traps or hangs the GPU: the only failure is a wait that nothing completes.
"""
import ctypes
import struct
import time

import pytest
import torch

import test_kv_waits as waits

pytestmark = pytest.mark.gpu

MBAR_TIMEOUT_BIT = 1


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def recovers(lm, call, ws, withheld, shared):
    """call(withheld or None) -> outputs, filled with 7 before."""
    lm.decode_error()  # what other tests have left
    want = call(None)
    assert lm.decode_error() == 0 and waits.error(ws) == 0
    t0 = time.perf_counter()
    got = call(withheld)
    ran_out = waits.error(ws)
    assert time.perf_counter() - t0 < 1.5  # gave up long before the regular limit
    assert lm.decode_error(clear=False) == lm.decode_error() == ran_out
    assert lm.decode_error() == 0
    if withheld == 0:
        assert ran_out & MBAR_TIMEOUT_BIT
    if not shared:
        assert ((got[0] == want[0]) | (got[0] == 7)).all()  # right, or not written
    ws.zero_()
    for a, b in zip(call(None), want):
        assert torch.equal(a, b)
    assert lm.decode_error() == 0 and waits.error(ws) == 0


# (a tile a CTA, pairs, k shared out over a cluster)
@pytest.mark.parametrize("m,k,n,shared", [(700, 200, 900, False), (6000, 512, 2048, False), (5, 1024, 1024, True)])
@pytest.mark.parametrize("withheld", [0, 1])
def test_gated_linear(lm, m, k, n, shared, withheld):
    g = torch.Generator(device="cuda").manual_seed(m)
    x, wg, wu = (torch.randn(s, generator=g, device="cuda").half() / 8 for s in ((m, k), (n, k), (n, k)))
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")

    def call(w):
        out = torch.full((m, n), 7.0, device="cuda", dtype=torch.float16)
        args = struct.pack("6P7q4i", x.data_ptr(), wg.data_ptr(), wu.data_ptr(), 0, 0, out.data_ptr(), m, k, n, k, k, k, n, 2,
                           0, 4, 0)
        stream = torch.cuda.current_stream().cuda_stream
        rc = (waits.lib().lm_gated_linear(args, ws.data_ptr(), ws.numel(), stream) if w is None else
              waits.lib().lm_debug_gated_linear_withhold(args, ws.data_ptr(), ws.numel(), w, 2_000_000, stream))
        assert rc == 0
        return [out]
    recovers(lm, call, ws, withheld, shared)


@pytest.mark.parametrize("m,k,n", [(700, 200, 904), (3000, 512, 2048), (5, 1024, 1024)])
@pytest.mark.parametrize("withheld", [0, 1])
def test_gated_linear_backward(lm, m, k, n, withheld):
    g = torch.Generator(device="cuda").manual_seed(m)
    x, wg, wu, go = (torch.randn(s, generator=g, device="cuda").half() / 8 for s in ((m, k), (n, k), (n, k), (m, n)))

    def args(outs):
        return struct.pack("6P7q4i6Pq", x.data_ptr(), wg.data_ptr(), wu.data_ptr(), 0, 0, 0, m, k, n, k, k, k, 0, 2, 0, 4, 0,
                           go.data_ptr(), *(o.data_ptr() for o in outs), 0, 0, n)
    shapes = ((m, k), (n, k), (n, k))
    need = ctypes.c_size_t()
    none = [torch.empty(s, device="cuda", dtype=torch.float16) for s in shapes]
    assert waits.lib().lm_gated_linear_backward_workspace_size(args(none), ctypes.byref(need)) == 0
    ws = torch.zeros(need.value, dtype=torch.uint8, device="cuda")

    def call(w):
        outs = [torch.full(s, 7.0, device="cuda", dtype=torch.float16) for s in shapes]
        stream = torch.cuda.current_stream().cuda_stream
        f = waits.lib().lm_gated_linear_backward if w is None else waits.lib().lm_debug_gated_linear_backward_withhold
        more = () if w is None else (w, 2_000_000)
        assert f(args(outs), ws.data_ptr(), ws.numel(), *more, stream) == 0
        return outs
    recovers(lm, call, ws, withheld, True)


@pytest.mark.parametrize("m,k,n,group,shared", [(90, 200, 900, 64, True), (200, 2048, 300, 32, True),
                                                (60, 300, 25000, 128, False), (256, 640, 20001, 32, False)])
@pytest.mark.parametrize("withheld", [0, 1])
def test_linear4(lm, m, k, n, group, shared, withheld):
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randn((m, k), generator=g, device="cuda").half()
    w4 = lm.quantize_weight(torch.randn((n, k), generator=g, device="cuda").half(), group)
    weight = struct.pack("2P2q2i", w4.packed.data_ptr(), w4.scale.data_ptr(), n, k, group, 0)
    ws = torch.zeros(1 << 18, dtype=torch.uint8, device="cuda")

    def call(w):
        out = torch.full((m, n), 7.0, device="cuda", dtype=torch.float16)
        args = struct.pack("5P9q4ifi", x.data_ptr(), 0, 0, 0, out.data_ptr(), 1, m, k, n, 0, k, 0, 0, n, 2, 2, 2, 0, 1.0, 0)
        stream = torch.cuda.current_stream().cuda_stream
        rc = (waits.lib().lm_linear4(args, weight, ws.data_ptr(), ws.numel(), stream) if w is None else
              waits.lib().lm_debug_linear4_withhold(args, weight, ws.data_ptr(), ws.numel(), w, 2_000_000, stream))
        assert rc == 0
        return [out]
    recovers(lm, call, ws, withheld, shared)
