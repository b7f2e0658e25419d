"""A wait that runs out in a CTA other than the first is reported, too.

As tests/test_layer_waits.py, for CTA 1 of the forms whose CTAs each wait for their own copies: a tile a CTA, and
clusters that share out the sum.  (Of a pair only the first CTA counts copies.)  Nothing here faults, traps or hangs
the GPU: the only failure is a wait that nothing completes.
"""
import ctypes
import struct

import pytest
import torch

import test_kv_waits as waits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def runs_out(lm, ws, withheld, regular):
    """Both return outputs that were 7 before."""
    lm.decode_error()
    want = regular()
    assert lm.decode_error() == 0 and waits.error(ws) == 0
    got = withheld()
    assert lm.decode_error() & waits.MBAR_TIMEOUT_BIT and waits.error(ws) & waits.MBAR_TIMEOUT_BIT
    assert any(not torch.equal(a, b) for a, b in zip(got, want))  # (what CTA 1 computes is missing)
    ws.zero_()
    assert all(torch.equal(a, b) for a, b in zip(regular(), want))
    assert lm.decode_error() == 0 and waits.error(ws) == 0


def half(seed, *shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").half() / 8 for s in shapes]


def sevens(*shapes):
    return [torch.full(s, 7.0, device="cuda", dtype=torch.float16) for s in shapes]


@pytest.mark.parametrize("m,k,n", [(700, 200, 900), (5, 1024, 1024)])
def test_gated_linear(lm, m, k, n):
    x, wg, wu = half(m, (m, k), (n, k), (n, k))
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")

    def call(name, *more):
        outs = sevens((m, n))
        args = struct.pack("6P7q4i", x.data_ptr(), wg.data_ptr(), wu.data_ptr(), 0, 0, outs[0].data_ptr(), m, k, n, k, k, k,
                           n, 2, 0, 4, 0)
        f = getattr(waits.lib(), name)
        assert f(args, ws.data_ptr(), ws.numel(), *more, torch.cuda.current_stream().cuda_stream) == 0
        return outs
    runs_out(lm, ws, lambda: call("lm_debug_gated_linear_withhold", 1, 2_000_000), lambda: call("lm_gated_linear"))


@pytest.mark.parametrize("m,k,n", [(700, 200, 904), (5, 1024, 1024)])
def test_gated_linear_backward(lm, m, k, n):
    x, wg, wu, go = half(m, (m, k), (n, k), (n, k), (m, n))
    need = ctypes.c_size_t()

    def args(outs):
        return struct.pack("6P7q4i6Pq", x.data_ptr(), wg.data_ptr(), wu.data_ptr(), 0, 0, 0, m, k, n, k, k, k, 0, 2, 0, 4, 0,
                           go.data_ptr(), *(o.data_ptr() for o in outs), 0, 0, n)
    assert waits.lib().lm_gated_linear_backward_workspace_size(args(sevens((m, k), (n, k), (n, k))), ctypes.byref(need)) == 0
    ws = torch.zeros(need.value, dtype=torch.uint8, device="cuda")

    def call(name, *more):
        outs = sevens((m, k), (n, k), (n, k))
        f = getattr(waits.lib(), name)
        assert f(args(outs), ws.data_ptr(), ws.numel(), *more, torch.cuda.current_stream().cuda_stream) == 0
        return outs
    runs_out(lm, ws, lambda: call("lm_debug_gated_linear_backward_withhold", 1, 2_000_000),
             lambda: call("lm_gated_linear_backward"))


@pytest.mark.parametrize("m,k,n,group", [(90, 200, 900, 64), (200, 2048, 300, 32), (60, 300, 25000, 128),
                                         (256, 640, 20001, 32)])
def test_linear4(lm, m, k, n, group):
    x, w = half(m, (m, k), (n, k))
    w4 = lm.quantize_weight(w, group)
    weight = struct.pack("2P2q2i", w4.packed.data_ptr(), w4.scale.data_ptr(), n, k, group, 0)
    ws = torch.zeros(1 << 18, dtype=torch.uint8, device="cuda")

    def call(name, *more):
        outs = sevens((m, n))
        args = struct.pack("5P9q4ifi", x.data_ptr(), 0, 0, 0, outs[0].data_ptr(), 1, m, k, n, 0, k, 0, 0, n, 2, 2, 2, 0, 1.0,
                           0)
        f = getattr(waits.lib(), name)
        assert f(args, weight, ws.data_ptr(), ws.numel(), *more, torch.cuda.current_stream().cuda_stream) == 0
        return outs
    runs_out(lm, ws, lambda: call("lm_debug_linear4_withhold", 1, 2_000_000), lambda: call("lm_linear4"))
