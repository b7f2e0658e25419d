"""Refusals of the C ABI of layer norm, the gated layer and weights in 4 bits: found on the host, on a machine
without a GPU (the pointers are never used)."""
import ctypes
import struct

import pytest

from test_decode_abi import linear_args

P = 0x100000
FAR = 1 << 32  # apart from everything


@pytest.fixture(scope="module")
def L():
    from log_mel_spectrogram_gb300 import build, _native
    build.build()
    return _native.lib()


def norm(x=FAR, w=2 * FAR, b=3 * FAR, out=4 * FAR, stats=5 * FAR, rows=4, width=64, xr=64, orow=64, dtype=2, wd=0, bd=0,
         eps=1e-5):
    return struct.pack("5P4q3if", x, w, b, out, stats, rows, width, xr, orow, dtype, wd, bd, eps)


def norm_back(x=FAR, w=2 * FAR, stats=3 * FAR, g=4 * FAR, dx=5 * FAR, dw=6 * FAR, db=7 * FAR, rows=4, width=64, xr=64, gr=64,
              dtype=2, wd=0, bd=0):
    return struct.pack("7P4q4i", x, w, stats, g, dx, dw, db, rows, width, xr, gr, dtype, wd, bd, 0)


def gated(x=FAR, wg=2 * FAR, wu=3 * FAR, bg=0, bu=0, out=4 * FAR, rows=4, k=64, n=32, xr=64, gr=64, ur=64, orow=32, dtype=2,
          bd=0, act=4):
    return struct.pack("6P7q4i", x, wg, wu, bg, bu, out, rows, k, n, xr, gr, ur, orow, dtype, bd, act, 0)


def gated_back(g=5 * FAR, dx=6 * FAR, dwg=7 * FAR, dwu=8 * FAR, dbg=0, dbu=0, grow=32, **a):
    return gated(**a) + struct.pack("6Pq", g, dx, dwg, dwu, dbg, dbu, grow)


def weight(packed=FAR, scale=2 * FAR, n=32, k=64, group=64):
    return struct.pack("2P2q2i", packed, scale, n, k, group, 0)


def test_struct_sizes():
    assert (len(norm()), len(norm_back()), len(gated()), len(gated_back()), len(weight())) == (88, 104, 120, 176, 40)


def test_layer_norm(L):
    f = lambda **a: L.lm_layer_norm(norm(**a), None)  # noqa: E731
    assert L.lm_layer_norm(None, None) == 1
    assert f(rows=0) == 0 and f(width=0) == 0
    for bad in (dict(rows=-1), dict(width=-1), dict(xr=-1), dict(orow=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(x=0),
                dict(out=0), dict(orow=63), dict(out=FAR + 64), dict(out=2 * FAR), dict(out=3 * FAR), dict(stats=FAR),
                dict(stats=4 * FAR), dict(out=FAR, orow=128)):
        assert f(**bad) == 1, bad
    for bad in (dict(dtype=1), dict(dtype=4), dict(wd=3), dict(bd=1), dict(rows=2 ** 31), dict(width=2 ** 31)):
        assert f(**bad) == 2, bad
    for bad in (dict(x=FAR + 1), dict(w=2 * FAR + 2), dict(out=4 * FAR + 1), dict(stats=5 * FAR + 2), dict(dtype=0, x=FAR + 2)):
        assert f(**bad) == 3, bad


def test_layer_norm_backward(L):
    n = ctypes.c_size_t()

    def size(**a):
        return L.lm_layer_norm_backward_workspace_size(norm_back(**a), ctypes.byref(n))

    def f(ws=9 * FAR, ws_bytes=1 << 30, **a):
        return L.lm_layer_norm_backward(norm_back(**a), ws, ws_bytes, None)
    assert size() == 0 and n.value >= 256 and L.lm_layer_norm_backward_workspace_size(None, ctypes.byref(n)) == 1
    assert L.lm_layer_norm_backward_workspace_size(norm_back(), None) == 1
    assert f(width=0) == 0 and f(dx=0, dw=0, db=0) == 0
    for bad in (dict(rows=-1), dict(gr=-1), dict(x=0), dict(g=0), dict(stats=0), dict(dx=4 * FAR), dict(dw=7 * FAR),
                dict(db=2 * FAR), dict(dx=3 * FAR), dict(dw=5 * FAR)):
        assert f(**bad) == 1, bad
    assert f(dtype=7) == 2 and f(wd=3) == 2 and f(g=4 * FAR + 1) == 3 and f(dw=6 * FAR + 2) == 3 and f(ws=9 * FAR + 8) == 3
    assert f(ws=0) == 7 and f(ws_bytes=64) == 7


def test_gated(L):
    n = ctypes.c_size_t()

    def size(**a):
        return L.lm_gated_linear_workspace_size(gated(**a), ctypes.byref(n))

    def f(ws=9 * FAR, ws_bytes=1 << 30, **a):
        return L.lm_gated_linear(gated(**a), ws, ws_bytes, None)
    assert size() == 0 and n.value >= 16 and L.lm_gated_linear_workspace_size(None, ctypes.byref(n)) == 1
    assert f(rows=0) == 0 and f(n=0) == 0
    for bad in (dict(rows=-1), dict(k=-1), dict(n=-1), dict(xr=-1), dict(gr=-1), dict(ur=-1), dict(act=-1), dict(act=6),
                dict(x=0), dict(wg=0), dict(wu=0), dict(out=0), dict(orow=31), dict(out=FAR), dict(out=2 * FAR + 128),
                dict(out=3 * FAR), dict(bg=4 * FAR)):
        assert f(**bad) == 1, bad
    for bad in (dict(dtype=0), dict(dtype=1), dict(bg=10 * FAR, bd=3), dict(k=2 ** 31), dict(n=2 ** 30), dict(rows=2 ** 31)):
        assert f(**bad) == 2, bad
    assert f(x=FAR + 1) == 3 and f(out=4 * FAR + 1) == 3 and f(bg=10 * FAR + 2) == 3 and f(ws=9 * FAR + 8) == 3
    assert f(ws=0) == 7 and f(ws_bytes=8) == 7


def test_gated_backward(L):
    n = ctypes.c_size_t()

    def size(**a):
        return L.lm_gated_linear_backward_workspace_size(gated_back(**a), ctypes.byref(n))

    def f(ws=10 * FAR, ws_bytes=1 << 30, **a):
        return L.lm_gated_linear_backward(gated_back(**a), ws, ws_bytes, None)
    assert size() == 0 and n.value >= 4 * 4 * 32 and L.lm_gated_linear_backward_workspace_size(None, ctypes.byref(n)) == 1
    assert f(dx=0, dwg=0, dwu=0) == 0
    for bad in (dict(grow=-1), dict(g=0), dict(x=0), dict(wu=0), dict(dx=FAR), dict(dwg=2 * FAR), dict(dwu=7 * FAR),
                dict(dx=5 * FAR), dict(dbg=6 * FAR), dict(act=6)):
        assert f(**bad) == 1, bad
    assert f(dtype=0) == 2 and f(dbg=11 * FAR, bd=3) == 2
    assert f(g=5 * FAR + 1) == 3 and f(dx=6 * FAR + 1) == 3 and f(dbg=11 * FAR + 2) == 3 and f(ws=10 * FAR + 4) == 3
    assert f(ws=0) == 7 and f(ws_bytes=64) == 7


def test_weight4(L):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.lm_weight4_size(weight(n=17, k=65, group=32), ctypes.byref(a), ctypes.byref(b)) == 0
    assert a.value == 2 * 4096 and b.value == 3 * 512
    assert L.lm_weight4_size(None, ctypes.byref(a), ctypes.byref(b)) == 1
    assert L.lm_weight4_size(weight(n=-1), ctypes.byref(a), ctypes.byref(b)) == 1
    assert L.lm_weight4_size(weight(group=16), ctypes.byref(a), ctypes.byref(b)) == 2
    assert L.lm_weight4_pack(weight(), 0, P, None) == 1 and L.lm_weight4_pack(weight(packed=0), P, P, None) == 1
    assert L.lm_weight4_pack(weight(packed=FAR + 8), P, P, None) == 3 and L.lm_weight4_pack(weight(n=0), 0, 0, None) == 0
    assert L.lm_weight4_quantize(weight(), P, 64, 1, None) == 2 and L.lm_weight4_quantize(weight(), P, -1, 0, None) == 1
    assert L.lm_weight4_quantize(weight(), P + 2, 64, 0, None) == 3 and L.lm_weight4_quantize(weight(), 0, 64, 0, None) == 1
    assert L.lm_weight4_values(weight(), P, 63, 0, None) == 1 and L.lm_weight4_values(weight(), 0, 64, 0, None) == 1
    assert L.lm_weight4_values(weight(), P + 1, 64, 2, None) == 3 and L.lm_weight4_values(weight(), P, 64, 5, None) == 2


def test_linear4(L):
    n = ctypes.c_size_t()

    def f(ws=9 * FAR, ws_bytes=1 << 30, w=None, **a):
        a = {**dict(x=3 * FAR, out=4 * FAR, w=0, wr=0), **a}
        return L.lm_linear4(linear_args(**a), w or weight(), ws, ws_bytes, None)
    assert L.lm_linear4_workspace_size(linear_args(), weight(), ctypes.byref(n)) == 0 and n.value >= 16
    assert L.lm_linear4_workspace_size(linear_args(), None, ctypes.byref(n)) == 1
    assert L.lm_linear4_workspace_size(linear_args(), weight(), None) == 1
    assert f(rows=0) == 0 and f(n=0, w=weight(n=0)) == 0
    for bad in (dict(w=weight(n=16)), dict(w=weight(k=128)), dict(w=weight(packed=0)), dict(x=0), dict(out=0), dict(act=5),
                dict(out=FAR), dict(out=2 * FAR), dict(out=3 * FAR), dict(orow=31), dict(rows=-1)):
        assert f(**bad) == 1, bad
    assert f(dtype=0) == 2 and f(w=weight(group=48)) == 2
    assert f(x=3 * FAR + 1) == 3 and f(w=weight(scale=2 * FAR + 4)) == 3 and f(ws=9 * FAR + 8) == 3
    assert f(ws=0) == 7 and f(ws_bytes=8) == 7
