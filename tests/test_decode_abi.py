"""Refusals of the decoding entry points' C ABI: all are found on the host, on a
machine without a GPU (the pointers are never used)."""
import ctypes
import struct

import pytest

P = 0x100000  # a pointer that is aligned to anything


@pytest.fixture(scope="module")
def L():
    from log_mel_spectrogram_gb300 import build, _native
    build.build()
    return _native.lib()


def linear_args(x=P, w=2 * P, bias=0, res=0, out=3 * P, groups=1, rows=4, k=64, n=32, xg=0, xr=64, wr=64, rr=32, orow=32,
                dtype=2, bias_dtype=2, out_dtype=2, act=0, scale=1.0):
    return struct.pack("5P9q4ifi", x, w, bias, res, out, groups, rows, k, n, xg, xr, wr, rr, orow, dtype, bias_dtype,
                       out_dtype, act, scale, 0)


def test_struct_sizes_match_the_header():
    assert struct.calcsize("5P9q4ifi") == 136 and struct.calcsize("7Pq6i") == 88 and struct.calcsize("9P6q2i") == 128


def test_linear(L):
    n = ctypes.c_size_t()

    def size(**a):
        return L.lm_linear_workspace_size(linear_args(**a), ctypes.byref(n))

    def call(ws=P, ws_bytes=1 << 20, **a):
        return L.lm_linear(linear_args(**a), ws, ws_bytes, None)
    assert size() == 0 and n.value >= 16
    plain = n.value
    assert size(k=65, xr=65, wr=65) == 0 and n.value > plain  # rows off 16 bytes are copied into the workspace
    assert L.lm_linear_workspace_size(None, ctypes.byref(n)) == 1
    assert L.lm_linear_workspace_size(linear_args(), None) == 1
    for bad in (dict(rows=-1), dict(k=-1), dict(n=-1), dict(groups=-1), dict(xr=-8), dict(wr=-8), dict(orow=-1),
                dict(act=5), dict(act=-1)):
        assert size(**bad) == 1, bad
    for bad in (dict(dtype=0), dict(dtype=1), dict(bias=P, bias_dtype=3), dict(out_dtype=3), dict(k=2 ** 31),
                dict(n=2 ** 31), dict(rows=2 ** 31), dict(groups=2 ** 20, rows=2 ** 20)):
        assert size(**bad) == 2, bad
    assert call(x=0) == 1 and call(w=0) == 1 and call(out=0) == 1
    assert call(x=P + 1) == 3 and call(out=P + 1) == 3 and call(bias=P + 2, bias_dtype=0) == 3 and call(ws=P + 8) == 3
    assert call(ws=0) == 7 and call(ws_bytes=8) == 7
    assert call(rows=0) == 0 and call(n=0) == 0 and call(groups=0) == 0


def cache_args(k8=P, v8=P, ks=P, vs=P, table=P, spare=P, lens=P, blocks=20, layers=2, rows=6, width=3, heads=2, dim=64,
               block=32):
    return struct.pack("7Pq6i", k8, v8, ks, vs, table, spare, lens, blocks, layers, rows, width, heads, dim, block)


def test_cache(L):
    st = struct.pack("3q", 128, 128, 64)

    def append(c=None, layer=0, k=P, v=P, ks=st, vs=st, t=1, dtype=2, kv=0, vv=0, **a):
        return L.lm_kv_append(c or cache_args(**a), layer, k, v, ks, vs, t, None, dtype, kv, vv, None)

    def attend(layer=0, q=P, qs=st, t=1, hq=2, dtype=2, out=P, ws=P, ws_bytes=1 << 24, **a):
        return L.lm_kv_attend(cache_args(**a), layer, q, qs, t, hq, None, t, 1, 0.1, dtype, out, ws, ws_bytes, None)

    def read(layer=0, start=0, count=1, dtype=2, k=P, v=P, **a):
        return L.lm_kv_read(cache_args(**a), layer, start, count, dtype, k, v, None)

    def reorder(parents=P, beams=3, ws=P, ws_bytes=4096, **a):
        return L.lm_kv_reorder(cache_args(**a), parents, beams, ws, ws_bytes, None)
    for f in (append, attend, read, reorder):
        for bad in (dict(lens=0), dict(k8=0), dict(v8=0), dict(table=0), dict(layers=0), dict(heads=0), dict(rows=-1),
                    dict(width=-1), dict(blocks=-1)):
            assert f(**bad) == 1, (f.__name__, bad)
        for bad in (dict(dim=48), dict(dim=256), dict(block=24), dict(block=8), dict(width=2 ** 30)):
            assert f(**bad) == 2, (f.__name__, bad)
        assert f(k8=P + 8) == 3, f.__name__
    assert append(layer=2) == 1 and append(layer=-1) == 1 and append(t=-1) == 1 and append(ks=None) == 1
    assert append(dtype=0) == 2 and append(k=P + 1) == 3 and append(kv=P) == 1 and append(kv=P + 8, vv=P) == 3
    assert append(t=0) == 0 and append(rows=0) == 0
    assert append(ks=struct.pack("3q", -1, 0, 0)) == 1
    assert attend(layer=2) == 1 and attend(hq=3) == 1 and attend(hq=0) == 1 and attend(qs=None) == 1
    assert attend(dtype=0) == 2 and attend(out=P + 8) == 3 and attend(ws=0) == 7 and attend(ws_bytes=16) == 7
    assert attend(t=0) == 0 and attend(rows=0) == 0
    n = ctypes.c_size_t()
    assert L.lm_kv_attend_workspace_size(cache_args(), 1, 2, ctypes.byref(n)) == 0 and n.value >= 256
    assert L.lm_kv_attend_workspace_size(cache_args(), 1, 2, None) == 1
    assert read(layer=2) == 1 and read(layer=-2) == 1 and read(start=-1) == 1 and read(count=-1) == 1
    assert read(dtype=0) == 2 and read(k=0) == 1 and read(k=P + 4) == 3 and read(count=0) == 0
    assert reorder(beams=0) == 1 and reorder(beams=4) == 1 and reorder(parents=0) == 1 and reorder(spare=0) == 1
    assert reorder(beams=33, rows=66) == 2 and reorder(ws=0) == 7 and reorder(ws_bytes=8) == 7
    assert reorder(ws=P + 4) == 3 and reorder(rows=0) == 0


def beam_args(x=P, sc=P, fin=0, hist=0, osc=P, ot=P, op=P, of=P, oh=0, clips=2, vocab=100, row=100, width=0, length=0,
              eos=-1, beams=5, dtype=0):
    return struct.pack("9P6q2i", x, sc, fin, hist, osc, ot, op, of, oh, clips, vocab, row, width, length, eos, beams,
                       dtype)


def test_beam_step(L):
    n = ctypes.c_size_t()

    def size(**a):
        return L.lm_beam_step_workspace_size(beam_args(**a), ctypes.byref(n))

    def call(ws=P, ws_bytes=1 << 24, **a):
        return L.lm_beam_step(beam_args(**a), ws, ws_bytes, None)
    assert size() == 0 and n.value > 256
    for bad in (dict(clips=-1), dict(vocab=0), dict(beams=0), dict(row=-1), dict(eos=100), dict(eos=-2),
                dict(fin=P), dict(hist=P), dict(oh=P), dict(hist=P, oh=P, width=4, length=4),
                dict(hist=P, oh=P, width=4, length=-1)):
        assert size(**bad) == 1, bad
    for bad in (dict(beams=33), dict(dtype=1), dict(vocab=2 ** 24 + 1, row=2 ** 24 + 1)):
        assert size(**bad) == 2, bad
    assert call(x=0) == 1 and call(sc=0) == 1 and call(ot=0) == 1 and call(of=0) == 1
    assert call(x=P + 2) == 3 and call(sc=P + 2) == 3 and call(ws=P + 8) == 3
    assert call(ws=0) == 7 and call(ws_bytes=256) == 7 and call(clips=0) == 0
