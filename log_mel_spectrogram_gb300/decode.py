"""From log-mel frames to text: linear layers, an 8-bit key/value cache with
its attention, and beam search, over the same C ABI (include/logmel.h).

* ``linear(x, weight, bias, ...)`` -- act(x W^T + bias), scaled, plus residual;
  x may be overlapping windows of feature frames, read in place.
* ``KvCache`` -- keys and values of a model's rows in 8 bits, one scale per
  block of tokens and head: ``append``, ``attend``, ``advance``, ``read`` and
  ``reorder``.
* ``beam_step(logits, scores, ...)`` -- the best continuations of every clip.

Inference only, CUDA only, on torch's current stream unless `stream` is given.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _native

__all__ = ["linear", "KvCache", "beam_step", "BeamStep"]

_HALF = {torch.float16: _native.DTYPES["f16"], torch.bfloat16: _native.DTYPES["bf16"]}
_FLOAT = {torch.float32: _native.DTYPES["f32"], **_HALF}
_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_raw_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing
_WORKSPACES: dict = {}


def _workspace(op: str, device: int, stream: int, nbytes: int):
    """(tensor, pointer, bytes) of a zeroed workspace.  An operation's kernels
    leave its counters at zero, so one per operation, device and stream serves
    every call on it; a call that a graph captures gets one of its own, cleared
    on each replay."""
    if _capturing():
        t = torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
        return t, t.data_ptr(), nbytes
    ws = _WORKSPACES.get((op, device, stream))
    if ws is None or ws[2] < nbytes:
        size = max(1 << 16, 1 << (nbytes - 1).bit_length())
        t = torch.zeros(size, dtype=torch.uint8, device=torch.device("cuda", device))
        ws = _WORKSPACES[(op, device, stream)] = (t, t.data_ptr(), size)
    return ws


def _on(device: torch.device, stream):
    """A context in which `device` is current and `stream` (if any) too."""
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(device)


def _elsewhere(t: torch.Tensor, stream) -> bool:
    return stream is not None or t.get_device() != torch._C._cuda_getDevice()


def _refuse_grad(*tensors) -> None:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise RuntimeError("log_mel_spectrogram_gb300 ops are inference-only: inputs must not require grad "
                                   "(use torch.no_grad() or detach())")


def _require(t, name: str, like: torch.Tensor, dtypes, shape=None) -> None:
    """t is a tensor on like's device, of one of `dtypes` and of `shape`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be on the same device as the other inputs")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be of dtype {' or '.join(str(d) for d in dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------

_LINEAR = struct.Struct("5P9q4ifi")


def _rows_of(t: torch.Tensor, name: str):
    """The stride of t's rows when its leading dimensions are one."""
    s = t.stride()
    if t.dim() == 1 or t.numel() == 0:
        return t.shape[-1]
    row, n = s[-2], t.shape[-2]
    for d in range(t.dim() - 3, -1, -1):
        if t.shape[d] != 1:
            if n == 1:
                row = s[d]
            elif s[d] != row * n:
                raise ValueError(f"{name}'s leading dimensions must be evenly spaced rows")
            n *= t.shape[d]
    return row


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, *,
           activation: str | None = None, residual: torch.Tensor | None = None, scale: float = 1.0,
           out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """residual + scale * act(x @ weight.T + bias), rounded once.

    x [..., K] and weight [N, K] float16 or bfloat16 with K contiguous; the
    other dimensions of x may have any stride, overlapping windows included
    (a convolution over log-mel frames [B, F, M] with `taps` taps is
    ``frames.as_strided((B, F - taps + 1, taps * M), (F * M, M, 1))`` against a
    [N, taps * M] weight).  bias [N] float32 or x's dtype; residual [..., N] of
    x's dtype.  activation: None, "relu", "gelu" (erf), "gelu_tanh" or "silu".
    out_dtype: x's dtype (default) or float32; out may be residual itself."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() < 1:
        raise ValueError("x must be a CUDA tensor [..., K]")
    if stream is not None or x.get_device() != torch._C._cuda_getDevice():
        with _on(x.device, stream):
            return linear(x, weight, bias, activation=activation, residual=residual, scale=scale, out=out,
                          out_dtype=out_dtype)
    dt = x.dtype
    code = _HALF.get(dt)
    if code is None:
        raise ValueError("x must be float16 or bfloat16")
    _refuse_grad(x, weight, bias, residual)
    shape = x.shape
    k = shape[-1]
    _require(weight, "weight", x, (dt,))
    if weight.dim() != 2 or weight.shape[1] != k:
        raise ValueError(f"weight must be [N, {k}]")
    n = weight.shape[0]
    ws_ = weight.stride()
    xs = x.stride()
    if (k > 1) and (xs[-1] != 1 or ws_[1] != 1):
        raise ValueError("the last dimension of x and weight must be contiguous")
    dims = len(shape)
    if dims == 2:
        groups, rows, gs, rs = 1, shape[0], 0, xs[0]
    elif dims == 1:
        groups, rows, gs, rs = 1, 1, 0, 0
    elif dims == 3:
        groups, rows, gs, rs = shape[0], shape[1], xs[0], xs[1]
    else:
        if x.numel():
            lead = torch.empty(0, device="meta").as_strided(shape[:-1], xs[:-1])
            try:
                lead = lead.view(-1, shape[-2])
            except RuntimeError:
                raise ValueError("x's leading dimensions must be evenly spaced") from None
            groups, rows, gs, rs = *lead.shape, *lead.stride()
        else:
            groups, rows, gs, rs = math.prod(shape[:-2]), shape[-2], 0, 0
    if bias is not None:
        _require(bias, "bias", x, (torch.float32, dt), (n,))
        if n > 1 and bias.stride(0) != 1:
            raise ValueError("bias must be contiguous")
    act = _ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {[a for a in _ACTIVATIONS if a]} or None")
    out_shape = shape[:-1] + (n,)
    od = dt if out_dtype is None else out_dtype
    if out is None:
        if od is not dt and od is not torch.float32:
            raise ValueError("out_dtype must be x's dtype or float32")
        out = torch.empty(out_shape, dtype=od, device=x.device)
        out_row = n
    else:
        _require(out, "out", x, (dt, torch.float32) if out_dtype is None else (od,), out_shape)
        if n > 1 and out.stride(-1) != 1:
            raise ValueError("the last dimension of out must be contiguous")
        od = out.dtype
        out_row = _rows_of(out, "out")
    res_ptr = res_row = 0
    if residual is not None:
        _require(residual, "residual", x, (dt,), out_shape)
        if n > 1 and residual.stride(-1) != 1:
            raise ValueError("the last dimension of residual must be contiguous")
        res_ptr, res_row = residual.data_ptr(), _rows_of(residual, "residual")
    args = _LINEAR.pack(x.data_ptr(), weight.data_ptr(), 0 if bias is None else bias.data_ptr(), res_ptr,
                        out.data_ptr(), groups, rows, k, n, gs, rs, ws_[0], res_row, out_row, code,
                        code if bias is None else _FLOAT[bias.dtype], _FLOAT[od], act, scale, 0)
    L = _native.lib()
    need = _size_of()
    rc = L.lm_linear_workspace_size(args, need)
    if rc == 0:
        dev = x.get_device()
        s = _raw_stream(dev)
        ws = _workspace("linear", dev, s, need._obj.value)
        rc = L.lm_linear(args, ws[1], ws[2], s)
    if rc:
        _native.check(rc, "lm_linear")
    return out


def _size_of():
    return ctypes.byref(ctypes.c_size_t())


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

class KvCache:
    """Keys and values of `rows` sequences in 8 bits.

    A row's tokens lie in blocks of `block` tokens, named by ``table`` [rows,
    blocks per row]; each layer, block and head has one float32 scale:
    key = k8 * k_scale.  ``lens`` [rows] int32 counts the tokens of the steps
    so far.  A step appends to each layer and attends (tokens from lens[r] on),
    then advances:

        cache.append(layer, k, v)          # for each layer
        out = cache.attend(layer, q)
        cache.advance(tokens)              # once, after the last layer

    Tokens past max_tokens (rounded up to whole blocks) are dropped.  The
    tensors k8, v8 [layers, blocks, heads, block, head_dim], k_scale, v_scale
    [layers, blocks, heads], table, spare and lens may be written in place."""

    def __init__(self, rows: int, max_tokens: int, heads: int, head_dim: int, *, layers: int = 1, block: int = 32,
                 dtype: torch.dtype = torch.bfloat16, device=None):
        if dtype not in _HALF:
            raise ValueError("dtype must be torch.float16 or torch.bfloat16")
        if min(rows, max_tokens) < 0 or min(heads, layers) < 1:
            raise ValueError("rows and max_tokens must be >= 0, heads and layers >= 1")
        if head_dim not in (32, 64, 128):
            raise ValueError("head_dim must be 32, 64 or 128")
        if block not in (16, 32, 64, 128):
            raise ValueError("block must be 16, 32, 64 or 128")
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("device must be a CUDA device")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.rows, self.heads, self.head_dim, self.layers, self.block = rows, heads, head_dim, layers, block
        self.dtype, self.device = dtype, dev
        self.width = width = -(-max_tokens // block)
        self.max_tokens = width * block
        blocks = rows * (width + 1)
        self.blocks = blocks
        self._k8, self._v8 = (torch.empty((layers, blocks, heads, block, head_dim), dtype=torch.int8, device=dev)
                              for _ in range(2))
        self._k_scale, self._v_scale = (torch.empty((layers, blocks, heads), dtype=torch.float32, device=dev)
                                        for _ in range(2))
        order = torch.arange(blocks, dtype=torch.int32, device=dev)
        self._table = order[:rows * width].view(rows, width)
        self._spare = order[rows * width:]
        self._lens = torch.zeros(rows, dtype=torch.int32, device=dev)
        self._code = _HALF[dtype]
        self._args = struct.pack("7Pq6i", *(t.data_ptr() for t in (self._k8, self._v8, self._k_scale, self._v_scale,
                                                                  self._table, self._spare, self._lens)),
                                 blocks, layers, rows, width, heads, head_dim, block)
        self._need: dict = {}

    k8 = property(lambda self: self._k8)
    v8 = property(lambda self: self._v8)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)
    table = property(lambda self: self._table)
    spare = property(lambda self: self._spare)
    lens = property(lambda self: self._lens)

    def _tokens(self, t, name: str, heads: int | None):
        """Checks [rows, tokens, heads, head_dim] and returns its strides, packed."""
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.get_device() != self.device.index:
            raise ValueError(f"{name} must be on the cache's device")
        if t.dtype is not self.dtype:
            raise ValueError(f"{name} must be {self.dtype}")
        sh = t.shape
        if len(sh) != 4 or sh[0] != self.rows or sh[3] != self.head_dim or (heads is not None and sh[2] != heads):
            raise ValueError(f"{name} must be [{self.rows}, tokens, {'heads' if heads is None else heads}, "
                             f"{self.head_dim}]")
        s = t.stride()
        if s[3] != 1:
            raise ValueError(f"the last dimension of {name} must be contiguous")
        return struct.pack("3q", s[0], s[1], s[2])

    def _counts(self, counts):
        if counts is None:
            return None
        if not isinstance(counts, torch.Tensor) or not counts.is_cuda or counts.dtype is not torch.int32 or \
                counts.shape != (self.rows,) or not counts.is_contiguous() or \
                counts.get_device() != self.device.index:
            raise ValueError(f"counts must be a contiguous int32 CUDA tensor [{self.rows}] on the cache's device")
        return counts.data_ptr()

    def _layer(self, layer) -> int:
        if not 0 <= layer < self.layers:
            raise ValueError(f"layer must be in 0 .. {self.layers - 1}")
        return int(layer)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None, *,
               values: bool = False, stream=None):
        """Appends k, v [rows, tokens, heads, head_dim] to one layer, row r's
        first counts[r] tokens (all, where counts is None) at lens[r] on.  A
        block's scale grows to its largest value / 127; where it grows, what
        the block held is rounded anew.  lens stays as it is (see advance).

        values=True returns (k, v) as the cache then holds them: [rows, span,
        heads, head_dim] from the first token of the block that lens[r] falls
        in, zeros past the row's last token."""
        dev = self.device
        if stream is not None or dev.index != torch._C._cuda_getDevice():
            with _on(dev, stream):
                return self.append(layer, k, v, counts, values=values)
        _refuse_grad(k, v)
        ks = self._tokens(k, "k", self.heads)
        vs = self._tokens(v, "v", self.heads)
        t = k.shape[1]
        if v.shape[1] != t:
            raise ValueError("k and v must have as many tokens")
        kv = vv = None
        kp = vp = 0
        if values:
            span = ((t - 1 + self.block - 1) // self.block + 1) * self.block if t else 0
            both = torch.empty((2, self.rows, span, self.heads, self.head_dim), dtype=self.dtype, device=dev)
            kv, vv = both.unbind(0)
            kp = both.data_ptr()
            vp = kp + both.numel()  # half of the elements, two bytes each
        rc = _native.lib().lm_kv_append(self._args, self._layer(layer), k.data_ptr(), v.data_ptr(), ks, vs, t,
                                        self._counts(counts), self._code, kp, vp, _raw_stream(dev.index))
        if rc:
            _native.check(rc, "lm_kv_append")
        return (kv, vv) if values else None

    def attend(self, layer: int, q: torch.Tensor, counts: torch.Tensor | None = None, *, causal: bool = True,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """softmax(scale * q k^T) v over one layer, for q [rows, tokens,
        q_heads, head_dim]; q_heads is a multiple of heads (query head h reads
        key head h // (q_heads // heads)).  scale defaults to head_dim ** -0.5.

        causal: the step's counts[r] tokens (all, where counts is None) are in
        the cache from lens[r] on, and query i sees up to token lens[r] + i;
        queries past counts[r] see nothing.  Otherwise every query sees the
        lens[r] + counts[r] tokens (lens[r] where counts is None).  A query
        that sees nothing gives zeros."""
        dev = self.device
        if stream is not None or dev.index != torch._C._cuda_getDevice():
            with _on(dev, stream):
                return self.attend(layer, q, counts, causal=causal, scale=scale, out=out)
        _refuse_grad(q)
        qs = self._tokens(q, "q", None)
        _, t, hq, d = shape = q.shape
        if hq == 0 or hq % self.heads:
            raise ValueError(f"q must have a multiple of {self.heads} heads")
        if out is None:
            out = torch.empty(shape, dtype=self.dtype, device=dev)
        else:
            _require(out, "out", q, (self.dtype,), shape)
            if not out.is_contiguous():
                raise ValueError("out must be contiguous")
        L = _native.lib()
        need = self._need.get((t, hq))
        if need is None:
            n = ctypes.c_size_t()
            _native.check(L.lm_kv_attend_workspace_size(self._args, t, hq, ctypes.byref(n)),
                          "lm_kv_attend_workspace_size")
            need = self._need[(t, hq)] = n.value
        s = _raw_stream(dev.index)
        ws = _workspace("attend", dev.index, s, need)
        rc = L.lm_kv_attend(self._args, self._layer(layer), q.data_ptr(), qs, t, hq, self._counts(counts),
                            t if causal else 0, causal, d ** -0.5 if scale is None else scale, self._code,
                            out.data_ptr(), ws[1], ws[2], s)
        if rc:
            _native.check(rc, "lm_kv_attend")
        return out

    def advance(self, tokens) -> None:
        """Adds a step's tokens (a number, or a [rows] int32 tensor) to lens."""
        self._lens.add_(tokens)

    def read(self, layer: int | None, start: int, count: int, *, stream=None):
        """(k, v), the values that tokens start .. start + count - 1 stand for:
        [rows, count, heads, head_dim], or [layers, rows, ...] where layer is
        None; zeros from lens[r] on."""
        dev = self.device
        if stream is not None or dev.index != torch._C._cuda_getDevice():
            with _on(dev, stream):
                return self.read(layer, start, count)
        if start < 0 or count < 0:
            raise ValueError("start and count must be >= 0")
        lead = (2, self.layers) if layer is None else (2,)
        both = torch.empty(lead + (self.rows, count, self.heads, self.head_dim), dtype=self.dtype, device=dev)
        kp = both.data_ptr()
        rc = _native.lib().lm_kv_read(self._args, -1 if layer is None else self._layer(layer), start, count,
                                      self._code, kp, kp + both.numel(), _raw_stream(dev.index))
        if rc:
            _native.check(rc, "lm_kv_read")
        return both.unbind(0)

    def reorder(self, parents: torch.Tensor, *, stream=None) -> None:
        """Lets rows [clips * beams] follow a beam step: row (c, i) takes the
        tokens of row (c, parents[c, i]) of its clip (parents [clips, beams]
        int32, as beam_step returns it).  Whole blocks are shared through the
        table, the open block is copied.  Rows of a clip have one length."""
        dev = self.device
        if stream is not None or dev.index != torch._C._cuda_getDevice():
            with _on(dev, stream):
                return self.reorder(parents)
        if not isinstance(parents, torch.Tensor) or not parents.is_cuda or parents.dtype is not torch.int32 or \
                parents.dim() != 2 or parents.numel() != self.rows or not parents.is_contiguous() or \
                parents.get_device() != dev.index:
            raise ValueError(f"parents must be a contiguous [clips, beams] int32 CUDA tensor of {self.rows} rows on "
                             "the cache's device")
        s = _raw_stream(dev.index)
        ws = _workspace("reorder", dev.index, s, 16 + 4 * parents.shape[0])
        rc = _native.lib().lm_kv_reorder(self._args, parents.data_ptr(), parents.shape[1], ws[1], ws[2], s)
        if rc:
            _native.check(rc, "lm_kv_reorder")


# ---------------------------------------------------------------------------
# beam search
# ---------------------------------------------------------------------------

class BeamStep(NamedTuple):
    """The beams of a step, best first: [clips, beams] each, and the history."""
    scores: torch.Tensor    # float32 totals
    tokens: torch.Tensor    # int32
    parents: torch.Tensor   # int32, the beams that they continue
    finished: torch.Tensor  # bool
    history: torch.Tensor | None  # int32 [clips, beams, width]


_BEAM = struct.Struct("9P6q2i")


def beam_step(logits: torch.Tensor, scores: torch.Tensor, finished: torch.Tensor | None = None,
              history: torch.Tensor | None = None, length: int = 0, *, eos: int | None = None,
              stream=None) -> BeamStep:
    """One step of beam search over logits [clips, beams, vocab] (float32,
    float16 or bfloat16): the `beams` continuations of each clip with the
    largest scores[c, i] + log_softmax(logits[c, i])[token].

    Among equal totals the lower beam goes first, then the larger logit, then
    the lower token.  A finished beam (finished [clips, beams] bool; needs eos)
    offers eos alone, at its score.  A score of -inf marks a beam that is not
    in use (all but the first, in the first step).  history [clips, beams,
    width] int32 follows its beams and gets the token at place `length`."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 3:
        raise ValueError("logits must be a CUDA tensor [clips, beams, vocab]")
    if stream is not None or logits.get_device() != torch._C._cuda_getDevice():
        with _on(logits.device, stream):
            return beam_step(logits, scores, finished, history, length, eos=eos)
    code = _FLOAT.get(logits.dtype)
    if code is None:
        raise ValueError("logits must be float32, float16 or bfloat16")
    _refuse_grad(logits, scores)
    clips, beams, vocab = shape = logits.shape
    ls = logits.stride()
    if (vocab > 1 and ls[2] != 1) or (clips > 1 and beams > 0 and ls[0] != beams * ls[1] and beams > 1):
        raise ValueError("logits must be evenly spaced rows of contiguous values")
    row = ls[1] if beams > 1 else ls[0]
    lead = shape[:2]
    dev = logits.get_device()
    device = logits.device
    if scores.dtype is not torch.float32 or scores.shape != lead or not scores.is_contiguous() or \
            scores.get_device() != dev:
        raise ValueError("scores must be a contiguous [clips, beams] float32 CUDA tensor on the logits' device")
    fp = hp = ohp = width = 0
    if finished is not None:
        if finished.dtype is not torch.bool or finished.shape != lead or not finished.is_contiguous() or \
                finished.get_device() != dev:
            raise ValueError("finished must be a contiguous [clips, beams] bool CUDA tensor on the logits' device")
        if eos is None:
            raise ValueError("finished beams need eos")
        fp = finished.data_ptr()
    if eos is not None and not 0 <= eos < vocab:
        raise ValueError("eos must be a token of the vocabulary")
    new_history = None
    if history is not None:
        if history.dtype is not torch.int32 or history.dim() != 3 or history.shape[:2] != lead or \
                not history.is_contiguous() or history.get_device() != dev:
            raise ValueError("history must be a contiguous [clips, beams, width] int32 CUDA tensor on the logits' "
                             "device")
        width = history.shape[2]
        if not 0 <= length < width:
            raise ValueError("length must be a place of the history")
        new_history = torch.empty_like(history)
        hp, ohp = history.data_ptr(), new_history.data_ptr()
    new_scores = torch.empty_like(scores)
    tokens, parents = torch.empty((2, clips, beams), dtype=torch.int32, device=device).unbind(0)
    ended = torch.empty(lead, dtype=torch.bool, device=device)
    args = _BEAM.pack(logits.data_ptr(), scores.data_ptr(), fp, hp, new_scores.data_ptr(), tokens.data_ptr(),
                      parents.data_ptr(), ended.data_ptr(), ohp, clips, vocab, row, width, length,
                      -1 if eos is None else eos, beams, code)
    L = _native.lib()
    need = _size_of()
    rc = L.lm_beam_step_workspace_size(args, need)
    if rc == 0:
        s = _raw_stream(dev)
        ws = _workspace("beam", dev, s, need._obj.value)
        rc = L.lm_beam_step(args, ws[1], ws[2], s)
    if rc:
        _native.check(rc, "lm_beam_step")
    return BeamStep(new_scores, tokens, parents, ended, new_history)
