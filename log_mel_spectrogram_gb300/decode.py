"""From log-mel frames to text: linear layers, an 8-bit key/value cache with
its attention, and beam search, over the same C ABI (include/logmel.h).

* ``linear(x, weight, bias, ...)`` -- act(x W^T + bias), scaled, plus residual;
  x may be overlapping windows of feature frames, read in place.  The weight may be
  a ``Weight4``, in 4 bits (``quantize_weight``).
* ``layer_norm(x, weight, bias)`` and ``gated_linear(x, w_gate, w_up, ...)``, the
  norm and the gated block of a layer; these two have gradients.
* ``KvCache`` -- keys and values of a model's rows in 8 bits, one scale per
  block of tokens and head: ``append``, ``attend``, ``advance``, ``read``,
  ``reorder`` and ``reset``.
* ``beam_step(logits, scores, ...)`` -- the best continuations of every clip.
* ``decode_error()`` -- whether a wait inside a kernel of these has run out.

Inference only but for layer_norm and gated_linear, CUDA only, on torch's current stream unless `stream` is given.
"""
from __future__ import annotations

import ctypes
import importlib.util
import struct
from typing import NamedTuple

import torch

from . import _native
from . import build as _build

__all__ = ["linear", "Weight4", "quantize_weight", "layer_norm", "gated_linear", "KvCache", "beam_step", "BeamStep", "decode_error"]

_HALF = {torch.float16: _native.DTYPES["f16"], torch.bfloat16: _native.DTYPES["bf16"]}
_FLOAT = {torch.float32: _native.DTYPES["f32"], **_HALF}
_ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_GATES = {**_ACTIVATIONS, "sigmoid": 5}

_DTYPE_CODES = {None: -1, **_FLOAT}
_ext = None


def _binding():
    """The compiled binding (csrc/binding.cpp).  Raises if it is missing."""
    global _ext
    if _ext is None:
        _native.lib()  # liblogmel.so first: the binding is linked against it
        if not _build.BINDING.exists():
            raise RuntimeError(f"the torch binding is not built ({_build.BINDING}); run __graft_entry__.build() "
                               "or python -m log_mel_spectrogram_gb300.build")
        spec = importlib.util.spec_from_file_location("_decode", _build.BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _ext = module
    return _ext


def _checked(r, what: str):
    """r, unless it is a status."""
    if type(r) is int:
        _native.check(r, what)
    return r


def decode_error(device=None, *, clear: bool = True) -> int:
    """Waits for the device and returns the error bits that linear(), gated_linear()
    (and its backward pass) and KvCache.attend() have reported on it since the last call (0: none), replayed
    graphs included.  Every wait inside their kernels is bounded; one that runs out
    ends the kernel, sets a bit here, and leaves outputs that are not whole."""
    v = ctypes.c_uint32()
    with torch.cuda.device(device):
        torch.cuda.synchronize()
        rc = _native.lib().lm_decode_error(ctypes.byref(v), int(clear), torch.cuda.current_stream().cuda_stream)
    if v.value == 0:
        _native.check(rc, "lm_decode_error")
    return v.value


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------

def linear(x: torch.Tensor, weight: torch.Tensor | Weight4, bias: torch.Tensor | None = None, *,
           activation: str | None = None, residual: torch.Tensor | None = None, scale: float = 1.0,
           out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """residual + scale * act(x @ weight.T + bias), rounded once.

    x [..., K] and weight [N, K] float16 or bfloat16 with K contiguous; the
    other dimensions of x may have any stride, overlapping windows included
    (a convolution over log-mel frames [B, F, M] with `taps` taps is
    ``frames.as_strided((B, F - taps + 1, taps * M), (F * M, M, 1))`` against a
    [N, taps * M] weight).  bias [N] float32 or x's dtype; residual [..., N] of
    x's dtype.  activation: None, "relu", "gelu" (erf), "gelu_tanh" or "silu".
    out_dtype: x's dtype (default) or float32; out may be residual itself, and
    overlaps no other input.

    A Weight4 as weight is multiplied as it is where x has few rows (a decoding step): up to 16, or up to 64
    where ceil(rows / 16) * N is at most 16384 (12000 for K above 1024).  For more its values are rounded to
    x's dtype on their way, in each call, by half a step and up to a sixteenth of that: what a prompt and its
    single tokens are multiplied with differs by as much."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear(x, weight, bias, activation=activation, residual=residual, scale=scale, out=out,
                          out_dtype=out_dtype)
    act, code = _ACTIVATIONS.get(activation), _DTYPE_CODES.get(out_dtype)
    if act is None:
        raise ValueError(f"activation must be one of {[a for a in _ACTIVATIONS if a]} or None")
    if code is None:
        raise ValueError("out_dtype must be x's dtype or float32")
    if isinstance(weight, Weight4):
        return _checked((_ext or _binding()).linear(x, weight._head(), bias, act, residual, scale, out, code),
                        "lm_linear4")
    return _checked((_ext or _binding()).linear(x, weight, bias, act, residual, scale, out, code), "lm_linear")


class Weight4:
    """A linear layer's weight [N, K] as whole numbers of -8 .. 7, with one float32 scale for each row and
    `group` consecutive k: value = q * scale.  ``quantize_weight`` rounds a weight to one, ``Weight4.pack`` takes
    numbers and scales that are at hand; ``linear`` takes it as its weight, for x of `dtype`.

    The tensors packed [ceil(N / 128), ceil(K / 64), 4096] uint8 and scale [ceil(N / 128), ceil(K / group), 128]
    float32 hold it in the order of include/logmel.h (lm_weight4)."""

    def __init__(self, packed: torch.Tensor, scale: torch.Tensor, shape, group: int, dtype: torch.dtype):
        self.packed, self.scale, self.shape, self.group, self.dtype = packed, scale, tuple(shape), group, dtype

    device = property(lambda self: self.packed.device)

    def _head(self):
        return (self.packed, self.scale, self.shape[0], self.shape[1], self.group, _HALF[self.dtype])

    @staticmethod
    def _check(group, dtype):
        if dtype not in _HALF:
            raise ValueError("dtype must be torch.float16 or torch.bfloat16")
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")

    @staticmethod
    def pack(q: torch.Tensor, scale: torch.Tensor, *, group: int | None = None, dtype: torch.dtype = torch.bfloat16,
             stream=None) -> Weight4:
        """Lays out q [N, K] int8 (clamped to -8 .. 7) and scale [N, ceil(K / group)] float32.  group
        is the one of 32, 64 and 128 that fits scale's shape (any of those that do, where a row has one scale)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return Weight4.pack(q, scale, group=group, dtype=dtype)
        if group is None:
            fits = [g for g in (32, 64, 128) if q.dim() == 2 == scale.dim() and -(-q.shape[1] // g) == scale.shape[1]]
            if not fits:
                raise ValueError("scale must be [N, ceil(K / group)] with a group of 32, 64 or 128")
            group = fits[-1]
        Weight4._check(group, dtype)
        return Weight4(*_checked(_binding().weight4_pack(q, scale, group), "lm_weight4_pack"), q.shape, group, dtype)

    def values(self, dtype: torch.dtype | None = None, *, stream=None) -> torch.Tensor:
        """The weight [N, K] that it stands for, rounded to dtype (its own; float32 is exact to one rounding)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.values(dtype)
        code = _FLOAT.get(dtype or self.dtype)
        if code is None:
            raise ValueError("dtype must be float32, float16 or bfloat16")
        return _checked(_binding().weight4_values(self._head(), code), "lm_weight4_values")


def quantize_weight(weight: torch.Tensor, group: int = 64, *, dtype: torch.dtype | None = None, stream=None) -> Weight4:
    """Rounds weight [N, K] (float32, float16 or bfloat16) to 4 bits: scale = max |w| of a row's group / 7, q =
    w / scale to the nearest whole number (ties to even).  dtype: of the x that linear will take (weight's own,
    bfloat16 for float32)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantize_weight(weight, group, dtype=dtype)
    if dtype is None:
        dtype = torch.bfloat16 if weight.dtype == torch.float32 else weight.dtype
    Weight4._check(group, dtype)
    return Weight4(*_checked(_binding().weight4_quantize(weight, group), "lm_weight4_quantize"), weight.shape, group,
                   dtype)


# ---------------------------------------------------------------------------
# the rest of a layer
# ---------------------------------------------------------------------------

def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None, *,
               eps: float = 1e-5, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension, rounded once.

    x [..., width] float32, float16 or bfloat16, the last dimension contiguous and
    the others evenly spaced rows; weight and bias [width] float32 or x's dtype.
    out may be x itself, and overlaps no other input; it goes without gradients.

    The gradients of x, weight and bias are those of the formula (first derivatives only);
    sums over rows are taken in 32 bits and in one order.  So are sums of a row's squared
    deviations: where one passes 3.4e38 the row's results are bias, or NaN."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return layer_norm(x, weight, bias, eps=eps, out=out)
    return _checked((_ext or _binding()).layer_norm(x, weight, bias, eps, out), "lm_layer_norm")


def gated_linear(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, b_gate: torch.Tensor | None = None,
                 b_up: torch.Tensor | None = None, *, activation: str | None = "silu", out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """act(x @ w_gate.T + b_gate) * (x @ w_up.T + b_up), rounded once: the gated block of a
    feed-forward layer in one kernel.

    x [..., K], w_gate and w_up [N, K] float16 or bfloat16 with K contiguous, x's other dimensions
    evenly spaced rows; b_gate and b_up [N] float32 or x's dtype, one for both.  activation: "silu",
    "gelu" (erf), "gelu_tanh", "relu", "sigmoid" or None.  out overlaps no input and goes without
    gradients.

    The gradients of all inputs are those of the formula (first derivatives only), from both
    projections computed anew: the forward pass keeps nothing but its inputs.  The projections' own
    gradients are rounded to x's dtype on their way into the products (in float16 one past 65504 is infinite)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_linear(x, w_gate, w_up, b_gate, b_up, activation=activation, out=out)
    act = _GATES.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {[a for a in _GATES if a]} or None")
    return _checked((_ext or _binding()).gated_linear(x, w_gate, w_up, b_gate, b_up, act, out), "lm_gated_linear")


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
    [layers, blocks, heads], table, spare and lens may be written in place.
    copy.deepcopy and pickle give a cache of its own with the same contents.

    A row's blocks from the one that lens[r] falls in onwards must be its own, or
    two rows write one block at once.  ``reorder`` lets the rows of a clip share the
    blocks in front of that one: after it lens must not be set back, and a cache
    that takes other sequences is emptied by ``reset`` first."""

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
        self._bind()

    def _bind(self):
        """The C struct of this object's own tensors."""
        tensors = (self._k8, self._v8, self._k_scale, self._v_scale, self._table, self._spare, self._lens)
        if len({t.device for t in tensors}) != 1 or not self._k8.is_cuda:
            raise ValueError("a KvCache's tensors must be on one CUDA device")
        self.device = self._k8.device
        self._args = struct.pack("7Pq6i", *(t.data_ptr() for t in tensors), self.blocks, self.layers, self.rows,
                                 self.width, self.heads, self.head_dim, self.block)
        self._head = (self._args, self.device.index, self._code)

    # Copies and pickles hold tensors of their own (copy.copy shares them), and their addresses.
    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_args", "_head")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._bind()

    k8 = property(lambda self: self._k8)
    v8 = property(lambda self: self._v8)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)
    table = property(lambda self: self._table)
    spare = property(lambda self: self._spare)
    lens = property(lambda self: self._lens)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, counts: torch.Tensor | None = None, *,
               values: bool = False, stream=None):
        """Appends k, v [rows, tokens, heads, head_dim] to one layer, row r's
        first counts[r] tokens (all, where counts is None) at lens[r] on.  A
        block's scale grows to its largest value times float32(1 / 127); where it
        grows, what the block held is rounded anew.  lens stays as it is (see advance).

        values=True returns (k, v) as the cache then holds them: [rows, span,
        heads, head_dim] from the first token of the block that lens[r] falls
        in, zeros past the row's last token."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.append(layer, k, v, counts, values=values)
        return _checked((_ext or _binding()).kv_append(*self._head, layer, k, v, counts, bool(values)),
                        "lm_kv_append")

    def attend(self, layer: int, q: torch.Tensor, counts: torch.Tensor | None = None, *, causal: bool = True,
               scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """softmax(scale * q k^T) v over one layer, for q [rows, tokens,
        q_heads, head_dim]; q_heads is a multiple of heads (query head h reads
        key head h // (q_heads // heads)).  scale defaults to head_dim ** -0.5.

        causal: the step's counts[r] tokens (all, where counts is None) are in
        the cache from lens[r] on, and query i sees up to token lens[r] + i;
        queries past counts[r] see nothing.  Otherwise every query sees the
        lens[r] + counts[r] tokens (lens[r] where counts is None).  A query
        that sees nothing gives zeros.  out does not overlap q."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.attend(layer, q, counts, causal=causal, scale=scale, out=out)
        return _checked((_ext or _binding()).kv_attend(*self._head, layer, q, counts, causal, scale, out),
                        "lm_kv_attend")

    def advance(self, tokens, *, stream=None) -> None:
        """Adds a step's tokens (a number, or a [rows] int32 tensor) to lens."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.advance(tokens)
        self._lens.add_(tokens)

    def reset(self, *, stream=None) -> None:
        """Empties the cache: no tokens, and every row has blocks of its own again
        (table and spare as at construction)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.reset()
        own = self.rows * self.width
        torch.arange(own, dtype=torch.int32, device=self.device, out=self._table.view(-1))
        torch.arange(own, self.blocks, dtype=torch.int32, device=self.device, out=self._spare)
        self._lens.zero_()

    def read(self, layer: int | None, start: int, count: int, *, stream=None):
        """(k, v), the values that tokens start .. start + count - 1 stand for:
        [rows, count, heads, head_dim], or [layers, rows, ...] where layer is
        None; zeros from lens[r] on."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.read(layer, start, count)
        if layer is not None and layer < 0:
            raise ValueError(f"layer must be in 0 .. {self.layers - 1}, or None")
        return _checked((_ext or _binding()).kv_read(*self._head, -1 if layer is None else layer, start, count),
                        "lm_kv_read")

    def reorder(self, parents: torch.Tensor, *, stream=None) -> None:
        """Lets rows [clips * beams] follow a beam step: row (c, i) takes the
        tokens of row (c, parents[c, i]) of its clip (parents [clips, beams]
        int32, as beam_step returns it).  Whole blocks are shared through the
        table, the open block is copied.  Rows of a clip have one length."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.reorder(parents)
        _checked((_ext or _binding()).kv_reorder(*self._head, parents), "lm_kv_reorder")


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
    width] int32 follows its beams and gets the token at place `length`, a number of
    the host's: a captured call writes at that place on every replay."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return beam_step(logits, scores, finished, history, length, eos=eos)
    return BeamStep(*_checked((_ext or _binding()).beam_step(logits, scores, finished, history, length, eos),
                              "lm_beam_step"))
