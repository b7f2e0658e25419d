"""From waveforms to tokens: log-mel features, an encoder, and beam search with
a decoder whose keys and values are held in 8 bits.

The model is a small encoder-decoder of random weights (there is none to
download here), so the tokens mean nothing; every call is the one a real model
makes.  Steps, with this package's part of each:

  waveform -> log-mel frames          MelSpectrogram(log_mel=True)
  frames -> model width               linear over windows of frames, in place
  encoder layers                      linear, KvCache.append / attend (not causal)
  decoder layers, one token a beam    linear, KvCache (own tokens, causal; the
                                      encoder's frames, shared by a clip's beams)
  next tokens                         linear onto the vocabulary, beam_step,
                                      KvCache.reorder

    python examples/transcribe.py [--clips 2] [--seconds 3] [--beams 5] [--tokens 24]
"""
from __future__ import annotations

import argparse
import math
import pathlib
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parents[1]))
import log_mel_spectrogram_gb300 as lm  # noqa: E402

MELS, TAPS = 80, 3


class Layer:
    """Weights of one block: attention (and, in a decoder, attention over the encoder), feed-forward."""

    def __init__(self, width: int, cross: bool, rand):
        def dense(n, k):
            return rand(n, k) / math.sqrt(k)
        self.qkv, self.qkv_bias = dense(3 * width, width), torch.zeros(3 * width, device="cuda")
        self.out = dense(width, width)
        self.cross_q, self.cross_kv, self.cross_out = (dense(n * width, width) if cross else None for n in (1, 2, 1))
        self.up, self.up_bias = dense(4 * width, width), torch.zeros(4 * width, device="cuda")
        self.down = dense(width, 4 * width)


class Model:
    def __init__(self, width: int = 256, heads: int = 4, encoder: int = 2, decoder: int = 2, vocab: int = 1009,
                 dtype: torch.dtype = torch.bfloat16, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(dtype)
        self.width, self.heads, self.dim, self.vocab, self.dtype = width, heads, width // heads, vocab, dtype
        self.stem = rand(width, TAPS * MELS) / math.sqrt(TAPS * MELS)
        self.stem_bias = torch.zeros(width, device="cuda")
        self.encoder = [Layer(width, False, rand) for _ in range(encoder)]
        self.decoder = [Layer(width, True, rand) for _ in range(decoder)]
        self.tokens = rand(vocab, width)
        self.head = 3 * rand(vocab, width) / math.sqrt(width)
        self.mel = lm.MelSpectrogram(n_fft=400, hop_length=160, n_mels=MELS, f_max=8000.0, log_mel=True)

    def norm(self, x):
        return F.layer_norm(x, (self.width,))

    def split(self, x, parts: int):
        """[rows, tokens, parts * width] as `parts` views [rows, tokens, heads, dim]."""
        return x.unflatten(-1, (parts, self.heads, self.dim)).unbind(2)

    def encode(self, wave: torch.Tensor) -> torch.Tensor:
        """wave [clips, samples] float32 -> [clips, frames, width]."""
        frames = self.mel(wave).transpose(1, 2)
        clips, n, _ = frames.shape
        padded = F.pad(frames, (0, 0, TAPS // 2, TAPS // 2)).to(self.dtype).contiguous()
        windows = padded.as_strided((clips, n, TAPS * MELS), (padded.stride(0), MELS, 1))
        x = lm.linear(windows, self.stem, self.stem_bias, activation="gelu")
        cache = lm.KvCache(clips, n, self.heads, self.dim, layers=len(self.encoder), dtype=self.dtype)
        for i, layer in enumerate(self.encoder):
            q, k, v = self.split(lm.linear(self.norm(x), layer.qkv, layer.qkv_bias), 3)
            cache.append(i, k, v)
            seen = torch.full((clips,), n, dtype=torch.int32, device="cuda")
            a = cache.attend(i, q, seen, causal=False)
            x = lm.linear(a.flatten(2), layer.out, residual=x)
            h = lm.linear(self.norm(x), layer.up, layer.up_bias, activation="gelu")
            x = lm.linear(h, layer.down, residual=x)
        return self.norm(x)

    def remember(self, x: torch.Tensor) -> lm.KvCache:
        """The decoder's keys and values of the encoder's frames, one row per clip."""
        cache = lm.KvCache(x.shape[0], x.shape[1], self.heads, self.dim, layers=len(self.decoder), dtype=self.dtype)
        for i, layer in enumerate(self.decoder):
            cache.append(i, *self.split(lm.linear(x, layer.cross_kv), 2))
        cache.advance(x.shape[1])
        return cache

    def step(self, tokens: torch.Tensor, own: lm.KvCache, frames: lm.KvCache) -> torch.Tensor:
        """tokens [clips, beams] -> logits [clips, beams, vocab]; appends to `own`."""
        clips, beams = tokens.shape
        x = F.embedding(tokens, self.tokens).view(clips * beams, 1, self.width)
        for i, layer in enumerate(self.decoder):
            q, k, v = self.split(lm.linear(self.norm(x), layer.qkv, layer.qkv_bias), 3)
            own.append(i, k, v)
            x = lm.linear(own.attend(i, q).flatten(2), layer.out, residual=x)
            q = lm.linear(self.norm(x), layer.cross_q).view(clips, beams, self.heads, self.dim)
            a = frames.attend(i, q, causal=False)  # a clip's beams are the queries of one row
            x = lm.linear(a.view(clips * beams, 1, self.width), layer.cross_out, residual=x)
            h = lm.linear(self.norm(x), layer.up, layer.up_bias, activation="gelu")
            x = lm.linear(h, layer.down, residual=x)
        own.advance(1)
        return lm.linear(self.norm(x), self.head, out_dtype=torch.float32).view(clips, beams, self.vocab)


@torch.no_grad()
def transcribe(model: Model, wave: torch.Tensor, beams: int = 5, tokens: int = 24, start: int = 0):
    """The best `beams` token sequences of each clip: scores [clips, beams], tokens [clips, beams, tokens]."""
    clips, eos = wave.shape[0], model.vocab - 1
    frames = model.remember(model.encode(wave))
    own = lm.KvCache(clips * beams, tokens, model.heads, model.dim, layers=len(model.decoder), dtype=model.dtype)
    scores = torch.full((clips, beams), -math.inf, device="cuda")
    scores[:, 0] = 0  # one beam to start from
    finished = torch.zeros((clips, beams), dtype=torch.bool, device="cuda")
    history = torch.full((clips, beams, tokens), eos, dtype=torch.int32, device="cuda")
    last = torch.full((clips, beams), start, dtype=torch.int32, device="cuda")
    for i in range(tokens):
        step = lm.beam_step(model.step(last, own, frames), scores, finished, history, i, eos=eos)
        scores, last, finished, history = step.scores, step.tokens, step.finished, step.history
        own.reorder(step.parents)
    return scores, history


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--clips", type=int, default=2)
    ap.add_argument("--seconds", type=float, default=3.0)
    ap.add_argument("--beams", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=24)
    a = ap.parse_args()
    wave = torch.randn(a.clips, int(16000 * a.seconds), device="cuda") * 0.1
    scores, tokens = transcribe(Model(), wave, a.beams, a.tokens)
    for c in range(a.clips):
        print(f"clip {c}: {scores[c, 0].item():.2f}  {' '.join(map(str, tokens[c, 0].tolist()))}")


if __name__ == "__main__":
    main()
