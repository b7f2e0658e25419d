"""examples/transcribe.py end to end: the sequences that beam search returns are
scored again token by token, with one beam that is told what to say and whose
cache is never reordered.

Both runs hold the same keys and values (a row's tokens are quantised in the
same order); what differs is the rounding of activations to bf16 where sums
were cut differently.  A logit's rounding is 2^-8 of values of up to about 10
through a few layers: 0.1 a token is allowed.
"""
import importlib.util
import math
import pathlib

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    path = pathlib.Path(__file__).resolve().parents[1] / "examples" / "transcribe.py"
    spec = importlib.util.spec_from_file_location("transcribe_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("beams,tokens", [(1, 8), (4, 40)])
def test_beams_score_what_their_tokens_score(ex, beams, tokens):
    import log_mel_spectrogram_gb300 as lm
    model = ex.Model(seed=beams)
    wave = torch.randn(3, 16000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.1
    scores, said = ex.transcribe(model, wave, beams, tokens)
    assert scores.shape == (3, beams) and said.shape == (3, beams, tokens)
    assert (scores[:, :-1] >= scores[:, 1:]).all() and scores.isfinite().all()
    assert ((said >= 0) & (said < model.vocab)).all()
    eos = model.vocab - 1
    with torch.no_grad():
        frames = model.remember(model.encode(wave))
        for b in range(beams):
            own = lm.KvCache(3, tokens, model.heads, model.dim, layers=len(model.decoder), dtype=model.dtype)
            last = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
            total = torch.zeros(3, dtype=torch.float64, device="cuda")
            alive = torch.ones(3, dtype=torch.bool, device="cuda")
            for i in range(tokens):
                logp = torch.log_softmax(model.step(last, own, frames)[:, 0].double(), -1)
                last = said[:, b, i:i + 1].contiguous()
                total += torch.where(alive, logp.gather(1, last.long())[:, 0], 0.0)
                alive &= last[:, 0] != eos
            assert ((total - scores[:, b].double()).abs() <= 0.1 * tokens).all(), (total, scores[:, b])
    assert not math.isnan(float(total.sum()))


def test_the_decoder_step_can_be_captured(ex):
    """A decoding step as a CUDA graph gives what the same calls give."""
    model = ex.Model(seed=3)
    wave = torch.randn(2, 8000, device="cuda") * 0.1
    with torch.no_grad():
        import log_mel_spectrogram_gb300 as lm
        frames = model.remember(model.encode(wave))
        tokens = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32, device="cuda")
        eager = lm.KvCache(4, 32, model.heads, model.dim, layers=len(model.decoder), dtype=model.dtype)
        graphed = lm.KvCache(4, 32, model.heads, model.dim, layers=len(model.decoder), dtype=model.dtype)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            model.step(tokens, graphed, frames)  # warm-up
        torch.cuda.current_stream().wait_stream(s)
        graphed.lens.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = model.step(tokens, graphed, frames)
        graphed.lens.zero_()
        for _ in range(5):
            want = model.step(tokens, eager, frames)
            g.replay()
            assert torch.equal(got, want)
            tokens.add_(1)
