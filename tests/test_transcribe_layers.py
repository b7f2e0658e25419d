"""examples/transcribe.py with gated feed-forward layers and weights in 4 bits: it runs, and a decoding step can be
captured and gives what the same calls give."""
import pytest
import torch

from test_transcribe_example import ex  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated,four_bits", [(True, False), (False, True), (True, True)])
def test_runs(ex, gated, four_bits):  # noqa: F811
    model = ex.Model(seed=5, gated=gated, four_bits=four_bits)
    wave = torch.randn(2, 8000, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) * 0.1
    scores, said = ex.transcribe(model, wave, 4, 12)
    again, said2 = ex.transcribe(model, wave, 4, 12)
    assert scores.shape == (2, 4) and said.shape == (2, 4, 12) and scores.isfinite().all()
    assert (scores[:, :-1] >= scores[:, 1:]).all() and ((said >= 0) & (said < model.vocab)).all()
    assert torch.equal(scores, again) and torch.equal(said, said2)


def test_a_step_can_be_captured(ex):  # noqa: F811
    import log_mel_spectrogram_gb300 as lm
    model = ex.Model(seed=6, gated=True, four_bits=True)
    wave = torch.randn(2, 8000, device="cuda") * 0.1
    tokens = torch.randint(0, model.vocab, (2, 3), device="cuda")
    with torch.no_grad():
        frames = model.remember(model.encode(wave))
        own = lm.KvCache(6, 32, model.heads, model.dim, layers=len(model.decoder), dtype=model.dtype)
        want = model.step(tokens, own, frames)
        own.reset()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = model.step(tokens, own, frames)
        own.reset()
        graph.replay()
    assert torch.equal(got, want)
