"""The decoding operations and differentiation: refused in both directions, and outputs that they write into count
as written."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import test_kv_cache as kv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


@pytest.fixture
def data(lm):
    r = kv.gen(1)
    c = kv.filled(lm, 2, 64, 2, 64, 32, torch.float16)
    return dict(x=r(4, 64).half(), w=r(32, 64).half(), bias=r(32), res=r(4, 32).half(), c=c, q=r(2, 1, 2, 64).half(),
                logits=r(2, 3, 50), scores=r(2, 3))


def calls(lm, d):
    """name of the argument, call with it replaced."""
    x, w, b, r, c, q = (d[k] for k in ("x", "w", "bias", "res", "c", "q"))
    yield x, lambda t: lm.linear(t, w)
    yield w, lambda t: lm.linear(x, t)
    yield b, lambda t: lm.linear(x, w, t)
    yield r, lambda t: lm.linear(x, w, residual=t)
    yield torch.empty_like(r), lambda t: lm.linear(x, w, out=t)
    yield q, lambda t: c.append(0, t, q)
    yield q, lambda t: c.append(0, q, t)
    yield q, lambda t: c.attend(0, t)
    yield torch.empty_like(q), lambda t: c.attend(0, q, out=t)
    yield d["logits"], lambda t: lm.beam_step(t, d["scores"])
    yield d["scores"], lambda t: lm.beam_step(d["logits"], t)


def test_tensors_that_require_grad_are_refused(lm, data):
    for t, f in calls(lm, data):
        t = t.clone().requires_grad_()
        with pytest.raises(RuntimeError, match="inference-only"):
            f(t)
        with torch.no_grad():
            f(t)
        f(t.detach())


def test_tangents_are_refused(lm, data):
    for t, f in calls(lm, data):
        with fwd.dual_level():
            dual = fwd.make_dual(t, torch.ones_like(t))
            with pytest.raises(RuntimeError, match="inference-only"):
                f(dual)
            with torch.no_grad(), pytest.raises(RuntimeError, match="inference-only"):
                f(dual)
            f(fwd.unpack_dual(dual).primal)
        f(t)


def test_outputs_count_as_written(lm, data):
    x, w, c, q = (data[k] for k in ("x", "w", "c", "q"))
    for shape, f in (((4, 32), lambda o: lm.linear(x, w, out=o)), ((2, 1, 2, 64), lambda o: c.attend(0, q, out=o))):
        out = torch.ones(shape, device="cuda", dtype=torch.float16)
        leaf = torch.ones(shape, device="cuda", requires_grad=True)
        y = (leaf * out.float().square()).sum() + (leaf * out).sum()  # saves out
        f(out)
        assert out._version == 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
        with torch.inference_mode():
            kept = torch.ones(shape, device="cuda", dtype=torch.float16)
        f(kept)  # no version to count
        assert torch.equal(kept, out)
        with torch.inference_mode():
            assert torch.equal(f(torch.empty_like(out)), out)
