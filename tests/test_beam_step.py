"""beam_step() against its definition in 64 bits.

Tokens, parents, ended marks and histories have to be equal; inputs are drawn
until no two totals of different beams that the choice depends on are within
1e-4 of each other (or they are the same by construction).  Totals are sums of
32-bit values: off by 2^-21 of |score| + |logit| + |max| + |log z|, which the
tolerance 2e-6 * (1 + those) covers.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    import __graft_entry__
    __graft_entry__.build()
    import log_mel_spectrogram_gb300
    return log_mel_spectrogram_gb300


def reference(logits, scores, finished, eos):
    """Per clip: [(total, beam, token)], best first, and the smallest gap between beams around the choice."""
    x = logits.double().cpu()
    clips, beams, vocab = x.shape
    chosen, gap = [], math.inf
    for c in range(clips):
        offers = []
        for b in range(beams):
            s = float(scores[c, b])
            if finished is not None and finished[c, b]:
                offers += [(s if i == 0 else -math.inf, b, i, eos) for i in range(min(beams, vocab))]
                continue
            row = x[c, b]
            dead = bool((~(row < math.inf)).any()) or row.max() == -math.inf
            lse = 0.0 if dead else float(torch.logsumexp(row, 0))
            order = torch.sort(torch.zeros_like(row) if dead else row, descending=True, stable=True)[1][:beams].tolist()
            for i, t in enumerate(order):
                total = -math.inf if dead or math.isnan(s) else s + (float(row[t]) - lse)
                offers.append((total, b, i, t))
        offers.sort(key=lambda o: (-o[0], o[1], o[2]))
        near = offers[:beams + 1]
        for p, q in zip(near, near[1:]):
            if p[1] != q[1] and p[0] > -math.inf:
                gap = min(gap, p[0] - q[0])
        chosen.append([(o[0], o[1], o[3]) for o in offers[:beams]])
    return chosen, gap


def check(lm, logits, scores, finished=None, eos=None, width=0, length=0, need_gap=True):
    want, gap = reference(logits, scores, finished, eos)
    if need_gap:
        assert gap > 1e-4 or gap == 0
    clips, beams, vocab = logits.shape
    history = None
    if width:
        history = torch.randint(0, vocab, (clips, beams, width), device="cuda", dtype=torch.int32)
        kept = history.clone()
    step = lm.beam_step(logits, scores, finished, history, length, eos=eos)
    assert step.tokens.tolist() == [[o[2] for o in w] for w in want]
    assert step.parents.tolist() == [[o[1] for o in w] for w in want]
    tot = torch.tensor([[o[0] for o in w] for w in want], dtype=torch.float64)
    got = step.scores.double().cpu()
    big = 1 + scores.double().cpu().nan_to_num(0, 0, 0).abs().amax() + \
        2 * logits.double().nan_to_num(0, 0, 0).abs().amax().cpu()
    same = (got == tot) | ((got - tot).abs() <= 2e-6 * big)
    assert same.all()
    ended = [[bool(finished is not None and finished[c, o[1]]) or o[2] == eos for o in w] for c, w in enumerate(want)]
    assert step.finished.tolist() == ended
    if width:
        assert torch.equal(history, kept)
        told = torch.stack([kept[c, step.parents[c].long()] for c in range(clips)])
        told[..., length] = step.tokens
        assert torch.equal(step.history, told)
    else:
        assert step.history is None
    return step


def draw(clips, beams, vocab, dtype, seed, finished=False, spread=2.5):
    """Logits and scores whose choice does not hang on a near tie."""
    for s in range(seed * 1000, seed * 1000 + 200):
        g = torch.Generator(device="cuda").manual_seed(s)
        x = (torch.randn((clips, beams, vocab), generator=g, device="cuda") * spread).to(dtype)
        sc = -torch.rand((clips, beams), generator=g, device="cuda").mul_(15).sort(-1)[0]
        fin = torch.rand((clips, beams), generator=g, device="cuda") < 0.3 if finished else None
        if reference(x, sc, fin, vocab - 1)[1] > 1e-4:
            return x, sc, fin
    raise AssertionError("no inputs without near ties")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("clips,beams,vocab", [(1, 1, 1), (1, 5, 5), (2, 5, 3), (1, 5, 50001), (3, 8, 1000), (2, 16, 777),
                                               (1, 32, 2049), (4, 3, 8193), (2, 4, 131073), (7, 2, 64)])
def test_sizes(lm, dtype, clips, beams, vocab):
    x, sc, fin = draw(clips, beams, vocab, dtype, beams + vocab, finished=vocab > 40)
    check(lm, x, sc, fin, eos=vocab - 1, width=37, length=clips % 37)
    check(lm, *draw(clips, beams, vocab, dtype, beams + vocab + 1)[:2], width=3, length=2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_ties_go_to_the_lower_beam_and_token(lm, dtype):
    x = torch.zeros((2, 4, 3000), device="cuda", dtype=dtype)  # every token of every beam alike
    sc = torch.zeros((2, 4), device="cuda")
    step = check(lm, x, sc, need_gap=False)
    assert step.tokens.tolist() == [[0, 1, 2, 3]] * 2 and step.parents.tolist() == [[0] * 4] * 2
    x[:, :, 2999] = 1.0
    x[:, :, 17] = 1.0
    x[:, 0, 17] = -0.0
    x[:, 0, 2999] = 0.0
    check(lm, x, sc, need_gap=False)
    same = torch.arange(3000, device="cuda").remainder(40).to(dtype).expand(2, 4, 3000).contiguous()
    # Beam 0's four lowest tokens of the largest logit: its copies in other beams come later.
    step = check(lm, same, sc, need_gap=False)
    assert step.tokens.tolist() == [[39, 79, 119, 159]] * 2 and step.parents.tolist() == [[0] * 4] * 2


def test_the_first_step_and_dead_beams(lm):
    x, sc, _ = draw(3, 4, 999, torch.float32, 77)
    sc[:, 1:] = -math.inf
    step = check(lm, x, sc)
    assert (step.parents == 0).all()
    sc[1] = -math.inf
    check(lm, x, sc)
    sc[2, 1] = math.nan
    check(lm, x, sc)


def test_masked_logits_nan_and_infinity(lm):
    for s in range(5, 50):
        x, sc, _ = draw(4, 3, 600, torch.float32, s)
        x[0, :, 5:] = -math.inf                       # five tokens left
        x[1, 0] = -math.inf                           # nothing left
        x[1, 1, 9] = math.nan
        x[1, 2, 599] = math.inf
        x[2, 1, :] = torch.finfo(torch.float32).min   # the lowest value: a uniform beam
        x[3, 2, 1:] = -math.inf                       # one token, at no cost
        if reference(x, sc, None, None)[1] > 1e-4:
            break
    step = check(lm, x, sc)
    assert step.scores[1].tolist() == [-math.inf] * 3 and step.tokens[1].tolist() == [0, 1, 2]


def test_finished_beams(lm):
    x, sc, _ = draw(2, 4, 500, torch.bfloat16, 31)
    fin = torch.tensor([[True] * 4, [False, True, False, False]], device="cuda")
    x[0, 2, 3] = math.nan
    step = check(lm, x, sc, fin, eos=7, width=9, length=4)
    assert step.finished[0].all() and (step.tokens[0] == 7).all()
    x[1, 0, 7] = 40.0  # a live beam ends
    step = check(lm, x, sc, fin, eos=7)
    assert step.finished[1, step.tokens[1].tolist().index(7)]


def test_strided_rows_streams_and_graphs(lm):
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn((2, 5, 1003), generator=g, device="cuda").half()
    x = wide[:, :, 2:1001]
    sc = -torch.rand((2, 5), generator=g, device="cuda")
    want = lm.beam_step(x.contiguous(), sc)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        a, b = lm.beam_step(x, sc), lm.beam_step(x, sc, stream=s)
        s.synchronize()
        for p, q, r in zip(want[:4], a, b):
            assert torch.equal(p, q) and torch.equal(p, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lm.beam_step(x, sc)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want[:4], got):
            assert torch.equal(p, q)


def test_refusals(lm):
    x = torch.zeros((2, 3, 10), device="cuda")
    sc = torch.zeros((2, 3), device="cuda")
    fin = torch.zeros((2, 3), device="cuda", dtype=torch.bool)
    h = torch.zeros((2, 3, 4), device="cuda", dtype=torch.int32)
    for bad in (lambda: lm.beam_step(x.cpu(), sc), lambda: lm.beam_step(x[0], sc), lambda: lm.beam_step(x.int(), sc),
                lambda: lm.beam_step(x, sc[:1]), lambda: lm.beam_step(x, sc.half()), lambda: lm.beam_step(x, sc, fin),
                lambda: lm.beam_step(x, sc, fin.int(), eos=1), lambda: lm.beam_step(x, sc, eos=10),
                lambda: lm.beam_step(x, sc, None, h, 4), lambda: lm.beam_step(x, sc, None, h, -1),
                lambda: lm.beam_step(x, sc, None, h.long(), 0), lambda: lm.beam_step(x[:, :, ::2], sc),
                lambda: lm.beam_step(x.expand(2, 3, 10)[:, :2], sc[:, :2]),
                lambda: lm.beam_step(torch.zeros((1, 33, 40), device="cuda"), torch.zeros((1, 33), device="cuda"))):
        with pytest.raises((ValueError, lm.LogmelError)):
            bad()
    assert lm.beam_step(x[:0], sc[:0]).tokens.shape == (0, 3)
