"""Timed cases of the transcription operators: what follows the log-mel front end in a speech
model.  linear() projects feature frames and decoder states, KvCache holds keys and values in 8 bits
and attends over them, beam_step() picks the next tokens of every beam and the cache follows.

Each case is one pass through one operator.  run() has it in two forms: elementary torch operations in
32 bits (own = False), and the calls of this package (own = True).  exact() has the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decoder projection of one clip's five beams: latency, and 2 MB of weights.
        dict(name="linear step", op="linear", clips=1, rows=5, k=1024, n=1024, window=0, dtype="bf16", bias=True,
             act="none", residual=True, scale=1.0),
        # The output projection onto an odd vocabulary for 64 clips' beams of one step.
        dict(name="linear vocab", op="linear", clips=1, rows=320, k=1024, n=50001, window=0, dtype="f16", bias=False,
             act="none", residual=False, scale=1.0),
        # The encoder's first layer: windows of 3 frames of 80 mel bands, read in place from the padded
        # features of 8 clips of 3000 frames (the batch of the library's own STFT workload).
        dict(name="linear stem", op="linear", clips=8, rows=3000, k=240, n=512, window=80, dtype="f16", bias=True,
             act="gelu", residual=False, scale=1.0),
        # A feed-forward layer over the encoder frames of 16 clips.
        dict(name="linear frames", op="linear", clips=1, rows=24000, k=1024, n=4096, window=0, dtype="bf16",
             bias=True, act="gelu", residual=False, scale=1.0),
        # One decoding step of one clip's five beams over their own tokens.
        dict(name="attend step", op="attend", rows=5, t=1, q_heads=8, kv_heads=8, dim=64, block=32, tokens=448,
             causal=True, spread="ragged", dtype="f16"),
        # One decoding step of 64 clips, five beams each, over the encoder frames of clips of unequal length.
        dict(name="attend clips", op="attend", rows=64, t=5, q_heads=16, kv_heads=16, dim=64, block=32, tokens=1500,
             causal=False, spread="ragged", dtype="bf16"),
        # Two long recordings, one new token each, shared key heads.
        dict(name="attend long", op="attend", rows=2, t=1, q_heads=32, kv_heads=8, dim=128, block=64, tokens=131000,
             causal=True, spread="full", dtype="bf16"),
        # The prompts of 16 clips (earlier text), causal, of unequal length.
        dict(name="attend prompt", op="attend", rows=16, t=223, q_heads=16, kv_heads=16, dim=64, block=32, tokens=448,
             causal=True, spread="ragged", dtype="f16"),
        # One step's keys and values of 64 clips' beams into the cache, with the values of the blocks they fall in.
        dict(name="append step", op="append", rows=320, t=1, heads=16, dim=64, block=32, tokens=448, dtype="f16"),
        # The encoder frames of 64 clips of unequal length into the cache, with the values that it then holds.
        dict(name="append clips", op="append", rows=64, t=1500, heads=16, dim=64, block=32, tokens=1536,
             dtype="bf16"),
        # One beam step of one clip, with the cache of a 4-layer decoder.
        dict(name="beam step", op="beam", clips=1, beams=5, vocab=50001, length=100, width=448, layers=4, heads=8,
             dim=64, block=32, dtype="bf16", first=False),
        # The same for 64 clips.
        dict(name="beam clips", op="beam", clips=64, beams=5, vocab=50001, length=203, width=448, layers=4, heads=16,
             dim=64, block=32, dtype="f32", first=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "attend", "attend", "append", "beam"])
    big = {c["name"]: work(c) for c in listed()}
    while True:
        half = rng.choice(["f16", "bf16"])
        if op == "linear":
            window = rng.choice([0, 0, 0, 80, 128])
            c = dict(op=op, clips=rng.randint(1, 8) if window else 1, rows=_log(rng, 1, 24000),
                     k=3 * window if window else _log(rng, 16, 5000), n=_log(rng, 16, 50001), window=window, dtype=half,
                     bias=rng.random() < 0.7, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                     residual=rng.random() < 0.4, scale=rng.choice([1.0, 1.0, 0.5]))
            if not window and rng.random() < 0.7:
                c["k"] = max(16, c["k"] // 8 * 8)
            top = big["linear frames"]
        elif op == "attend":
            heads, group, dim = _log(rng, 1, 20), rng.choice([1, 1, 2, 4, 8]), rng.choice([32, 64, 64, 128])
            tokens = _log(rng, 1, 131000)
            t = rng.choice([1, 1, 1, 5, _log(rng, 1, 223)])
            c = dict(op=op, rows=_log(rng, 1, 320), t=min(t, tokens), q_heads=heads * group, kv_heads=heads, dim=dim,
                     block=rng.choice([16, 32, 64, 128]), tokens=tokens, causal=rng.random() < 0.6,
                     spread=rng.choice(["full", "ragged"]), dtype=half)
            top = big["attend long"]
        elif op == "append":
            t = rng.choice([1, 1, _log(rng, 1, 1500)])
            c = dict(op=op, rows=_log(rng, 1, 320), t=t, heads=_log(rng, 1, 20), dim=rng.choice([32, 64, 64, 128]),
                     block=rng.choice([16, 32, 64, 128]), tokens=t + rng.randint(0, 448), dtype=half)
            top = big["append clips"]
        else:
            beams, width = rng.randint(1, 16), rng.randint(8, 448)
            c = dict(op=op, clips=_log(rng, 1, 64), beams=beams, vocab=_log(rng, 50, 100001),
                     length=rng.randint(0, width - 1), width=width, layers=rng.randint(1, 6), heads=_log(rng, 1, 20),
                     dim=rng.choice([32, 64, 64, 128]), block=rng.choice([16, 32, 64]),
                     dtype=rng.choice(["f32", "f16", "bf16"]), first=rng.random() < 0.2)
            top = big["beam clips"]
        w = work(c)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return c


def _spread(case):
    """Tokens held per row before the step, and new ones, as lists: full rows, or unequal ones with an empty one."""
    rows, t, tokens = case["rows"], case["t"], case["tokens"]
    if case["op"] == "append":
        if t == 1:
            return [(tokens - 1) * (r % 7) // 7 for r in range(rows)], [1] * rows
        held = tokens - t
        new = [t - (t * (r % 5)) // 9 if r % 11 != 10 else 0 for r in range(rows)]
        return [held * (r % 4) // 4 for r in range(rows)], new
    new = [t] * rows
    if case["spread"] == "full" or rows == 1:
        total = [tokens] * rows
    else:
        total = [max(1, tokens - (tokens * (r % 8)) // 9) for r in range(rows)]
        total[-1] = 0 if not case["causal"] else total[-1]
    if case["causal"]:
        new = [min(n, s) for n, s in zip(new, total)]
        return [s - n for s, n in zip(total, new)], new
    return total, [0] * rows


def _window_blocks(case):
    return (case["t"] - 1 + case["block"] - 1) // case["block"] + 1


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantised(shape, gen, dev):
    """8-bit blocks [..., block, dim] and their scales, of normal values with a scale of its own per block."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
    x *= torch.rand(shape[:-2] + (1, 1), generator=gen, device=dev) + 0.5
    s = x.abs().amax((-1, -2)) / 127
    return torch.round(x / s[..., None, None]).to(torch.int8), s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    op = case["op"]
    st = dict(case)
    if op == "linear":
        dt = DTYPES[case["dtype"]]
        clips, rows, k, n, window = case["clips"], case["rows"], case["k"], case["n"], case["window"]
        if window:  # log-mel frames (about 0 to 1.5), padded by one frame on both sides
            x = torch.rand((clips, rows + 2, window), generator=gen, device=dev).mul_(1.5)
            x[:, 0] = 0
            x[:, -1] = 0
            x = x.to(dt)
            st["x"] = x.as_strided((clips, rows, k), ((rows + 2) * window, window, 1))
        else:
            st["x"] = randn(rows, k).to(dt)
        st["weight"] = (randn(n, k) / math.sqrt(k)).to(dt)
        st["bias_"] = randn(n) if case["bias"] else None
        lead = (clips, rows) if window else (rows,)
        st["residual_"] = randn(*lead, n).to(dt) if case["residual"] else None
        return st

    if op == "beam":
        clips, beams, vocab = case["clips"], case["beams"], case["vocab"]
        x = randn(clips, beams, vocab) * 2.5
        st["logits"] = x.to(DTYPES[case["dtype"]])
        st["logits"][..., vocab // 3:vocab // 3 + 7] = -math.inf  # suppressed tokens
        st["scores"] = -torch.rand((clips, beams), generator=gen, device=dev).mul_(20).sort(-1)[0]
        st["finished"] = torch.rand((clips, beams), generator=gen, device=dev) < 0.15
        if case["first"]:
            st["scores"][:, 1:] = -math.inf
            st["finished"][:] = False
        st["history"] = torch.randint(0, vocab, (clips, beams, case["width"]), generator=gen, device=dev,
                                      dtype=torch.int32)
        st["eos"] = vocab - 1
        rows, heads, layers, tokens = clips * beams, case["heads"], case["layers"], case["width"]
    else:
        rows, layers, tokens = case["rows"], 1, case["tokens"]
        heads = case["kv_heads"] if op == "attend" else case["heads"]
        dt = DTYPES[case["dtype"]]
        held, new = (torch.tensor(v, dtype=torch.int32, device=dev) for v in _spread(case))
        order = torch.randperm(rows, generator=gen, device=dev)
        held, new = held[order], new[order]

    block, dim = case["block"], case["dim"]
    width = -(-tokens // block)
    blocks = rows * (width + 1)
    order = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)  # blocks in no order
    table, spare = order[:rows * width].view(rows, width), order[rows * width:]
    shape = (layers, blocks, heads, block, dim)
    k8, ks = _quantised(shape, gen, dev)
    v8, vs = _quantised(shape, gen, dev)
    if op == "append":
        st["k"], st["v"] = (randn(rows, case["t"], heads, dim).to(dt) for _ in range(2))
    if op == "attend":
        st["q"] = (randn(rows, case["t"], case["q_heads"], dim) * 1.5).to(dt)
    if op == "beam":
        held, new = torch.full((rows,), case["length"], dtype=torch.int32, device=dev), None
    st["counts"] = new
    if own:  # the handle that a user's program keeps; the same contents
        import log_mel_spectrogram_gb300 as lm
        cache = lm.KvCache(rows, tokens, heads, dim, layers=layers, block=block,
                           dtype=torch.bfloat16 if op == "beam" else dt, device=dev)
        for a, b in ((cache.k8, k8), (cache.v8, v8), (cache.k_scale, ks), (cache.v_scale, vs), (cache.table, table),
                     (cache.spare, spare), (cache.lens, held)):
            a.copy_(b)
        st["cache"] = cache
    else:
        st.update(k8=k8, v8=v8, ks=ks, vs=vs, table=table.clone(), spare=spare.clone(), lens=held)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _calls(s) if own else _plain(s)


def _calls(s):
    import log_mel_spectrogram_gb300 as lm
    op = s["op"]
    if op == "linear":
        return lm.linear(s["x"], s["weight"], s["bias_"], activation=None if s["act"] == "none" else s["act"],
                         residual=s["residual_"], scale=s["scale"])
    cache = s["cache"]
    if op == "attend":
        return cache.attend(0, s["q"], s["counts"], causal=s["causal"])
    if op == "append":
        return cache.append(0, s["k"], s["v"], s["counts"], values=True)
    step = lm.beam_step(s["logits"], s["scores"], s["finished"], s["history"], s["length"], eos=s["eos"])
    cache.reorder(step.parents)
    k, v = cache.read(None, s["length"] // s["block"] * s["block"], s["block"])
    return {**step._asdict(), "table": cache.table, "spare": cache.spare, "k": k, "v": v}


def _act(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y / (1 + torch.exp(-y)) if act == "silu" else y


def _plain(s):
    op = s["op"]
    if op == "linear":
        y = s["x"].float() @ s["weight"].float().t()
        if s["bias_"] is not None:
            y = y + s["bias_"]
        y = _act(y, s["act"]) * s["scale"]
        if s["residual_"] is not None:
            y = s["residual_"].float() + y
        return y.to(s["x"].dtype)
    if op == "attend":
        return _plain_attend(s)
    if op == "append":
        return tuple(_plain_append(s, *n) for n in (("k", "k8", "ks"), ("v", "v8", "vs")))
    return _plain_beam(s)


def _plain_attend(s):
    q, table, lens, new = s["q"], s["table"].long(), s["lens"], s["counts"]
    rows, t, hq, d = q.shape
    h = s["kv_heads"]

    def held(x8, scale):  # [rows, heads, tokens, dim]
        x = x8[0][table].float() * scale[0][table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(rows, h, -1, d)[:, :, :s["tokens"]]

    keys, values = held(s["k8"], s["ks"]), held(s["v8"], s["vs"])
    qf = q.float().reshape(rows, t, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(rows, h, -1, d)
    x = qf @ keys.transpose(-1, -2) / math.sqrt(d)
    at = torch.arange(x.shape[-1], device=q.device)
    i = torch.arange(t, device=q.device)
    total = lens + new
    if s["causal"]:
        seen = (at[None, None] <= (lens[:, None] + i)[..., None]) & (i < new[:, None])[..., None]
    else:
        seen = (at[None, None] < total[:, None, None]).expand(rows, t, -1)
    seen = seen[:, None, None].expand(rows, h, hq // h, t, -1).reshape(rows, h, -1, x.shape[-1])
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(-1, keepdim=True)
    o = torch.where(z > 0, (p @ values) / z, 0.0)
    return o.reshape(rows, h, hq // h, t, d).permute(0, 3, 1, 2, 4).reshape(rows, t, hq, d).to(q.dtype)


def _plain_append(s, name, name8, name_s):
    """New tokens into their blocks: a block's scale grows to its largest value / 127, and what the block held
    before is rounded anew where it grew.  Returns the values that the touched blocks now stand for."""
    x, table, lens, new, bs = s[name], s["table"].long(), s["lens"].long(), s["counts"].long(), s["block"]
    rows, t, h, d = x.shape
    x8, scale = s[name8][0], s[name_s][0]
    wide = _window_blocks(s)
    first = lens // bs
    at = first[:, None] + torch.arange(wide, device=x.device)  # the blocks' places in the rows
    touched = at * bs < (lens + new)[:, None]
    pages = table.gather(1, at.clamp(max=table.shape[1] - 1))  # [rows, wide]
    token = at[:, :, None] * bs + torch.arange(bs, device=x.device)  # [rows, wide, bs]
    i = token - lens[:, None, None]
    is_old, is_new = i < 0, (i >= 0) & (i < new[:, None, None])
    fresh = x.float()[torch.arange(rows, device=x.device)[:, None, None], i.clamp(0, t - 1)]  # [rows, wide, bs, h, d]
    fresh = torch.where(is_new[..., None, None], fresh, 0.0).transpose(2, 3)  # [rows, wide, h, bs, d]
    before = torch.where(is_old.any(-1)[..., None], scale[pages], 0.0)  # [rows, wide, h]
    now = torch.maximum(before, fresh.abs().amax((-1, -2)) / 127)
    now = torch.where(now > 0, now, 1.0)
    was8 = x8[pages]
    kept = torch.round(was8.float() * (before / now)[..., None, None])
    got = torch.round(fresh / now[..., None, None])
    old_, new_ = is_old[:, :, None, :, None], is_new[:, :, None, :, None]
    x8n = torch.where(old_, kept, torch.where(new_, got, was8.float())).to(torch.int8)
    x8[pages[touched]] = x8n[touched]
    scale[pages[touched]] = now[touched]
    value = torch.where(old_ | new_, x8n.float() * now[..., None, None], 0.0)
    value = torch.where(touched[:, :, None, None, None] & (token < (lens + new)[:, None, None])[:, :, None, :, None],
                        value, 0.0)
    return value.transpose(2, 3).reshape(rows, wide * bs, h, d).to(x.dtype)


def _plain_beam(s):
    x, scores, finished, history = s["logits"].float() + 0.0, s["scores"], s["finished"], s["history"]
    b, k, v = x.shape
    n = min(k, v)
    m = x.amax(-1, keepdim=True)
    live = torch.isfinite(m)
    m = torch.where(live, m, 0.0)
    logz = torch.log(torch.exp(x - m).sum(-1, keepdim=True))
    best, token = torch.sort(torch.where(live, x, -math.inf), dim=-1, descending=True, stable=True)
    best, token = best[..., :n], token[..., :n].to(torch.int32)
    total = scores[..., None] + ((best - m) - logz)
    total = torch.where(live & ~torch.isnan(total), total, -math.inf)
    done = torch.full_like(total, -math.inf)
    done[..., 0] = scores
    total = torch.where(finished[..., None], done, total)
    token = torch.where(finished[..., None], s["eos"], token)
    total, order = torch.sort(total.reshape(b, -1), dim=-1, descending=True, stable=True)
    total, order = total[:, :k], order[:, :k]
    parents = order // n
    tokens = token.reshape(b, -1).gather(1, order)
    ended = finished.gather(1, parents) | (tokens == s["eos"])
    told = history.gather(1, parents[..., None].expand(-1, -1, history.shape[-1]))
    told[..., s["length"]] = tokens

    # the cache follows: whole blocks are shared through the table, the open block is copied to the row's spare
    table, spare, bs = s["table"], s["spare"], s["block"]
    rows, wide = table.shape
    from_ = (torch.arange(b, device=x.device)[:, None] * k + parents).reshape(-1)
    j, part = s["length"] // bs, s["length"] % bs
    moved = from_ != torch.arange(rows, device=x.device)
    was, old_spare = table.clone(), spare.clone()
    col = torch.arange(wide, device=x.device)
    table.copy_(torch.where(col[None] < j, was[from_], was))
    if part:
        to, source = old_spare[moved].long(), was[from_, j][moved].long()
        s["k8"][:, to], s["v8"][:, to] = s["k8"][:, source], s["v8"][:, source]
        s["ks"][:, to], s["vs"][:, to] = s["ks"][:, source], s["vs"][:, source]
        table[:, j] = torch.where(moved, old_spare, was[:, j])
        spare.copy_(torch.where(moved, was[:, j], old_spare))
    return {"scores": total, "tokens": tokens, "parents": parents.to(torch.int32), "finished": ended, "history": told,
            "table": table, "spare": spare, "k": _plain_read(s, "k8", "ks"), "v": _plain_read(s, "v8", "vs")}


def _plain_read(s, name8, name_s):
    j, bs = s["length"] // s["block"], s["block"]
    pages = s["table"][:, j].long()
    x = s[name8][:, pages].float() * s[name_s][:, pages][..., None, None]  # [layers, rows, heads, block, dim]
    x = torch.where((torch.arange(bs, device=x.device) < s["length"] % bs)[:, None], x, 0.0)
    return x.transpose(2, 3).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"linear": _exact_linear, "attend": _exact_attend, "append": _exact_append, "beam": _exact_beam}[case["op"]](s)


def _exact_linear(s):
    y = torch.einsum("...k,nk->...n", s["x"].double(), s["weight"].double())
    y = y if s["bias_"] is None else y + s["bias_"].double()
    a = s["act"]
    if a == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif a == "gelu":
        y = y * (1 - 0.5 * torch.erfc(y * 0.5 ** 0.5))
    elif a == "gelu_tanh":
        y = y * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3))
    elif a == "silu":
        y = y * torch.sigmoid(y)
    y = s["scale"] * y
    return y if s["residual_"] is None else y + s["residual_"].double()


def _row(s, name8, name_s, row, tokens, layer=0):
    """The first `tokens` tokens of a row as [tokens, heads, dim] doubles."""
    pages = s["table"][row].long()[:-(-tokens // s["block"])]
    x = s[name8][layer, pages].double() * s[name_s][layer, pages].double()[..., None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1)[:tokens]


def _exact_attend(s):
    q = s["q"].double()
    rows, t, hq, d = q.shape
    group = hq // s["kv_heads"]
    out = torch.zeros_like(q)
    for r in range(rows):
        held, new = int(s["lens"][r]), int(s["counts"][r])
        total = held + new
        if not total:
            continue
        keys, values = _row(s, "k8", "ks", r, total), _row(s, "v8", "vs", r, total)
        for h in range(s["kv_heads"]):
            heads = slice(h * group, (h + 1) * group)
            count = new if s["causal"] else t
            x = torch.einsum("igd,ld->igl", q[r, :count, heads], keys[:, h]) * d ** -0.5
            if s["causal"]:
                late = torch.arange(total, device=q.device)[None] > held + torch.arange(count, device=q.device)[:, None]
                x = torch.where(late[:, None], -math.inf, x)
            out[r, :count, heads] = torch.softmax(x, -1) @ values[:, h]
    return out


def _exact_append(s):
    bs, out = s["block"], []
    for name, name8, name_s in (("k", "k8", "ks"), ("v", "v8", "vs")):
        x = s[name]
        rows, t, h, d = x.shape
        wide = _window_blocks(s)
        val = torch.zeros((rows, wide * bs, h, d), dtype=torch.float64, device=x.device)
        for r in range(rows):
            held, new = int(s["lens"][r]), int(s["counts"][r])
            base, pad = held // bs * bs, held % bs
            n = pad + new
            blocks = -(-n // bs)
            if not blocks:
                continue
            y = torch.zeros((blocks * bs, h, d), dtype=torch.float64, device=x.device)
            y[pad:n] = x[r, :new].double()
            grown = y.view(blocks, bs, h, d).abs().amax((1, 3)) / 127
            if pad:
                page = int(s["table"][r, held // bs])
                before = s[name_s][0, page].double()
                grown[0] = torch.maximum(grown[0], before)
                was = s[name8][0, page].double()[:, :pad].transpose(0, 1)
                y[:pad] = torch.round(was * (before / grown[0])[:, None]) * grown[0][:, None]
            grown = torch.where(grown > 0, grown, 1.0).repeat_interleave(bs, 0)[..., None]
            y[pad:] = (torch.round(y / grown) * grown)[pad:]
            val[r, :n] = y[:n]
        out.append(val)
    return tuple(out)


def _exact_beam(s):
    logp = torch.log_softmax(s["logits"].double(), -1)
    best, token = logp.topk(min(logp.shape[1], logp.shape[2]), -1)
    total = s["scores"].double()[..., None] + best
    total = torch.where(s["finished"][..., None], -math.inf, total)
    total[..., 0] = torch.where(s["finished"], s["scores"].double(), total[..., 0])
    scores, order = total.flatten(1).topk(total.shape[1], -1)
    parents = order // total.shape[2]
    k, v = [], []
    rows = parents.shape[0] * parents.shape[1]
    from_ = (parents + torch.arange(parents.shape[0], device=parents.device)[:, None] * parents.shape[1]).flatten().tolist()
    bs, length = s["block"], s["length"]
    for name8, name_s, to in (("k8", "ks", k), ("v8", "vs", v)):
        page = s["table"][from_, length // bs].long()
        x = s[name8][:, page].double() * s[name_s][:, page].double()[..., None, None]
        x[:, :, :, length % bs:] = 0
        to.append(x.transpose(2, 3).reshape(x.shape[0], rows, bs, x.shape[2], x.shape[4]))
    return {"scores": scores, "tokens": None, "parents": None, "finished": None, "history": None, "table": None,
            "spare": None, "k": k[0], "v": v[0]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "linear":
        m, k, n = case["clips"] * case["rows"], case["k"], case["n"]
        x = case["clips"] * (case["rows"] + 2) * case["window"] if case["window"] else m * k
        return {"bytes": 2 * (x + n * k + m * n * (2 if case["residual"] else 1)) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    bs, dim = case["block"], case["dim"]
    if op == "beam":
        rows = case["clips"] * case["beams"]
        size = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
        block = case["layers"] * case["heads"] * (bs * dim + 4)
        used = min(1.0, (case["length"] % bs) / bs)
        return {"bytes": rows * case["vocab"] * size + rows * case["width"] * 8 + rows * 26
                + int(rows * 2 * block * used) + rows * 2 * case["layers"] * case["heads"] * bs * dim * 2,
                "flops": 4 * rows * case["vocab"]}
    held, new = _spread(case)
    if op == "append":
        h = case["heads"]
        parts = sum(n % bs for n in held)  # tokens already in the open blocks
        blocks = sum(-(-(p % bs + n) // bs) for p, n in zip(held, new))
        out = case["rows"] * _window_blocks(case) * bs
        return {"bytes": 2 * h * (sum(new) * dim * 3 + parts * dim + blocks * 4 + out * dim * 2),
                "flops": 2 * h * dim * 4 * (sum(new) + parts)}
    hq, h, t = case["q_heads"], case["kv_heads"], case["t"]
    total = [a + b for a, b in zip(held, new)]
    blocks = sum(-(-n // bs) for n in total)
    if case["causal"]:
        pairs = sum(sum(a + i + 1 for i in range(b)) for a, b in zip(held, new))
    else:
        pairs = sum(n * t for n in total)
    return {"bytes": 2 * h * (sum(total) * dim + 4 * blocks) + 4 * blocks + case["rows"] * (t * hq * dim * 4 + 8),
            "flops": 4 * hq * dim * pairs}
