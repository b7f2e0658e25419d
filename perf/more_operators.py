"""Timed cases of what stands around attention in the layers of a speech model: layer_norm() and
gated_linear(), forward and with their gradients, and linear() with weights in 4 bits.

Each case is one pass through one operator.  run() has it in two forms: elementary torch operations in
32 bits (own = False), and the calls of this package (own = True).  exact() has the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # The norm in front of a decoder projection of one clip's five beams: latency.
        dict(name="norm step", op="norm", rows=5, width=1024, train=False, dtype="bf16", wtype="f32"),
        # The norm over the encoder frames of 16 clips.
        dict(name="norm frames", op="norm", rows=24000, width=1024, train=False, dtype="f16", wtype="f16"),
        # The same in training, with the gradients of x, weight and bias.
        dict(name="norm train", op="norm", rows=24000, width=1024, train=True, dtype="bf16", wtype="f32"),
        # One clip's frames in 32 bits, of an odd width whose rows lie off every vector's boundary.
        dict(name="norm odd", op="norm", rows=1499, width=771, train=True, dtype="f32", wtype="f32"),
        # The gated feed-forward block of one decoding step of one clip's beams: 16 MB of weights.
        dict(name="gated step", op="gated", rows=5, k=1024, n=4096, act="silu", bias=False, train=False, dtype="bf16"),
        # The same over the encoder frames of 16 clips.
        dict(name="gated frames", op="gated", rows=24000, k=1024, n=4096, act="silu", bias=False, train=False,
             dtype="bf16"),
        # A training step over the frames of 8 clips: the block's output and all gradients.
        dict(name="gated train", op="gated", rows=12000, k=1024, n=4096, act="silu", bias=False, train=True,
             dtype="bf16"),
        # A small training step of odd sizes, with biases.
        dict(name="gated odd", op="gated", rows=777, k=500, n=1001, act="gelu", bias=True, train=True, dtype="f16"),
        # A decoder layer's first feed-forward projection for one clip's five beams.
        dict(name="linear4 step", op="linear4", rows=5, k=1024, n=4096, group=64, bias=True, act="gelu",
             residual=False, scale=1.0, dtype="bf16"),
        # The output projection onto an odd vocabulary for the same.
        dict(name="linear4 vocab", op="linear4", rows=5, k=1024, n=50001, group=128, bias=False, act="none",
             residual=False, scale=1.0, dtype="f16"),
        # The second feed-forward projection for 64 clips' beams.
        dict(name="linear4 beams", op="linear4", rows=320, k=4096, n=1024, group=64, bias=True, act="none",
             residual=True, scale=1.0, dtype="bf16"),
        # The first one over the encoder frames of two clips.
        dict(name="linear4 frames", op="linear4", rows=3000, k=1024, n=4096, group=32, bias=True, act="gelu",
             residual=False, scale=1.0, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "linear4"])
    all_ = [work(c) for c in listed() if c["op"] == op]
    most = {key: max(w[key] for w in all_) for key in ("bytes", "flops")}
    while True:
        half = rng.choice(["f16", "bf16"])
        if op == "norm":
            dtype = rng.choice(["f32", half, half])
            c = dict(op=op, rows=_log(rng, 1, 24000), width=_log(rng, 1, 8192), train=rng.random() < 0.6, dtype=dtype,
                     wtype=rng.choice(["f32", dtype]))
            if rng.random() < 0.5 and c["width"] > 8:
                c["width"] = c["width"] // 8 * 8
        elif op == "gated":
            c = dict(op=op, rows=_log(rng, 1, 24000), k=_log(rng, 16, 4096), n=_log(rng, 16, 8192),
                     act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu", "sigmoid", "none"]),
                     bias=rng.random() < 0.5, train=rng.random() < 0.5, dtype=half)
            if rng.random() < 0.6:
                c["k"], c["n"] = max(16, c["k"] // 8 * 8), max(16, c["n"] // 8 * 8)
        else:
            group = rng.choice([32, 64, 128])
            c = dict(op=op, rows=_log(rng, 1, 3000), k=_log(rng, 32, 8192), n=_log(rng, 16, 50001), group=group,
                     bias=rng.random() < 0.7, act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]),
                     residual=rng.random() < 0.4, scale=rng.choice([1.0, 1.0, 0.5]), dtype=half)
            if rng.random() < 0.7:
                c["k"] = max(group, c["k"] // group * group)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=gen, device=dev)  # noqa: E731
    op, rows, dt = case["op"], case["rows"], DTYPES[case["dtype"]]
    st = dict(case)
    if op == "norm":
        # A residual stream: rows of unequal size, off zero, with a few large channels.
        width = case["width"]
        x = randn(rows, width) * (rand(rows, 1) * 2.5 + 0.5) + 0.3 * randn(rows, 1)
        st["x"] = (x * torch.where(rand(width) < 0.01, 10.0, 1.0)).to(dt)
        wt = DTYPES[case["wtype"]]
        st["weight"], st["shift"] = (1 + 0.2 * randn(width)).to(wt), (0.2 * randn(width)).to(wt)
        leaves = ["x", "weight", "shift"]
        shape = (rows, width)
    elif op == "gated":
        k, n = case["k"], case["n"]
        st["x"] = randn(rows, k).to(dt)
        st["w_gate"], st["w_up"] = ((randn(n, k) / math.sqrt(k)).to(dt) for _ in range(2))
        leaves = ["x", "w_gate", "w_up"]
        st["b_gate"], st["b_up"] = (0.3 * randn(n) if case["bias"] else None for _ in range(2))
        leaves += ["b_gate", "b_up"] if case["bias"] else []
        shape = (rows, n)
    else:
        k, n, group = case["k"], case["n"], case["group"]
        st["x"] = randn(rows, k).to(dt)
        q = torch.randint(-7, 8, (n, k), generator=gen, device=dev, dtype=torch.int8)
        s = (rand(n, -(-k // group)) + 0.5) * (0.25 / math.sqrt(k))  # so that values are about 1 / sqrt(k)
        st["bias_"] = randn(n) if case["bias"] else None
        st["residual_"] = randn(rows, n).to(dt) if case["residual"] else None
        if own:  # the weight as a user's program keeps it
            import log_mel_spectrogram_gb300 as lm
            st["weight"] = lm.Weight4.pack(q, s, dtype=dt)
        else:
            st["q"], st["s"] = q, s
        return st
    if case["train"]:
        st["grad"] = randn(*shape).to(dt)
        st["leaves"] = leaves
        if own:
            for name in leaves:
                st[name].requires_grad_()
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _calls(s) if own else _plain(s)


def _calls(s):
    import log_mel_spectrogram_gb300 as lm
    op = s["op"]
    if op == "linear4":
        return lm.linear(s["x"], s["weight"], s["bias_"], activation=None if s["act"] == "none" else s["act"],
                         residual=s["residual_"], scale=s["scale"])
    if op == "norm":
        y = lm.layer_norm(s["x"], s["weight"], s["shift"], eps=1e-5)
    else:
        y = lm.gated_linear(s["x"], s["w_gate"], s["w_up"], s["b_gate"], s["b_up"],
                            activation=None if s["act"] == "none" else s["act"])
    if not s["train"]:
        return y
    return (y.detach(), *torch.autograd.grad(y, [s[name] for name in s["leaves"]], s["grad"]))


def _act(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-y))
    return y / (1 + torch.exp(-y)) if act == "silu" else y


def _slope(y, act):
    """The activation's derivative."""
    if act == "relu":
        return (y > 0).to(y.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(y / math.sqrt(2))) + y * torch.exp(-0.5 * y * y) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (y + 0.044715 * y * y * y))
        return 0.5 * (1 + t) + 0.5 * y * (1 - t * t) * c * (1 + 3 * 0.044715 * y * y)
    p = 1 / (1 + torch.exp(-y))
    if act == "sigmoid":
        return p * (1 - p)
    return p * (1 + y * (1 - p)) if act == "silu" else torch.ones_like(y)


def _plain(s):
    op, dt = s["op"], s["x"].dtype
    x = s["x"].float()
    if op == "linear4":
        w = s["q"].float() * s["s"].repeat_interleave(s["group"], 1)[:, :s["k"]]
        y = x @ w.t()
        if s["bias_"] is not None:
            y = y + s["bias_"]
        y = _act(y, s["act"]) * s["scale"]
        if s["residual_"] is not None:
            y = s["residual_"].float() + y
        return y.to(dt)
    if op == "norm":
        w = s["weight"].float()
        d = x - x.mean(-1, keepdim=True)
        r = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)
        n = d * r
        y = (n * w + s["shift"].float()).to(dt)
        if not s["train"]:
            return y
        g = s["grad"].float()
        gw = g * w
        dx = r * (gw - gw.mean(-1, keepdim=True) - n * (gw * n).mean(-1, keepdim=True))
        wt = s["weight"].dtype
        return y, dx.to(dt), (g * n).sum(0).to(wt), g.sum(0).to(wt)
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    a, b = x @ wg.t(), x @ wu.t()
    if s["bias"]:
        a, b = a + s["b_gate"], b + s["b_up"]
    act = _act(a, s["act"])
    y = (act * b).to(dt)
    if not s["train"]:
        return y
    g = s["grad"].float()
    da, db = g * b * _slope(a, s["act"]), g * act
    out = [y, (da @ wg + db @ wu).to(dt), (da.t() @ x).to(dt), (db.t() @ x).to(dt)]
    if s["bias"]:
        out += [da.sum(0), db.sum(0)]
    return tuple(out)


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
    if case["op"] == "linear4":
        return _exact_linear4(s)
    names = s.get("leaves", [])
    t = {name: s[name].double().requires_grad_(name in names)
         for name in ("x", "weight", "shift", "w_gate", "w_up", "b_gate", "b_up") if s.get(name) is not None}
    with torch.enable_grad():
        y = (_exact_norm if case["op"] == "norm" else _exact_gated)(t, s)
    if not case["train"]:
        return y.detach()
    return (y.detach(), *torch.autograd.grad(y, [t[name] for name in names], s["grad"].double()))


def _exact_norm(t, s):
    var, mean = torch.var_mean(t["x"], -1, keepdim=True, correction=0)
    return (t["x"] - mean) * torch.rsqrt(var + 1e-5) * t["weight"] + t["shift"]


def _exact_act(z, a):
    if a == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if a == "gelu":
        return z * (1 - 0.5 * torch.erfc(z * 0.5 ** 0.5))
    if a == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if a == "sigmoid":
        return torch.sigmoid(z)
    return z * torch.sigmoid(z) if a == "silu" else z


def _exact_gated(t, s):
    a, b = (torch.einsum("rk,nk->rn", t["x"], t[w]) for w in ("w_gate", "w_up"))
    if s["bias"]:
        a, b = a + t["b_gate"], b + t["b_up"]
    return _exact_act(a, s["act"]) * b


def _exact_linear4(s):
    group, k = s["group"], s["k"]
    y = torch.zeros((s["rows"], s["n"]), dtype=torch.float64, device=s["x"].device)
    if k % group == 0:
        q = s["q"].double().view(s["n"], -1, group) * s["s"].double()[..., None]
        y += torch.einsum("rk,nk->rn", s["x"].double(), q.view(s["n"], k))
    else:
        for i in range(s["s"].shape[1]):
            at = slice(i * group, min(k, (i + 1) * group))
            y += torch.einsum("rk,nk->rn", s["x"][:, at].double(), s["q"][:, at].double()) * s["s"][:, i].double()
    if s["bias_"] is not None:
        y = y + s["bias_"].double()
    y = s["scale"] * _exact_act(y, s["act"])
    return y if s["residual_"] is None else y + s["residual_"].double()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, rows, size, train = case["op"], case["rows"], SIZES[case["dtype"]], case.get("train")
    if op == "norm":
        c, ws = case["width"], SIZES[case["wtype"]]
        return {"bytes": rows * c * size * (4 if train else 2) + c * ws * (4 if train else 2),
                "flops": rows * c * (20 if train else 8)}
    k, n = case["k"], case["n"]
    if op == "gated":
        each = rows * k + 2 * n * k  # x and the weights, or their gradients
        bias = 8 * n if case["bias"] else 0
        return {"bytes": size * (each * (2 if train else 1) + rows * n * (2 if train else 1)) + bias * (2 if train else 1),
                "flops": 4 * rows * n * k * (3 if train else 1)}
    groups = -(-k // case["group"])
    return {"bytes": size * (rows * k + rows * n * (2 if case["residual"] else 1)) + n * -(-k // 2) + 4 * n * groups
            + (4 * n if case["bias"] else 0), "flops": 2 * rows * n * k}
