"""What is measured of the second set of a training block's operators: the
gated feed-forward block (dense, or one per expert), rotary positions, and
dropout whose mask is never stored.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the package's operators.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # --- gated feed-forward (x, weights and outputs bf16) ---
        # five tokens through an expert-sized block: the launches are what counts
        dict(name="ffn_fwd_5_2048x768", op="ffn", dir="fwd", tokens=5, hidden=2048, inner=768,
             experts=0, act="silu"),
        # a shared expert (7168 -> 2048) over an odd number of tokens, kept for the backward pass
        dict(name="ffn_keep_4097_7168x2048", op="ffn", dir="keep", tokens=4097, hidden=7168, inner=2048,
             experts=0, act="silu"),
        # and its backward pass
        dict(name="ffn_bwd_4097_7168x2048", op="ffn", dir="bwd", tokens=4097, hidden=7168, inner=2048,
             experts=0, act="silu"),
        # a dense block's training step over a large batch
        dict(name="ffn_both_8192_4096x11008", op="ffn", dir="both", tokens=8192, hidden=4096, inner=11008,
             experts=0, act="gelu_tanh"),
        # 128 experts of 2048 -> 768: 8192 tokens, 8 experts each, both ways
        dict(name="ffn_fwd_128_experts", op="ffn", dir="fwd", tokens=65536, hidden=2048, inner=768,
             experts=128, act="silu"),
        dict(name="ffn_bwd_128_experts", op="ffn", dir="bwd", tokens=65536, hidden=2048, inner=768,
             experts=128, act="silu"),
        # --- rotary positions of queries and keys ---
        # a few tokens, 32 and 4 heads of 128
        dict(name="rotary_3x32x128", op="rotary", dir="fwd", batch=1, seq=3, heads=32, kheads=4, head=128,
             dim=128, layout="half", scaling="none", factor=1.0, far=0, dtype="bf16"),
        # a batch of sequences, counted positions
        dict(name="rotary_4x4096x32x128", op="rotary", dir="fwd", batch=4, seq=4096, heads=32, kheads=4,
             head=128, dim=128, layout="half", scaling="none", factor=1.0, far=0, dtype="bf16"),
        # the gradient of 64 heads of which 64 values of 192 turn, in pairs, at far positions of a
        # context stretched 32 times
        dict(name="rotary_bwd_8191x64x192", op="rotary", dir="bwd", batch=1, seq=8191, heads=64, kheads=1,
             head=192, dim=64, layout="interleaved", scaling="yarn", factor=32.0, far=1000000, dtype="bf16"),
        # --- dropout ---
        # a few tokens added to their residual stream
        dict(name="dropout_fwd_64x2048", op="dropout", dir="fwd", rows=64, cols=2048, p=0.1, residual=True,
             dtype="bf16"),
        # a large batch, the same
        dict(name="dropout_fwd_16384x7168", op="dropout", dir="fwd", rows=16384, cols=7168, p=0.1,
             residual=True, dtype="bf16"),
        # the gradient of odd rows in fp32
        dict(name="dropout_bwd_8191x2047_f32", op="dropout", dir="bwd", rows=8191, cols=2047, p=0.25,
             residual=False, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row's width: three in four a multiple of 8, the others as they fall."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "rotary", "dropout"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "ffn":
        grouped = rng.random() < 0.5
        hidden, inner = _width(rng, 64, 4096), _width(rng, 32, 2048 if grouped else 11008)
        return dict(op=op, dir=rng.choice(["fwd", "keep", "bwd", "both"]),
                    tokens=_log(rng, 1, 32768 if grouped else 8192), hidden=hidden, inner=inner,
                    experts=_log(rng, 4, 64) if grouped else 0,
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    if op == "rotary":
        layout = rng.choice(["half", "interleaved"])
        dim = 2 * _log(rng, 8, 128)
        head = dim + rng.choice([0, 0, 2 * _log(rng, 1, 64)])
        heads, batch = _log(rng, 1, 64), _log(rng, 1, 8)
        seq = _log(rng, 1, max(1, min(16384, (1 << 26) // (head * heads * batch))))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), batch=batch, seq=seq, heads=heads,
                    kheads=rng.randint(1, heads), head=head, dim=dim, layout=layout, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]),
                    far=rng.choice([0, 0, 5000, 1000000]), dtype=kind)
    cols = _width(rng, 32, 16384)
    return dict(op=op, dir=rng.choice(["fwd", "bwd"]), rows=_log(rng, 1, min(32768, (1 << 26) // cols)),
                cols=cols, p=rng.choice([0.1, 0.5, round(rng.random(), 3)]), residual=rng.random() < 0.5,
                dtype=kind)


# -------------------------------------------------------------- their inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "ffn":
        t, d, f, way = c["tokens"], c["hidden"], c["inner"], c["dir"]
        lead = (c["experts"],) if c["experts"] else ()
        c["x"] = _randn(g, t, d).bfloat16()
        c["wg"] = (_randn(g, *lead, f, d) * d ** -0.5).bfloat16()
        c["wu"] = (_randn(g, *lead, f, d) * d ** -0.5).bfloat16()
        c["wd"] = (_randn(g, *lead, d, f) * f ** -0.5).bfloat16()
        if way in ("bwd", "both"):
            c["dy"] = (0.01 * _randn(g, t, d)).bfloat16()
        if way == "bwd":
            c["g"], c["u"] = _randn(g, t, f).bfloat16(), _randn(g, t, f).bfloat16()
        if c["experts"]:
            # tokens as a router spreads them; some experts get none
            host = torch.Generator().manual_seed(seed)
            share = torch.exp(0.7 * torch.randn(c["experts"], generator=host))
            share[::7] = 0.0
            counts = torch.bincount(torch.multinomial(share, t, replacement=True, generator=host),
                                    minlength=c["experts"])
            c["longest"] = int(counts.max())
            offsets = torch.zeros(c["experts"] + 1, dtype=torch.int32)
            offsets[1:] = counts.cumsum(0)
            c["offsets"] = offsets.to(DEV)
        return c
    dtype = TYPES[c["dtype"]]
    if c["op"] == "rotary":
        b, s = c["batch"], c["seq"]
        c["q"] = _randn(g, b, s, c["heads"], c["head"]).to(dtype)
        c["k"] = _randn(g, b, s, c["kheads"], c["head"]).to(dtype)
        # counted from 0, or sequences that begin anywhere up to `far`
        c["positions"] = None
        if c["far"]:
            first = torch.randint(0, c["far"], (b, 1), generator=g, device=DEV)
            c["positions"] = first + torch.arange(s, device=DEV)
        return c
    c["x"] = _randn(g, c["rows"], c["cols"]).to(dtype)
    c["r"] = _randn(g, c["rows"], c["cols"]).to(dtype) if c["residual"] and c["dir"] == "fwd" else None
    host = torch.Generator().manual_seed(seed)
    c["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=host))
    c["offset"] = int(torch.randint(0, 1 << 40, (1,), generator=host))
    return c


# ------------------------------------------------------------ the plain form

def _act(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    a = (2.0 / math.pi) ** 0.5
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * g * g)


def _rows(s, v):
    """Every expert's rows of v in fp32, filled up with zeros to the longest's
    number; one dense block's as a batch of one."""
    if not s["experts"]:
        return v.float()[None]
    at = s["offsets"][:-1, None] + torch.arange(s["longest"], device=v.device)
    live = at < s["offsets"][1:, None]
    return v[torch.where(live, at, 0).long()].float() * live[..., None]


def _flat(s, v):
    """The way back: tokens x columns."""
    if not s["experts"]:
        return v[0]
    live = torch.arange(s["longest"], device=v.device) < s["offsets"].diff()[:, None]
    return v[live]


def _ffn(s):
    way, lead = s["dir"], s["experts"] > 0
    wg, wu, wd = (s[w].float() if lead else s[w].float()[None] for w in ("wg", "wu", "wd"))
    x = _rows(s, s["x"])
    low = torch.bfloat16
    first = ()
    if way == "bwd":
        g, u = _rows(s, s["g"]), _rows(s, s["u"])
    else:
        g, u = torch.bmm(x, wg.mT), torch.bmm(x, wu.mT)
        y = torch.bmm(_act(s["act"], g)[0] * u, wd.mT)
        first = (_flat(s, y).to(low),)
        if way == "fwd":
            return first
        if way == "keep":
            return (*first, _flat(s, g).to(low), _flat(s, u).to(low))
    dy = _rows(s, s["dy"])
    a, da = _act(s["act"], g)
    dh = torch.bmm(dy, wd)
    dg, du = dh * u * da, dh * a
    dx = torch.bmm(dg, wg) + torch.bmm(du, wu)
    grads = [torch.bmm(dg.mT, x), torch.bmm(du.mT, x), torch.bmm(dy.mT, a * u)]
    return (*first, _flat(s, dx).to(low), *((w if lead else w[0]).to(low) for w in grads))


def _frequencies(s):
    """(angle per position of every pair, as a list; the factor of the result)."""
    dim, base, f = s["dim"], 10000.0, s["factor"]
    if s["scaling"] == "ntk":
        base *= f ** (dim / (dim - 2))
    freq = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if s["scaling"] == "linear":
        freq = [v / f for v in freq]
    if s["scaling"] != "yarn":
        return freq, 1.0
    # pairs that turn less than once in the original 4096 positions are
    # stretched, those that turn over 32 times are not, a ramp between

    def place(turns):
        return dim * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), dim - 1)
    ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(dim // 2)]
    return [v / f * r + v * (1 - r) for v, r in zip(freq, ramp)], 0.1 * math.log(f) + 1.0


def _rotary(s):
    freq, m = _frequencies(s)
    freq = torch.tensor(freq, dtype=torch.float64, device=DEV)
    at = s["positions"] if s["positions"] is not None else torch.arange(s["seq"], device=DEV)[None]
    angle = (at.double()[..., None] * freq)[:, :, None]
    cos, sin = (m * torch.cos(angle)).float(), (m * torch.sin(angle)).float()
    if s["dir"] == "bwd":
        sin = -sin
    dim, out = s["dim"], []
    for x in (s["q"], s["k"]):
        v = x.float()
        r = v[..., :dim]
        a, b = (r[..., :dim // 2], r[..., dim // 2:]) if s["layout"] == "half" else (r[..., ::2], r[..., 1::2])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.cat(y, -1) if s["layout"] == "half" else torch.stack(y, -1).flatten(-2)
        out.append(torch.cat([y, v[..., dim:]], -1).to(x.dtype))
    return tuple(out)


def _philox(s, n):
    """n 16-bit numbers: Philox4x32-10 (Salmon et al., 2011) of the counters
    (block, offset) under the key seed, eight numbers a block, low half first."""
    low = 0xFFFFFFFF
    block = torch.arange(-(-n // 8), device=DEV)
    c = [block & low, block >> 32, torch.full_like(block, s["offset"] & low),
         torch.full_like(block, s["offset"] >> 32)]
    k0, k1 = s["seed"] & low, s["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57            # modulo 2^64
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    words = torch.stack(c, -1)
    return torch.stack([words & 0xFFFF, words >> 16], -1).flatten()[:n]


def _dropout(s):
    x = s["x"].float()
    limit = math.floor(s["p"] * 65536 + 0.5)
    keep = (_philox(s, x.numel()) >= limit).view(x.shape)
    y = torch.where(keep, x * (65536 / (65536 - limit) if limit < 65536 else 0.0), 0.0)
    return (y if s["r"] is None else y + s["r"].float()).to(s["x"].dtype)


_PLAIN = {"ffn": _ffn, "rotary": _rotary, "dropout": _dropout}


# ------------------------------------------------------- the package's calls

def _own(s):
    import newton_schulz_06_gb300 as ns
    way = s["dir"]
    if s["op"] == "dropout":
        if way == "bwd":
            return ns.dropout_backward(s["x"], s["p"], s["seed"], s["offset"])
        return ns.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["r"])
    if s["op"] == "rotary":
        plan = s.get("plan")          # a program keeps it with its model
        if plan is None:
            plan = s["plan"] = ns.RotaryPlan(s["dim"], layout=s["layout"], scaling=s["scaling"],
                                             factor=s["factor"], original=4096)
        turn = ns.rotary if way == "fwd" else ns.rotary_backward
        return turn(s["q"], s["k"], plan, positions=s["positions"])
    weights = s["wg"], s["wu"], s["wd"]
    more = dict(offsets=s.get("offsets"), activation=s["act"])
    first, saved = (), None
    if way == "bwd":
        saved = s["g"], s["u"]
    else:
        y, saved = ns.gated_ffn(s["x"], *weights, keep=way != "fwd", **more)
        first = (y,)
        if way == "fwd":
            return first
        if way == "keep":
            return (*first, *saved)
    return (*first, *ns.gated_ffn_backward(s["dy"], s["x"], saved, *weights, **more))


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------- what it costs

def work(case):
    c = case
    if c["op"] == "ffn":
        t, d, f, e = c["tokens"], c["hidden"], c["inner"], max(1, c["experts"])
        product, w = 2.0 * t * d * f, 2 * e * 3 * d * f
        fwd = 2 * 2 * t * d + w                        # x, y, the weights
        bwd = 2 * (3 * t * d + 2 * t * f) + 2 * w      # x, dy, dx, what was kept, weights, gradients
        bytes_, products = {"fwd": (fwd, 3), "keep": (fwd + 2 * 2 * t * f, 3), "bwd": (bwd, 6),
                            # in one pass x and the weights are read once, and what is kept is written once
                            "both": (2 * (4 * t * d + 2 * t * f) + 2 * w, 9)}[c["dir"]]
        return {"bytes": bytes_, "flops": products * product}
    size = {"bf16": 2, "f32": 4}[c["dtype"]]
    if c["op"] == "rotary":
        rows = c["batch"] * c["seq"] * (c["heads"] + c["kheads"])
        at = 8 * c["batch"] * c["seq"] if c["far"] else 0
        return {"bytes": 2 * rows * c["head"] * size + at, "flops": rows * c["dim"] * 3.0}
    n = c["rows"] * c["cols"]
    return {"bytes": n * size * (3 if c["residual"] and c["dir"] == "fwd" else 2), "flops": 2.0 * n}


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The outputs of `run` from the definitions in 64 bits, written apart
    from the plain form."""
    s = prepare(case, seed)
    return {"ffn": _exact_ffn, "rotary": _exact_rotary, "dropout": _exact_dropout}[s["op"]](s)


def _exact_ffn(s):
    D, way = torch.float64, s["dir"]
    ends = s["offsets"].tolist() if s["experts"] else [0, s["tokens"]]

    def act(g):
        if s["act"] == "silu":
            return g * torch.sigmoid(g)
        if s["act"] == "gelu":
            return g * torch.special.ndtr(g)
        return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))

    parts = []
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        wg, wu, wd = ((s[w][e] if s["experts"] else s[w]).to(D) for w in ("wg", "wu", "wd"))
        x = s["x"][a:b].to(D)
        got = []
        if way == "bwd":
            g, u = s["g"][a:b].to(D), s["u"][a:b].to(D)
        else:
            g, u = x.mm(wg.t()), x.mm(wu.t())
            got.append((act(g) * u).mm(wd.t()))
        if way == "keep":
            got += [g, u]
        if way in ("bwd", "both"):
            dy = s["dy"][a:b].to(D)
            dh = dy.mm(wd)
            with torch.enable_grad():
                gl, ul = g.detach().requires_grad_(), u.detach().requires_grad_()
                h = act(gl) * ul
                dg, du = torch.autograd.grad(h, (gl, ul), dh)
            got += [torch.addmm(dg.mm(wg), du, wu), dg.t().mm(x), du.t().mm(x), dy.t().mm(h.detach())]
        parts.append(got)
    n = len(parts[0])
    tall = {"fwd": n, "keep": n, "bwd": 1, "both": 2}[way]       # outputs with a row for every token
    return tuple(torch.cat([p[i] for p in parts]) if i < tall or not s["experts"]
                 else torch.stack([p[i] for p in parts]) for i in range(n))


def _exact_rotary(s):
    dim, D = s["dim"], torch.float64
    freq, m = _frequencies(s)
    at = s["positions"] if s["positions"] is not None else torch.arange(s["seq"], device=DEV).expand(s["batch"], -1)
    sign = -1.0 if s["dir"] == "bwd" else 1.0
    turn = torch.polar(torch.full((), m, dtype=D, device=DEV),
                       sign * at.to(D)[:, :, None, None] * torch.tensor(freq, dtype=D, device=DEV))
    i = torch.arange(dim // 2, device=DEV)
    one, two = (i, i + dim // 2) if s["layout"] == "half" else (2 * i, 2 * i + 1)
    out = []
    for x in (s["q"], s["k"]):
        y = x.to(D)
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_dropout(s):
    """The generator in 16-bit pieces, so that no product passes 2^53."""
    x = s["x"].to(torch.float64)
    n = x.numel()

    def mul(a, m):
        """High and low word of a m."""
        al, ah, ml, mh = a % 65536, a // 65536, m % 65536, m // 65536
        mid = al * mh + ah * ml + al * ml // 65536
        return ah * mh + mid // 65536, mid % 65536 * 65536 + al * ml % 65536

    i = torch.arange((n + 7) // 8, device=DEV)
    state = (i % 2 ** 32, i // 2 ** 32, torch.full_like(i, s["offset"] % 2 ** 32),
             torch.full_like(i, s["offset"] // 2 ** 32))
    for r in range(10):
        key = (s["seed"] + r * 0x9E3779B9) % 2 ** 32, (s["seed"] // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        h0, l0 = mul(state[0], 0xD2511F53)
        h1, l1 = mul(state[2], 0xCD9E8D57)
        state = (h1 ^ state[1] ^ key[0], l1, h0 ^ state[3] ^ key[1], l0)
    words = torch.stack([v for w in state for v in (w % 65536, w // 65536)], 1).reshape(-1)[:n]
    limit = math.floor(s["p"] * 65536 + 0.5)
    kept = (words.view(x.shape) >= limit).to(torch.float64)
    y = x * kept * (65536 / (65536 - limit)) if limit < 65536 else x * 0.0
    return y if s["r"] is None else y + s["r"].to(torch.float64)
