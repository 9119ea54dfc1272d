"""What is measured of the operators around the Muon step: layer norm, 8-bit
activation checkpoints, the weight gradient read from a checkpoint, and the
router with its balance loss.  They take a block from its activations to the
gradients that a Muon step reads.

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the package's operators.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
COEF = 0.01
BLOCK = 32                 # values of a row that share one scale
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # --- layer norm (x, dy and y of one type; weights of the other) ---
        # a few tokens of a 2048-wide block: the launch is what counts
        dict(name="norm_fwd_64x2048", op="norm", dir="fwd", rows=64, cols=2048,
             dtype="bf16", wdtype="bf16", bias=True),
        # the backward pass of an odd number of tokens, 7168 wide
        dict(name="norm_bwd_4099x7168", op="norm", dir="bwd", rows=4099, cols=7168,
             dtype="bf16", wdtype="f32", bias=True),
        # both passes in fp32 over a large batch, no bias
        dict(name="norm_both_16384x4096_f32", op="norm", dir="both", rows=16384, cols=4096,
             dtype="f32", wdtype="f32", bias=False),
        # --- checkpoints in 8 bits ---
        # an expert's activations (768 wide) of a few hundred tokens
        dict(name="pack_517x768_f32", op="checkpoint", dir="pack", rows=517, cols=768,
             dtype="f32", wdtype="f32", bias=False),
        # the norm's forward pass that keeps its normalised rows in 8 bits
        dict(name="ckpt_fwd_8192x7168", op="checkpoint", dir="norm_fwd", rows=8192, cols=7168,
             dtype="bf16", wdtype="bf16", bias=True),
        # and the backward pass that reads them
        dict(name="ckpt_bwd_8192x7168", op="checkpoint", dir="norm_bwd", rows=8192, cols=7168,
             dtype="bf16", wdtype="bf16", bias=True),
        # --- weight gradient from a checkpoint ---
        # k projection (512 x 2048) of a short sequence
        dict(name="wgrad_300_512x2048", op="weight_grad", tokens=300, n=512, k=2048,
             experts=0, out="bf16", add=False, affine=False),
        # q projection (4096 x 2048) after a norm, added to an fp32 gradient
        dict(name="wgrad_4097_4096x2048_f32", op="weight_grad", tokens=4097, n=4096, k=2048,
             experts=0, out="f32", add=True, affine=True),
        # o projection (7168 x 8192) over a large batch
        dict(name="wgrad_16384_7168x8192", op="weight_grad", tokens=16384, n=7168, k=8192,
             experts=0, out="bf16", add=False, affine=False),
        # 128 experts' gate matrices (768 x 2048): 8192 tokens, 8 experts each
        dict(name="wgrad_128_experts_768x2048", op="weight_grad", tokens=65536, n=768, k=2048,
             experts=128, out="bf16", add=False, affine=False),
        # --- router and balance loss ---
        # a short sequence's forward pass, 8 of 128 experts
        dict(name="route_fwd_200x128", op="route", dir="fwd", tokens=200, experts=128, k=8,
             dtype="f32", renormalise=True, mask=False),
        # a large batch with padding tokens, both passes, 8 of 384 experts
        dict(name="route_both_32769x384", op="route", dir="both", tokens=32769, experts=384, k=8,
             dtype="bf16", renormalise=True, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row's width: three in four a multiple of 8, the others as they fall."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.25 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "checkpoint", "weight_grad", "route"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "checkpoint"):
        cols = _width(rng, 64, 16384)
        rows = _log(rng, 1, min(32768, (1 << 26) // cols))
        way = rng.choice(["fwd", "bwd", "both"] if op == "norm" else ["pack", "norm_fwd", "norm_bwd"])
        return dict(op=op, dir=way, rows=rows, cols=cols, dtype=kind,
                    wdtype=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    if op == "weight_grad":
        grouped = rng.random() < 0.4
        experts = _log(rng, 4, 128) if grouped else 0
        n, k = _width(rng, 64, 2048 if grouped else 8192), _width(rng, 64, 2048 if grouped else 8192)
        tokens = _log(rng, 1, 65536 if grouped else 16384)
        return dict(op=op, tokens=tokens, n=n, k=k, experts=experts,
                    out=kind, add=rng.random() < 0.3, affine=rng.random() < 0.3)
    experts = _log(rng, 4, 512)
    return dict(op=op, dir=rng.choice(["fwd", "bwd", "both"]), tokens=_log(rng, 1, 32768),
                experts=experts, k=rng.randint(1, min(8, experts)), dtype=kind,
                renormalise=rng.random() < 0.5, mask=rng.random() < 0.5)


# -------------------------------------------------------------- their inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, cols):
    """Rows as a residual stream has them: column scales that differ, a few
    columns far larger than the rest, and a mean that is not zero."""
    scale = torch.exp(0.5 * _randn(g, cols))
    scale[torch.rand(cols, generator=g, device=DEV) < 0.01] *= 10.0
    return _randn(g, rows, cols).mul_(scale).add_(0.1 * _randn(g, cols))


def _affine(g, cols, dtype, bias):
    w = (1.0 + 0.2 * _randn(g, cols)).to(dtype)
    return w, (0.2 * _randn(g, cols)).to(dtype) if bias else None


def _stats(x):
    """Mean and 1 / deviation of every row."""
    mean = x.mean(-1)
    d = x - mean[:, None]
    return mean, 1.0 / torch.sqrt((d * d).mean(-1) + EPS)


def _encode(v):
    """q (int8) and scale bytes of the rows of v: blocks of 32 values, value =
    q 2^(E - 6) with E = floor(log2(max |v|)), E + 127 in a byte."""
    rows, cols = v.shape
    pad = -cols % BLOCK
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    b = v.view(rows, -1, BLOCK)
    top = b.abs().amax(-1)
    ex = torch.frexp(top)[1] - 1
    ex = torch.where(top == 0, -127, ex.clamp(-127, 127))
    unit = torch.exp2(-ex.float())[..., None]
    q = torch.clamp(torch.round(b * unit * 64.0), -127, 127).to(torch.int8)
    bad = ~torch.isfinite(top)
    e = torch.where(bad, 255, ex + 127).to(torch.uint8)
    return torch.where(bad[..., None], 0, q).view(rows, -1), e


def _decode(q, e, cols):
    """The values that q and the scale bytes stand for."""
    rows = q.shape[0]
    unit = torch.where(e == 255, math.nan, torch.exp2(e.float() - 127.0) / 64.0)
    v = q.view(rows, -1, BLOCK).float() * unit[..., None]
    return v.view(rows, -1)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] in ("norm", "checkpoint"):
        rows, cols, dtype = c["rows"], c["cols"], TYPES[c["dtype"]]
        x = _activations(g, rows, cols).to(dtype)
        c["w"], c["b"] = _affine(g, cols, TYPES[c["wdtype"]], c["bias"])
        dy = (0.01 * _randn(g, rows, cols)).to(dtype)
        if c["dir"] in ("fwd", "both", "pack"):
            c["x"] = x
        if c["dir"] in ("bwd", "norm_bwd", "both"):
            c["dy"] = dy
        if c["dir"] == "bwd":
            c["x"] = x
            c["mean"], c["rstd"] = _stats(x.float())
        elif c["dir"] == "norm_fwd":
            c["x"] = x
        elif c["dir"] == "norm_bwd":
            xf = x.float()
            mean, c["rstd"] = _stats(xf)
            c["q"], c["e"] = _encode((xf - mean[:, None]) * c["rstd"][:, None])
        return c
    if c["op"] == "weight_grad":
        t, n, k, out = c["tokens"], c["n"], c["k"], TYPES[c["out"]]
        x = _activations(g, t, k)
        mean, rstd = _stats(x)
        c["q"], c["e"] = _encode((x - mean[:, None]) * rstd[:, None])
        c["dy"] = (0.01 * _randn(g, t, n)).bfloat16()
        if c["affine"]:
            c["w"], c["b"] = _affine(g, k, torch.float32, True)
        shape = (n, k)
        if c["experts"]:
            # tokens as a router spreads them; some experts get none
            p = torch.exp(0.7 * torch.randn(c["experts"], generator=torch.Generator().manual_seed(seed)))
            p[::7] = 0.0
            at = torch.multinomial(p, t, replacement=True, generator=torch.Generator().manual_seed(seed + 1))
            counts = torch.bincount(at, minlength=c["experts"])
            c["longest"] = int(counts.max())
            offsets = torch.zeros(c["experts"] + 1, dtype=torch.int32)
            offsets[1:] = counts.cumsum(0)
            c["offsets"] = offsets.to(DEV)
            shape = (c["experts"], n, k)
        if c["add"]:
            c["base"] = (0.3 * _randn(g, *shape)).to(out)
        return c
    t, experts = c["tokens"], c["experts"]
    z = _randn(g, t, experts) + 0.5 * _randn(g, experts)
    c["logits"] = z.to(TYPES[c["dtype"]])
    c["keep"] = torch.rand(t, generator=g, device=DEV) < 0.9 if c["mask"] else None
    if c["dir"] != "fwd":
        c["dweights"] = 0.01 * _randn(g, t, c["k"])
        c["dloss"] = torch.ones((), device=DEV)
    if c["dir"] == "bwd":
        c["indices"], c["weights"], c["counts"], _, _, c["kept"] = _route(
            c["logits"], c["k"], c["keep"], c["renormalise"])
    return c


# ------------------------------------------------------------ the plain form

def _route(logits, k, keep, renormalise):
    """Indices, weights, counts, offsets, loss and the number of tokens kept."""
    z = logits.float()
    t, experts = z.shape
    top = z.amax(-1, keepdim=True)
    ex = torch.exp(z - top)
    s = ex.sum(-1, keepdim=True)
    p = ex / s
    order = torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, order)
    if renormalise:
        w = w / w.sum(-1, keepdim=True)
    if keep is None:
        keep = torch.ones(t, dtype=torch.bool, device=z.device)
    idx = torch.where(keep[:, None], order, -1)
    w = torch.where(keep[:, None], w, 0.0)
    counts = torch.bincount(idx.view(-1) + 1, minlength=experts + 1)[1:]
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=z.device)
    offsets[1:] = counts.cumsum(0)
    n = keep.sum().clamp(min=1).float()
    mean_p = torch.where(keep[:, None], p, 0.0).sum(0) / n
    loss = COEF * experts / (k * n) * (counts.float() * mean_p).sum()
    return (idx.to(torch.int32), w, counts.to(torch.int32), offsets, loss,
            keep.sum(dtype=torch.int32))


def _route_grad(logits, idx, w, counts, keep, dloss, dw, k, renormalise):
    z = logits.float()
    t, experts = z.shape
    ex = torch.exp(z - z.amax(-1, keepdim=True))
    p = ex / ex.sum(-1, keepdim=True)
    if keep is None:
        keep = torch.ones(t, dtype=torch.bool, device=z.device)
    n = keep.sum().clamp(min=1).float()
    at = idx.long().clamp(min=0)
    d = dw
    if renormalise:
        d = (d - (d * w).sum(-1, keepdim=True)) / p.gather(1, at).sum(-1, keepdim=True)
    h = (dloss * COEF * experts / (k * n * n) * counts.float()).expand(t, experts)
    h = h.scatter_add(1, at, d)
    dz = p * (h - (p * h).sum(-1, keepdim=True))
    return torch.where(keep[:, None], dz, 0.0)


def _norm(x, w, b):
    mean = x.mean(-1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(-1) + EPS)
    h = d * rstd[:, None]
    y = h * w
    return y if b is None else y + b, mean, rstd, h


def _norm_grad(dy, h, rstd, w):
    g = dy * w
    dx = (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True)) * rstd[:, None]
    return dx, (dy * h).sum(0), dy.sum(0)


def _weight_grad(s):
    h = _decode(s["q"], s["e"], s["k"])
    dy = s["dy"].float()
    if s["affine"]:
        h = h * s["w"] + s["b"]
    if s["experts"]:
        # every expert's rows, filled up with zeros to the longest's number
        at = s["offsets"][:-1, None] + torch.arange(s["longest"], device=h.device)
        live = at < s["offsets"][1:, None]
        at = torch.where(live, at, 0).long()
        grad = torch.bmm((dy[at] * live[..., None]).transpose(1, 2), h[at])
    else:
        grad = dy.t() @ h
    return grad + s["base"].float() if s["add"] else grad


def _plain(s):
    """The case's outputs with elementary operations in 32 bits."""
    if s["op"] == "weight_grad":
        return _weight_grad(s).to(TYPES[s["out"]])
    if s["op"] == "route":
        keep, k, way = s["keep"], s["k"], s["dir"]
        if way == "bwd":
            saved, first = (s["indices"], s["weights"], s["counts"]), ()
        else:
            idx, w, counts, offsets, loss, _ = _route(s["logits"], k, keep, s["renormalise"])
            saved, first = (idx, w, counts), (idx, w, counts, offsets, loss)
            if way == "fwd":
                return first
        dz = _route_grad(s["logits"], *saved, keep, s["dloss"], s["dweights"], k, s["renormalise"])
        return (*first, dz.to(TYPES[s["dtype"]]))
    way, dtype, wdtype = s["dir"], TYPES[s["dtype"]], TYPES[s["wdtype"]]
    if way == "pack":
        q, e = _encode(s["x"].float())
        return _decode(q, e, s["cols"]).to(torch.bfloat16)
    w, b = s["w"].float(), (s["b"].float() if s["bias"] else None)
    first = ()
    if way in ("fwd", "both", "norm_fwd"):
        y, mean, rstd, h = _norm(s["x"].float(), w, b)
        if way == "norm_fwd":
            q, e = _encode(h)
            return y.to(dtype), rstd, _decode(q, e, s["cols"]).to(torch.bfloat16)
        first = (y.to(dtype), mean, rstd)
        if way == "fwd":
            return first
    elif way == "bwd":
        rstd = s["rstd"]
        h = (s["x"].float() - s["mean"][:, None]) * rstd[:, None]
    else:
        rstd = s["rstd"]
        h = _decode(s["q"], s["e"], s["cols"])
    dx, dw, db = _norm_grad(s["dy"].float(), h, rstd, w)
    grads = (dx.to(dtype), dw.to(wdtype), db.to(wdtype))
    return (*first, *(grads if s["bias"] else grads[:2]))


# ------------------------------------------------------- the package's calls

def _own(s):
    import newton_schulz_06_gb300 as ns
    if s["op"] == "weight_grad":
        return ns.weight_grad(s["dy"], ns.Checkpoint8(s["q"], s["e"], s["k"]),
                              weight=s.get("w"), bias=s.get("b"), offsets=s.get("offsets"),
                              add=s.get("base"), dtype=TYPES[s["out"]])
    if s["op"] == "route":
        first = ()
        if s["dir"] == "bwd":
            r = ns.Routing(s["indices"], s["weights"], s["counts"], s["kept"],
                           coef=COEF, renormalise=s["renormalise"])
        else:
            r = ns.route(s["logits"], s["k"], mask=s["keep"], coef=COEF, renormalise=s["renormalise"])
            first = (r.indices, r.weights, r.counts, r.offsets, r.loss)
            if s["dir"] == "fwd":
                return first
        return (*first, ns.route_backward(s["logits"], r, dloss=s["dloss"], dweights=s["dweights"]))
    way = s["dir"]
    if way == "pack":
        return ns.checkpoint8(s["x"]).values()
    if way == "norm_fwd":
        y, rstd, saved = ns.layer_norm_checkpoint(s["x"], s["w"], s["b"], eps=EPS)
        return y, rstd, saved.values()
    first = ()
    if way == "norm_bwd":
        saved, mean, rstd = ns.Checkpoint8(s["q"], s["e"], s["cols"]), None, s["rstd"]
    elif way == "bwd":
        saved, mean, rstd = s["x"], s["mean"], s["rstd"]
    else:
        first = ns.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        if way == "fwd":
            return first
        saved, mean, rstd = s["x"], first[1], first[2]
    dx, dw, db = ns.layer_norm_backward(s["dy"], saved, mean, rstd, s["w"], s["b"])
    return (*first, dx, dw, db) if s["bias"] else (*first, dx, dw)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- what it costs

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "weight_grad":
        e, out = max(1, c["experts"]), size[c["out"]]
        grad = e * c["n"] * c["k"] * out
        read = c["tokens"] * (2 * c["n"] + c["k"] * (1 + 1 / BLOCK))
        return {"bytes": read + grad * (2 if c["add"] else 1),
                "flops": 2.0 * c["tokens"] * c["n"] * c["k"]}
    if c["op"] == "route":
        t, n = c["tokens"], c["tokens"] * c["experts"]
        s = size[c["dtype"]]
        fwd = n * s + t * (8 * c["k"] + 4)
        bwd = 2 * n * s + t * (12 * c["k"] + 4)
        return {"bytes": fwd if c["dir"] == "fwd" else bwd if c["dir"] == "bwd" else fwd + bwd,
                "flops": n * (4.0 if c["dir"] == "fwd" else 6.0)}
    n, s = c["rows"] * c["cols"], size[c["dtype"]]
    kept = n * (1 + 1 / BLOCK)
    small = 8 * c["rows"] + 2 * size[c["wdtype"]] * c["cols"]
    moved = {"fwd": 2 * n * s, "bwd": 3 * n * s, "both": 5 * n * s,
             # the values of a checkpoint are read back in bf16
             "pack": n * s + 2 * kept + 2 * n, "norm_fwd": 2 * n * s + 2 * kept + 2 * n,
             "norm_bwd": kept + 2 * n * s}[c["dir"]]
    return {"bytes": moved + small, "flops": n * (16.0 if c["dir"] == "both" else 8.0)}


# ----------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The outputs of `run` from the definitions in 64 bits, written apart
    from the plain form; indices and counts as whole numbers."""
    s = prepare(case, seed)
    D = torch.float64
    if s["op"] == "weight_grad":
        t, kk = s["q"].shape[0], s["k"]
        power = torch.ldexp(torch.ones_like(s["e"], dtype=D), s["e"].to(torch.int32) - 133)
        h = (s["q"].to(D) * power.repeat_interleave(BLOCK, 1))[:, :kk]
        if s["affine"]:
            h = torch.addcmul(s["b"].to(D), h, s["w"].to(D))
        dy = s["dy"].to(D)
        if s["experts"]:
            ends = s["offsets"].tolist()
            grad = torch.stack([dy[a:b].t().mm(h[a:b]) for a, b in zip(ends, ends[1:])])
        else:
            grad = dy.t().mm(h)
        return grad + s["base"].to(D) if s["add"] else grad
    if s["op"] == "route":
        return _exact_route(s, D)
    way, cols = s["dir"], s["cols"]
    w, b = s["w"].to(D), (s["b"].to(D) if s["bias"] else None)

    def nearest(v):
        """What the 8-bit blocks make of v."""
        out = torch.zeros(v.shape[0], -(-cols // BLOCK) * BLOCK, dtype=D, device=DEV)
        out[:, :cols] = v
        out = out.unflatten(1, (-1, BLOCK))
        top = out.abs().amax(-1, keepdim=True)
        step = torch.ldexp(torch.ones_like(top), torch.frexp(top)[1] - 7)
        return (torch.round(out / step).clamp(-127, 127) * step).flatten(1)[:, :cols]

    if way == "pack":
        return nearest(s["x"].to(D))
    if way == "norm_bwd":
        power = torch.ldexp(torch.ones_like(s["e"], dtype=D), s["e"].to(torch.int32) - 133)
        h = (s["q"].to(D) * power.repeat_interleave(BLOCK, 1))[:, :cols]
        rstd = s["rstd"].to(D)
    else:
        x = s["x"].to(D)
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        if way == "bwd":
            mean, rstd = s["mean"].to(D), s["rstd"].to(D)
        h = (x - mean[:, None]) * rstd[:, None]
        if way != "bwd":
            y = h * w if b is None else torch.addcmul(b, h, w)
            if way == "fwd":
                return y, mean, rstd
            if way == "norm_fwd":
                return y, rstd, nearest(h)
    dy = s["dy"].to(D)
    g = dy * w
    inner = torch.einsum("rc,rc->r", g, h) / cols
    dx = (g - g.sum(-1, keepdim=True) / cols - h * inner[:, None]) * rstd[:, None]
    grads = (dx, torch.einsum("rc,rc->c", dy, h)) + ((dy.sum(0),) if s["bias"] else ())
    return (y, mean, rstd, *grads) if way == "both" else grads


def _exact_route(s, D):
    z, k, experts = s["logits"].to(D), s["k"], s["experts"]
    t = z.shape[0]
    keep = s["keep"] if s["keep"] is not None else torch.ones(t, dtype=torch.bool, device=DEV)
    p = torch.exp(torch.log_softmax(z, -1))
    n = max(1, int(keep.sum()))
    # a value's place: how many are larger, or equal and before it
    order = torch.argsort(-z, dim=-1, stable=True)[:, :k]
    sel = p.gather(1, order)
    total = sel.sum(-1, keepdim=True)
    w = sel / total if s["renormalise"] else sel
    hot = torch.zeros(t, experts, dtype=D, device=DEV).scatter_(1, order, 1.0) * keep[:, None]
    counts = hot.sum(0)
    factor = COEF * experts / (k * n)
    loss = factor * (counts * (p * keep[:, None]).sum(0)).sum() / n
    first = ()
    if s["dir"] != "bwd":
        ends = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), counts.cumsum(0).to(torch.int32)])
        first = (torch.where(keep[:, None], order, -1).to(torch.int32), w * keep[:, None],
                 counts.to(torch.int32), ends, loss)
        if s["dir"] == "fwd":
            return first
    d = s["dweights"].to(D)
    if s["renormalise"]:
        d = d / total - (d * w).sum(-1, keepdim=True) / total
    up = torch.zeros(t, experts, dtype=D, device=DEV).scatter_(1, order, d)
    up = up + s["dloss"].to(D) * factor / n * counts
    dz = p * up - p * (p * up).sum(-1, keepdim=True)
    return (*first, dz * keep[:, None])
