"""64-bit forms of the operators inside a block (gated feed-forward, rotary
positions, dropout), straight from the formulas of include/muon.h, with bounds
on the error of a kernel that keeps to them."""
from __future__ import annotations

import math

import torch

D = torch.float64
U32 = 2.0 ** -24               # half a unit in the last place, relative
HALF = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}
# an activation's own error, relative to the size of its parts: an exponential,
# a reciprocal, and what is rounded on the way
ACT = 2.0 ** -19


def sums(k):
    """Relative to the sum of the magnitudes of k terms: the tensor cores add in
    steps of 16 and may cut off twice a step (2^-23 each)."""
    return (2 * (-(-k // 16)) + 4) * 2.0 ** -23


# ------------------------------------------------------- gated feed-forward

def act(name, g):
    """act(g), its derivative, and the size of the derivative's terms."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), s * (1 + g.abs() * (1 - s))
    if name == "gelu":
        phi = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        c = torch.special.ndtr(g)
        return g * c, c + g * phi, c + g.abs() * phi
    a = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * a * (g + 0.044715 * g ** 3))
    more = s * (1 - s) * 2 * a * (1 + 3 * 0.044715 * g * g)
    return g * s, s + g * more, s + g.abs() * more


def spans(offsets, rows):
    """Every expert's rows, with the offsets limited to a rising order."""
    if offsets is None:
        return [(0, rows)]
    got, low = [], 0
    for v in offsets.tolist():
        low = max(low, min(max(v, 0), rows))
        got.append(low)
    return list(zip(got, got[1:]))


def matrix(w, e):
    return (w[e] if w.dim() == 3 else w).to(D)


def ffn(x, wg, wu, wd, offsets=None, name="silu"):
    """((y, g, u), their bounds), rows x columns; NaN where no expert is."""
    rows, hidden = x.shape
    inner = wg.shape[-2]
    new = [torch.full((rows, n), math.nan, dtype=D, device=x.device) for n in (hidden, inner, inner)]
    bounds = [torch.zeros_like(v) for v in new]
    r = HALF[torch.bfloat16]
    for e, (a, b) in enumerate(spans(offsets, rows)):
        if a == b:
            continue
        v = x[a:b].to(D)
        g, u = v @ matrix(wg, e).t(), v @ matrix(wu, e).t()
        eg, eu = (sums(hidden) * (v.abs() @ matrix(w, e).abs().t()) for w in (wg, wu))
        h0, _, _ = act(name, g)
        h = h0 * u
        # h is held in bf16: past its largest value it is infinite
        h = torch.where(h.abs() > torch.finfo(torch.bfloat16).max, h * math.inf, h)
        # |act'| <= 1.13, and what rounding h to bf16 adds
        eh = 1.13 * eg * (u.abs() + eu) + h0.abs() * eu + ACT * g.abs() * u.abs()
        eh = eh + r * (h.abs() + eh)
        y = h @ matrix(wd, e).t()
        ey = eh @ matrix(wd, e).abs().t() + sums(inner) * ((h.abs() + eh) @ matrix(wd, e).abs().t())
        for to, bound, value, err in zip(new, bounds, (y, g, u), (ey, eg, eu)):
            to[a:b] = value
            bound[a:b] = err + r * (value.abs() + err) + 1e-38
    return new, bounds


def ffn_grad(dy, x, g, u, wg, wu, wd, offsets=None, name="silu", dtype=torch.bfloat16, before=None):
    """((dx, dwg, dwu, dwd), their bounds); the weights' with a leading expert
    axis where they have one.  before: what the gradients are added to."""
    rows, hidden = dy.shape
    r = HALF[torch.bfloat16]
    dx = torch.full((rows, hidden), math.nan, dtype=D, device=dy.device)
    bx = torch.zeros_like(dx)
    grads = [torch.zeros(w.shape, dtype=D, device=dy.device) for w in (wg, wu, wd)]
    bounds = [torch.zeros_like(v) for v in grads]
    for e, (a, b) in enumerate(spans(offsets, rows)):
        if a == b:
            continue
        d, v = dy[a:b].to(D), x[a:b].to(D)
        gg, uu = g[a:b].to(D), u[a:b].to(D)
        f, df, size = act(name, gg)
        dh = d @ matrix(wd, e)
        eh = sums(hidden) * (d.abs() @ matrix(wd, e).abs())
        dg, du, h = dh * uu * df, dh * f, f * uu
        edg = eh * uu.abs() * size + (dh.abs() + eh) * uu.abs() * ACT * (size + 1e-30)
        edu = eh * f.abs() + (dh.abs() + eh) * ACT * gg.abs()
        ehh = ACT * gg.abs() * uu.abs()
        edg, edu, ehh = (err + r * (val.abs() + err) for err, val in ((edg, dg), (edu, du), (ehh, h)))
        out = dg @ matrix(wg, e) + du @ matrix(wu, e)
        size = (dg.abs() + edg) @ matrix(wg, e).abs() + (du.abs() + edu) @ matrix(wu, e).abs()
        err = edg @ matrix(wg, e).abs() + edu @ matrix(wu, e).abs() + sums(2 * dg.shape[1]) * size
        dx[a:b], bx[a:b] = out, err + r * (out.abs() + err) + 1e-38
        for i, (one, eone, two, etwo) in enumerate(((dg, edg, v, 0 * v), (du, edu, v, 0 * v),
                                                    (d, 0 * d, h, ehh))):
            at = e if grads[i].dim() == 3 else slice(None)
            grads[i][at] = one.t() @ two
            bounds[i][at] = (eone.t() @ (two.abs() + etwo) + one.abs().t() @ etwo
                             + sums(b - a) * ((one.abs() + eone).t() @ (two.abs() + etwo)))
    for i in range(3):
        if before is not None:
            grads[i] += before[i].to(D)
            bounds[i] += U32 * (grads[i].abs() + bounds[i])
        bounds[i] += HALF[dtype] * (grads[i].abs() + bounds[i]) + 1e-38
    return [dx, *grads], [bx, *bounds]


# --------------------------------------------------------- rotary positions

def frequencies(dim, base=10000.0, scaling="none", factor=1.0, original=4096, fast=32.0, slow=1.0):
    """(radians a position of every pair, the results' factor)."""
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    freq = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling != "yarn":
        return freq, 1.0

    def place(turns):
        return dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = max(math.floor(place(fast)), 0), min(math.ceil(place(slow)), dim - 1)
    got = []
    for i, f in enumerate(freq):
        r = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        got.append(f / factor * r + f * (1 - r))
    return got, 0.1 * math.log(factor) + 1.0


def rotary(x, at, dim, freq, scale, layout, inverse=False):
    """x: batch x seq x heads x head; at: batch x seq positions (int64).  (the
    result in 64 bits, a bound for x's type)."""
    angle = at.to(D)[:, :, None, None] * torch.tensor(freq, dtype=D, device=x.device)
    c, s = scale * torch.cos(angle), scale * torch.sin(angle) * (-1 if inverse else 1)
    v = x.to(D)
    y, bound = v.clone(), torch.zeros_like(v)
    half = dim // 2
    one, two = (slice(0, half), slice(half, dim)) if layout == "half" else (slice(0, dim, 2), slice(1, dim, 2))
    a, b = v[..., one], v[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    # the 64-bit angle's own error (2^-53 of it, on both sides) and the turn
    # rounded to fp32 (2^-24 of half a turn at most), then the sine's error
    # (2 in the last place), the scale's and the sum's roundings
    err = angle.abs() * 2.0 ** -51 + 2 * math.pi * 2.0 ** -25 + 8 * U32
    size = abs(scale) * (a.abs() + b.abs()) * err
    bound[..., one], bound[..., two] = size, size
    h = HALF[x.dtype]
    turned = torch.zeros(dim + (v.shape[-1] - dim), dtype=D, device=x.device)
    turned[:dim] = 1.0
    return y, bound + turned * (h * (y.abs() + bound) + 1e-38)


# ----------------------------------------------------------------- dropout

def philox(counter, key):
    """One block of Philox4x32-10 with Python's whole numbers."""
    c, k, low = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [k[0] + 0x9E3779B9 & low, k[1] + 0xBB67AE85 & low]
    return c


def kept(n, p, seed, offset):
    """Which of n elements stay, as a list of truth values."""
    limit, low, got = math.floor(p * 65536 + 0.5), 0xFFFFFFFF, []
    for b in range(-(-n // 8)):
        for w in philox((b & low, b >> 32, offset & low, offset >> 32 & low), (seed & low, seed >> 32 & low)):
            got += [(w & 0xFFFF) >= limit, (w >> 16) >= limit]
    return got[:n]


def dropout(x, p, seed, offset, residual=None):
    """The result in 64 bits (CPU)."""
    limit = math.floor(p * 65536 + 0.5)
    keep = torch.tensor(kept(x.numel(), p, seed, offset)).view(x.shape)
    scale = 65536 / (65536 - limit) if limit < 65536 else 0.0
    y = torch.where(keep, x.to("cpu", D) * scale, torch.zeros((), dtype=D))
    return y if residual is None else y + residual.to("cpu", D)
