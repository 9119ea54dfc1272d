"""Plain 64-bit forms of the operators of a block's training step, on the
CPU, straight from the formulas of include/muon.h, and the inputs and error
bounds that their tests share."""
from __future__ import annotations

import math

import torch

D = torch.float64
U32 = 2.0 ** -24               # half a unit in the last place of fp32
U16 = 2.0 ** -8                # bf16: 2^-9 to nearest, doubled
OUT_ROUND = {torch.float32: 2.0 ** -23, torch.bfloat16: U16}


def to64(t):
    return None if t is None else t.detach().to("cpu", D)


# ---------------------------------------------------------------- checkpoint

def encode(v):
    """(q, e) of the rows of v (float64), as whole numbers."""
    rows, cols = v.shape
    blocks = -(-cols // 32)
    pad = torch.zeros(rows, 32 * blocks, dtype=D)
    pad[:, :cols] = v
    b = pad.view(rows, blocks, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    ex = torch.frexp(torch.where(bad | (top == 0), torch.ones_like(top), top))[1] - 1
    ex = torch.where(top == 0, -127, ex.clamp(min=-127)).to(torch.int32)
    step = torch.ldexp(torch.ones_like(top), ex - 6)
    q = torch.round(b / step[..., None]).clamp(-127, 127)       # ties to even
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    e = torch.where(bad, 255, ex + 127)
    return q.reshape(rows, 32 * blocks).to(torch.int64), e.to(torch.int64)


def decode(q, e, cols):
    q, e = q.to("cpu", torch.int64), e.to("cpu", torch.int32)
    blocks = -(-cols // 32)
    step = torch.ldexp(torch.ones(e.shape, dtype=D), e - 133)
    step = torch.where(e == 255, math.nan, step)[:, :blocks]
    v = q[:, :32 * blocks].view(q.shape[0], blocks, 32).to(D) * step[..., None]
    return v.reshape(q.shape[0], 32 * blocks)[:, :cols]


# ---------------------------------------------------------------- layer norm

def layer_norm(x, w, b, eps):
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + eps)
    h = d * rstd
    y = h if w is None else h * w
    return (y if b is None else y + b), mean[:, 0], rstd[:, 0], h


def layer_norm_grad(dy, h, rstd, w):
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0)


# --------------------------------------------------------------- weight grad

def weight_grad(dy, h, w=None, b=None, c=None, offsets=None):
    x = h if w is None else h * w
    x = x if b is None else x + b
    if offsets is None:
        g = dy.t() @ x
    else:
        o = offsets.tolist()
        g = torch.stack([dy[s:t].t() @ x[s:t] for s, t in zip(o, o[1:])])
    return g if c is None else g + c


# -------------------------------------------------------------------- router

def route(z, k, mask, coef, renormalise):
    """Token by token: (indices, weights, counts, offsets, loss, kept, p)."""
    tokens, experts = z.shape
    idx = torch.full((tokens, k), -1, dtype=torch.int64)
    wts = torch.zeros(tokens, k, dtype=D)
    p = torch.zeros(tokens, experts, dtype=D)
    kept = 0
    for t in range(tokens):
        row = z[t].tolist()
        if (mask is not None and not mask[t]) or max(row) == -math.inf:
            continue
        kept += 1
        top = max(row)
        ex = [math.exp(v - top) for v in row]
        s = math.fsum(ex)
        p[t] = torch.tensor([v / s for v in ex], dtype=D)
        order = sorted((e for e in range(experts) if row[e] > -math.inf),
                       key=lambda e: (-row[e], e))[:k]
        total = math.fsum(p[t, e].item() for e in order)
        for j, e in enumerate(order):
            idx[t, j] = e
            wts[t, j] = p[t, e] / (total if renormalise else 1.0)
    counts = torch.bincount(idx[idx >= 0], minlength=experts)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    loss = 0.0
    if kept:
        loss = coef * experts / (k * kept * kept) * (counts.to(D) * p.sum(0)).sum().item()
    return idx, wts, counts, offsets, loss, kept, p


def route_objective(z, idx, counts, kept, coef, renormalise, dloss, dweights):
    """dloss * loss + sum dweights * weights with the choice and the counts
    held fixed: what muon_route_grad is the gradient of."""
    experts, k = z.shape[1], idx.shape[1]
    live = idx[:, 0] >= 0
    p = torch.softmax(z[live], -1)
    total = dloss * coef * experts / (k * max(kept, 1) ** 2) * (counts.to(D) * p.sum(0)).sum()
    if dweights is not None:
        at = idx[live]
        w = torch.where(at >= 0, p.gather(1, at.clamp(min=0)), torch.zeros((), dtype=D))
        if renormalise:
            w = w / w.sum(-1, keepdim=True)
        total = total + (torch.where(at >= 0, dweights[live], torch.zeros((), dtype=D)) * w).sum()
    return total


def route_grad(z, idx, counts, kept, coef, renormalise, dloss, dweights):
    experts, k = z.shape[1], idx.shape[1]
    dz = torch.zeros_like(z)
    for t in range(z.shape[0]):
        if idx[t, 0] < 0:
            continue
        p = torch.softmax(z[t], -1)
        h = dloss * coef * experts / (k * max(kept, 1) ** 2) * counts.to(D)
        if dweights is not None:
            e = idx[t][idx[t] >= 0]
            d = dweights[t][idx[t] >= 0]
            if renormalise:
                s = p[e].sum()
                d = (d - (d * p[e]).sum() / s) / s
            h = h.clone()
            h[e] += d
        dz[t] = p * (h - (p * h).sum())
    return dz


# ------------------------------------------------------------------- compare

def close(got, want, bound, what):
    """|got - want| <= bound everywhere (NaN and infinities in the same
    places)."""
    got, want = to64(got), to64(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    diff = (got - want).abs()
    bound = bound.expand_as(diff) if isinstance(bound, torch.Tensor) else torch.full_like(diff, bound)
    over = fine & (diff > bound)
    if bool(over.any()):
        at = int(torch.argmax(torch.where(over, diff / bound.clamp(min=1e-300), torch.zeros_like(diff))))
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} out of bound; worst at "
                             f"{at}: {got.flatten()[at]} against {want.flatten()[at]}, bound "
                             f"{bound.flatten()[at]}")
