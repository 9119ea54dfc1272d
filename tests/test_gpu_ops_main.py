"""The operators at sizes at which a block or a warp has several rows, tokens or
tiles one after the other, as the main sizes have: rings that wrap, phases that
turn, reads ahead, sums over a block's rows, several chunks of a sum.

Bounds as in test_gpu_ops; a column sum's chain is the rows of one partial sum
(at most rows / 152 of them) and the partial sums (at most 80 in a row)."""
import pytest
import torch

import ops_oracle as O
from ops_oracle import D, OUT_ROUND, U32, close, to64
from test_gpu_ops import (COL, check_norm_grads, check_saved, check_weight_grad, norm_bounds, rand,
                          saved_of, strided)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


# ---------------------------------------------------------------- layer norm

# by lanes of 8, 16 and 32; one, two and four vectors a thread through the ring,
# on 16 bytes and off it; rows longer than a block's registers
ROWS = [(20000, 64, BF), (20001, 100, BF), (20000, 128, F32), (12000, 200, BF), (11000, 250, BF),
        (2000, 264, BF), (2001, 263, F32), (4000, 1032, BF), (4099, 2048, F32), (4099, 7168, BF),
        (1500, 7167, BF), (2500, 4096, F32), (1300, 4099, F32), (1000, 16384, BF), (700, 16383, BF),
        (700, 16384, F32), (500, 12001, F32), (3, 70000, BF), (130, 33000, F32), (130, 70001, BF)]


@pytest.mark.parametrize("rows,cols,dtype", ROWS)
def test_layer_norm_forward_of_several_rows_a_block(ns, rows, cols, dtype):
    assert COL >= (rows / 152 + 80) * U32
    x = rand(1, rows, cols, scale=2.0, shift=0.3, dtype=dtype)
    w, b = rand(2, cols), rand(3, cols)
    y, mean, rstd = ns.layer_norm(x, w, b)
    y64, mean64, rstd64, h = O.layer_norm(to64(x), to64(w), to64(b), 1e-5)
    d_mean, d_rel, d_h = norm_bounds(to64(x), mean64, rstd64, h)
    close(mean, mean64, d_mean, "mean")
    close(rstd, rstd64, d_rel * rstd64, "rstd")
    aw, ab = to64(w).abs(), to64(b).abs()
    close(y, y64, aw * d_h + 2 * U32 * (h.abs() * aw + ab) + OUT_ROUND[dtype] * y64.abs() + 1e-38, "y")
    y8, rstd8, saved = ns.layer_norm_checkpoint(x, w, b)
    assert torch.equal(y8, y) and torch.equal(rstd8, rstd)
    check_saved(saved, h, d_h)
    xi = x.clone()
    assert torch.equal(ns.layer_norm(xi, w, b, out=xi)[0], y)


@pytest.mark.parametrize("from_checkpoint", [False, True])
@pytest.mark.parametrize("rows,cols,dtype", ROWS)
def test_layer_norm_backward_of_several_rows_a_block(ns, rows, cols, dtype, from_checkpoint):
    x = rand(4, rows, cols, scale=2.0, shift=0.5, dtype=dtype)
    dy = rand(5, rows, cols, scale=0.1, dtype=dtype)
    w, b = rand(6, cols), rand(7, cols)
    if from_checkpoint:
        _, rstd, x = ns.layer_norm_checkpoint(x, w, b)
        mean, h, d_h = None, O.decode(x.q, x.e, cols), torch.zeros((), dtype=D)
    else:
        _, mean, rstd = ns.layer_norm(x, w, b)
        h = (to64(x) - to64(mean)[:, None]) * to64(rstd)[:, None]
        d_h = 2.01 * U32 * h.abs()
    got = ns.layer_norm_backward(dy, x, mean, rstd, w, b)
    check_norm_grads(got, to64(dy), h, to64(rstd), to64(w), dtype, d_h)
    for g, again in zip(got, ns.layer_norm_backward(dy, x, mean, rstd, w, b)):
        assert torch.equal(g, again)
    # in place, and into a view that leaves what is around it as it was
    di = dy.clone()
    assert torch.equal(ns.layer_norm_backward(di, x, mean, rstd, w, b, out=di)[0], got[0])
    out = strided(torch.zeros_like(dy), 16, 16)
    base = out._base.clone()
    dx = ns.layer_norm_backward(dy, x, mean, rstd, w, b, out=out)[0]
    close(dx, got[0], 2 * OUT_ROUND[dtype] * to64(got[0]).abs() + 1e-38, "dx")
    rest = out._base.clone()
    rest[16:16 + rows * (cols + 16)].view(rows, cols + 16)[:, :cols] = 0
    assert torch.equal(rest, base)


# --------------------------------------------------------------- weight grad

def check_chunked(got, dy, saved, w, b, c, offsets=None):
    """fp32 results: chunks of 1024 tokens (64 products of two cuts of 2^-23),
    one rounding each, and those of the epilogue.  C and the products' sums of
    magnitudes as in check_weight_grad."""
    h = O.decode(saved.q, saved.e, saved.cols)
    o = None if offsets is None else offsets.cpu()
    a64 = [None if v is None else to64(v) for v in (w, b, c)]
    want = O.weight_grad(to64(dy), h, *a64, o)
    mag = O.weight_grad(to64(dy).abs(), h.abs(), *(None if v is None else v.abs() for v in a64[:2]), None, o)
    longest = dy.shape[0] if o is None else int((o[1:] - o[:-1]).max())
    bound = (128 * 2.0 ** -23 + (longest / 1024 + 40) * U32) * mag + OUT_ROUND[F32] * want.abs() + 1e-38
    if c is not None:
        bound = bound + 2 * U32 * (mag + a64[2].abs())
    close(got, want, bound, "gradient")


@pytest.mark.parametrize("t,n,k", [(4097, 4096, 2048), (3137, 2300, 2100), (5000, 2049, 2305)])
def test_weight_grad_fp32_of_several_chunks_and_tiles(ns, t, n, k):
    dy, saved = rand(8, t, n, scale=0.1, dtype=BF), saved_of(ns, 9, t, k)
    got = ns.weight_grad(dy, saved, dtype=F32)
    check_chunked(got, dy, saved, None, None, None)
    for lead, pad in ((4, 4), (1, 3)):
        out = strided(torch.zeros(n, k, device=DEV), lead, pad)
        base = out._base.clone()
        assert torch.equal(ns.weight_grad(dy, saved, out=out), got)
        rest = out._base.clone()
        rest[lead:lead + n * (k + pad)].view(n, k + pad)[:, :k] = 0
        assert torch.equal(rest, base)
    w, b, c = rand(10, k), rand(11, k), rand(12, n, k)
    check_chunked(ns.weight_grad(dy, saved, weight=w, bias=b, add=c, dtype=F32), dy, saved, w, b, c)


def test_weight_grad_fp32_of_long_sums(ns):
    dy, saved = rand(13, 16384, 4096, scale=0.1, dtype=BF), saved_of(ns, 14, 16384, 4096)
    got = ns.weight_grad(dy, saved, dtype=F32)
    check_chunked(got[:512], dy[:, :512], saved, None, None, None)
    for _ in range(5):
        assert torch.equal(ns.weight_grad(dy, saved, dtype=F32), got)


@pytest.mark.parametrize("counts,n,k", [([3000, 0, 1, 4000, 63, 2900], 1024, 1500),
                                        ([2000, 2111, 0, 1900], 1100, 2050)])
def test_weight_grad_fp32_of_experts_with_many_tokens(ns, counts, n, k):
    t = sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    dy, saved = rand(15, t, n, scale=0.1, dtype=BF), saved_of(ns, 16, t, k)
    check_chunked(ns.weight_grad(dy, saved, offsets=offsets, dtype=F32), dy, saved, None, None, None, offsets)
    w, b, c = rand(17, k), rand(18, k), rand(19, len(counts), n, k)
    got = ns.weight_grad(dy, saved, weight=w, bias=b, add=c, offsets=offsets, dtype=F32)
    check_chunked(got, dy, saved, w, b, c, offsets)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_grad_of_short_tiles_again_and_again(ns, dtype):
    """Many tiles of a few steps each, some of none, for every pair: the same
    every time."""
    counts = [(37 * e * e) % 331 for e in range(60)]
    t = sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    dy, saved = rand(20, t, 520, scale=0.1, dtype=BF), saved_of(ns, 21, t, 776)
    got = ns.weight_grad(dy, saved, offsets=offsets, dtype=dtype)
    check_weight_grad(got, dy, saved, offsets=offsets)
    for _ in range(20):
        assert torch.equal(ns.weight_grad(dy, saved, offsets=offsets, dtype=dtype), got)


# -------------------------------------------------------------------- router

def route64(z, k, keep, coef, renormalise):
    """ops_oracle.route for all tokens at once."""
    p = torch.softmax(z, -1)
    order = torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, order)
    if renormalise:
        w = w / w.sum(-1, keepdim=True)
    idx = torch.where(keep[:, None], order, -1)
    w = torch.where(keep[:, None], w, 0.0)
    p = p * keep[:, None]
    counts = torch.bincount(idx[idx >= 0], minlength=z.shape[1])
    kept = int(keep.sum())
    loss = coef * z.shape[1] / (k * kept * kept) * (counts.to(D) * p.sum(0)).sum().item()
    return idx, w, counts, loss, kept, p


def route_grad64(p, idx, w, counts, kept, coef, renormalise, dloss, dw):
    """ops_oracle.route_grad for all tokens at once; also the size of its terms."""
    live = idx >= 0
    at = idx.clamp(min=0)
    d, size = dw * live, dw.abs() * live
    if renormalise:
        s = p.gather(1, at).sum(-1, keepdim=True).clamp(min=1e-300)
        d = (d - (d * w).sum(-1, keepdim=True)) / s * live
        size = (size + (size * w).sum(-1, keepdim=True)) / s * live
    factor = dloss * coef * p.shape[1] / (idx.shape[1] * kept * kept) * counts.to(D)
    h = factor.expand_as(p).scatter_add(1, at, d)
    big = factor.expand_as(p).scatter_add(1, at, size)
    return p * (h - (p * h).sum(-1, keepdim=True)), p * (big + (p * big).sum(-1, keepdim=True))


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,experts,k", [(40000, 12, 2), (45001, 32, 8), (20000, 33, 4), (20003, 128, 8),
                                              (24000, 384, 8), (9000, 509, 5), (9000, 1000, 3)])
def test_route_of_several_tokens_a_warp(ns, tokens, experts, k, dtype, renormalise):
    g = torch.Generator().manual_seed(22)
    z = (2.0 * torch.randn(tokens, experts, generator=g) + torch.randn(experts, generator=g)).to(dtype)
    z[::7, : experts // 2] = z[::7, :1]                       # ties
    keep = torch.rand(tokens, generator=g) < 0.9
    dw, dloss = torch.randn(tokens, k, generator=g), 0.7
    zd = z.to(DEV)
    r = ns.route(zd, k, mask=keep.to(DEV), coef=0.1, renormalise=renormalise)
    z64 = z.to(D)
    idx, w, counts, loss, kept, p = route64(z64, k, keep, 0.1, renormalise)
    few = O.route(z64[:30], k, keep[:30], 0.1, renormalise)
    assert torch.equal(few[0], idx[:30])
    assert torch.equal(r.indices.cpu().long(), idx) and torch.equal(r.counts.cpu().long(), counts)
    assert int(r.kept) == kept
    assert torch.equal(r.offsets.cpu().long()[1:], counts.cumsum(0))
    # as in test_gpu_ops: an exponential, its argument's rounding, the sum's chain
    rel = (2 * z64.abs().max().item() + 8 + 96) * U32 + 2.0 ** -22
    close(r.weights, w, 3 * rel * w + 1e-38, "weights")
    assert abs(r.loss.item() - loss) <= (2 * rel + COL) * abs(loss)
    got = ns.route_backward(zd, r, dloss=torch.tensor(dloss, device=DEV), dweights=dw.to(DEV))
    want, size = route_grad64(p, idx, w, counts, kept, 0.1, renormalise, dloss, dw.to(D))
    close(got, want, 6 * rel * size + OUT_ROUND[dtype] * want.abs() + 1e-38, "dlogits")
    zi = zd.clone()
    assert torch.equal(ns.route_backward(zi, r, dloss=torch.tensor(dloss, device=DEV), dweights=dw.to(DEV),
                                         out=zi), got)
