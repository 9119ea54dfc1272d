"""The operators of a block's training step against their 64-bit forms.

Bounds.  A sum of n fp32 terms in chains of at most L additions is off by at
most L 2^-24 times the sum of the terms' magnitudes.  A row's sums run in
chains of at most 96 (an element's place in its thread, then the tree over
the block); column sums over rows of at most 512 (the rows of one partial sum,
then the partial sums).  Products are rounded once more, and outputs once to
their type.  The weight gradient's products are exact; the tensor cores add
in steps of 16 and may truncate (2^-23 a step)."""
import math

import pytest
import torch

import ops_oracle as O
from ops_oracle import D, OUT_ROUND, U32, close, to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
ROW = 96 * U32
COL = 512 * U32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def rand(seed, *shape, scale=1.0, shift=0.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def strided(t, lead, pad):
    """t as a view: `lead` elements into a buffer whose rows are `pad` longer."""
    rows, cols = t.shape
    buf = torch.zeros(rows * (cols + pad) + lead + 8, dtype=t.dtype, device=t.device)
    v = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


# ---------------------------------------------------------------- checkpoint

SHAPES8 = [(1, 1), (1, 31), (3, 32), (2, 33), (7, 64), (5, 100), (64, 768), (33, 2048),
           (3, 4099), (2, 7168), (517, 257)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES8)
def test_checkpoint_is_the_code_of_its_values(ns, shape, dtype):
    x = rand(1, *shape, scale=3.0, dtype=dtype)
    c = ns.checkpoint8(x)
    q, e = O.encode(to64(x))
    assert torch.equal(c.q.cpu().long(), q) and torch.equal(c.e.cpu().long(), e)
    for t in (BF, F32):
        assert torch.equal(to64(c.values(t)), O.decode(q, e, shape[1]))


def test_checkpoint_edges(ns):
    """Magnitudes from the smallest to the largest, zeros of both signs, ties,
    the limit at 127, infinities and NaNs (their block alone reads as NaN)."""
    rows = []
    for p in (-149, -140, -133, -127, -126, -125, -60, -1, 0, 1, 60, 120, 126, 127):
        base = torch.ldexp(torch.ones(32, dtype=D), torch.tensor(p))
        rows.append(base * (torch.arange(32, dtype=D) / 16 - 1))
    rows.append(torch.zeros(32, dtype=D))
    rows.append(torch.full((32,), -0.0, dtype=D))
    rows.append((torch.arange(32, dtype=D) + 0.5) / 64)          # ties
    rows.append(2.0 - torch.ldexp(torch.ones(32, dtype=D), -torch.arange(32)))   # up to the limit
    rows.append(torch.full((32,), torch.finfo(F32).max, dtype=D))
    rows.append(torch.full((32,), torch.finfo(F32).min, dtype=D))
    x = torch.stack(rows)
    wide = torch.cat([x, x.flip(0), torch.ones_like(x)], 1).to(F32)
    for r, bad in enumerate((math.inf, -math.inf, math.nan)):
        wide[r, 40 + r] = bad
    c = ns.checkpoint8(wide.to(DEV))
    q, e = O.encode(to64(wide))
    assert torch.equal(c.q.cpu().long(), q) and torch.equal(c.e.cpu().long(), e)
    v = c.values(F32).cpu()
    assert torch.isnan(v[:3, 32:64]).all() and not torch.isnan(v[:3, :32]).any()
    close(v, O.decode(q, e, 96), 0.0, "values")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_checkpoint_of_views_and_no_rows(ns, dtype):
    x = rand(2, 37, 200, dtype=dtype)
    want = ns.checkpoint8(x)
    for lead, pad in ((1, 0), (3, 5), (8, 8), (0, 1)):
        got = ns.checkpoint8(strided(x, lead, pad))
        assert torch.equal(got.q, want.q) and torch.equal(got.e, want.e)
        out = strided(torch.zeros_like(x), lead, pad)
        assert torch.equal(want.values(out=out), want.values(dtype))
    row = x[:1].expand(9, -1)
    assert torch.equal(ns.checkpoint8(row).q, want.q[:1].expand(9, -1))
    none = ns.checkpoint8(x[:0])
    assert none.shape == (0, 200) and none.values().shape == (0, 200)
    # a wider container: what lies past the padded columns stays
    big = ns.Checkpoint8(torch.full((37, 256), 5, dtype=torch.int8, device=DEV),
                         torch.full((37, 9), 5, dtype=torch.uint8, device=DEV), 200)
    ns.checkpoint8(x, out=big)
    assert torch.equal(big.q[:, :224], want.q) and bool((big.q[:, 224:] == 5).all())
    assert torch.equal(big.e[:, :7], want.e) and bool((big.e[:, 7:] == 5).all())


# ---------------------------------------------------------------- layer norm

NORM_SHAPES = [(1, 1), (3, 2), (1, 7), (5, 32), (64, 2048), (3, 33), (17, 768), (130, 100),
               (2, 4099), (9, 7168), (2, 16384), (1, 40000), (700, 264)]


def norm_bounds(x, mean, rstd, h):
    """Bound on the error of h (fp32 arithmetic) for 64-bit x and statistics."""
    mag = x.abs().mean(-1, keepdim=True)
    d_mean = ROW * mag + 2 * U32 * mean[:, None].abs()
    d_h = rstd[:, None] * (d_mean + 2 * U32 * (x.abs() + mean[:, None].abs()))
    # 1 / deviation: half the relative error of the variance, whose terms are off by 2 d
    d_rel = 2 * ROW + 4 * U32 + rstd[:, None] * d_mean * 2 + 2 * U32 * rstd[:, None] * mag
    return d_mean[:, 0], d_rel[:, 0], d_h + h.abs() * d_rel


@pytest.mark.parametrize("wdtype,bias", [(BF, True), (F32, True), (F32, False), (None, False),
                                         (None, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_forward(ns, shape, dtype, wdtype, bias):
    x = rand(3, *shape, scale=2.0, shift=0.7, dtype=dtype)
    w = None if wdtype is None else rand(4, shape[1], dtype=wdtype)
    b = rand(5, shape[1], dtype=wdtype or F32) if bias else None
    y, mean, rstd = ns.layer_norm(x, w, b, eps=1e-5)
    assert y.dtype == dtype
    y64, mean64, rstd64, h = O.layer_norm(to64(x), to64(w), to64(b), 1e-5)
    d_mean, d_rel, d_h = norm_bounds(to64(x), mean64, rstd64, h)
    close(mean, mean64, d_mean, "mean")
    close(rstd, rstd64, d_rel * rstd64, "rstd")
    aw = torch.ones((), dtype=D) if w is None else to64(w).abs()
    ab = torch.zeros((), dtype=D) if b is None else to64(b).abs()
    close(y, y64, aw * d_h + 2 * U32 * (h.abs() * aw + ab) + OUT_ROUND[dtype] * y64.abs() + 1e-38, "y")


def check_saved(saved, h, d_h):
    """The checkpoint is that of some h within d_h of the 64-bit one."""
    cols = h.shape[1]
    v = O.decode(saved.q, saved.e, cols)
    e = saved.e.cpu().int()[:, :-(-cols // 32)].repeat_interleave(32, 1)[:, :cols]
    step = torch.ldexp(torch.ones_like(h), e - 133)
    limit = saved.q.cpu()[:, :cols].abs() == 127
    close(v, h, torch.where(limit, 1.0, 0.5) * step + d_h, "saved")
    pad = torch.zeros(h.shape[0], -(-cols // 32) * 32, dtype=D)
    pad[:, :cols] = h.abs()
    top, at = pad.view(h.shape[0], -1, 32).max(-1)
    pad[:, :cols] = d_h
    slack = pad.view(h.shape[0], -1, 32).gather(2, at[..., None])[..., 0] * 2
    lo = torch.ldexp(torch.ones_like(top), saved.e.cpu().int() - 127)
    assert bool(((saved.e.cpu() == 0) | (lo <= top + slack)).all())
    assert bool((top - slack < 2 * lo).all())
    assert not saved.q.cpu()[:, cols:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_checkpoint(ns, shape, dtype):
    x = rand(6, *shape, scale=2.0, shift=-0.3, dtype=dtype)
    w, b = rand(7, shape[1]), rand(8, shape[1])
    y, rstd, saved = ns.layer_norm_checkpoint(x, w, b)
    y0, _, rstd0 = ns.layer_norm(x, w, b)
    assert torch.equal(y, y0) and torch.equal(rstd, rstd0)
    _, mean64, rstd64, h = O.layer_norm(to64(x), None, None, 1e-5)
    check_saved(saved, h, norm_bounds(to64(x), mean64, rstd64, h)[2])


@pytest.mark.parametrize("rows,cols,dtype", [(9729, 1032, BF), (10000, 1536, BF), (9800, 2048, BF),
                                             (9728, 2056, BF), (9731, 516, F32), (9728, 1024, F32),
                                             (9729, 1028, F32), (9730, 2048, F32)])
def test_layer_norm_of_many_rows(ns, rows, cols, dtype):
    """Enough rows for a warp to have a long one, the last block partly
    filled, up to the row's length where blocks take over again."""
    x = rand(25, rows, cols, scale=2.0, shift=-0.4, dtype=dtype)
    w, b = rand(26, cols), rand(27, cols)
    y, mean, rstd = ns.layer_norm(x, w, b)
    y64, mean64, rstd64, h = O.layer_norm(to64(x), to64(w), to64(b), 1e-5)
    d_mean, d_rel, d_h = norm_bounds(to64(x), mean64, rstd64, h)
    close(mean, mean64, d_mean, "mean")
    close(rstd, rstd64, d_rel * rstd64, "rstd")
    aw, ab = to64(w).abs(), to64(b).abs()
    close(y, y64, aw * d_h + 2 * U32 * (h.abs() * aw + ab) + OUT_ROUND[dtype] * y64.abs() + 1e-38, "y")
    out = strided(torch.zeros(rows, cols, dtype=dtype, device=DEV), 16, 16)
    base = out._base.clone()
    assert torch.equal(ns.layer_norm(x, w, b, out=out)[0], y)
    rest = out._base.clone()
    rest[16:16 + rows * (cols + 16)].view(rows, cols + 16)[:, :cols] = 0
    assert torch.equal(rest, base)                          # nothing outside the view
    y1, rstd1, saved = ns.layer_norm_checkpoint(x, w, b)
    assert torch.equal(y1, y) and torch.equal(rstd1, rstd)
    check_saved(saved, h, d_h)


def check_norm_grads(got, dy, h, rstd, w, dtype, d_h):
    """got: (dx, dweight, dbias); h, rstd: 64-bit, d_h: how far off the fp32 h."""
    dx, dw, db = got
    dx64, dw64, db64 = O.layer_norm_grad(dy, h, rstd, w)
    g = (dy if w is None else dy * w).abs()
    mg, mgh = g.mean(-1, keepdim=True), (g * h.abs()).mean(-1, keepdim=True)
    bound = rstd[:, None] * (ROW * (mg + h.abs() * mgh) + 8 * U32 * (g + mg + h.abs() * mgh)
                             + d_h * mgh + h.abs() * (g * d_h).mean(-1, keepdim=True))
    close(dx, dx64, bound + OUT_ROUND[dtype] * dx64.abs() + 1e-38, "dx")
    if dw is not None:
        close(dw, dw64, COL * (dy * h).abs().sum(0) + (dy.abs() * d_h).sum(0)
              + OUT_ROUND[dw.dtype] * dw64.abs() + 1e-38, "dweight")
    if db is not None:
        close(db, db64, COL * dy.abs().sum(0) + OUT_ROUND[db.dtype] * db64.abs() + 1e-38, "dbias")


@pytest.mark.parametrize("wdtype,bias", [(BF, True), (F32, False), (None, False), (None, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_backward(ns, shape, dtype, wdtype, bias):
    x = rand(9, *shape, scale=2.0, shift=0.5, dtype=dtype)
    dy = rand(10, *shape, scale=0.1, dtype=dtype)
    w = None if wdtype is None else rand(11, shape[1], dtype=wdtype)
    b = rand(12, shape[1], dtype=wdtype or F32) if bias else None
    _, mean, rstd = ns.layer_norm(x, w, b)
    got = ns.layer_norm_backward(dy, x, mean, rstd, w, b)
    assert (got[1] is None) == (w is None) and (got[2] is None) == (b is None)
    m, r = to64(mean)[:, None], to64(rstd)
    h = (to64(x) - m) * r[:, None]
    d_h = 2 * U32 * r[:, None] * (to64(x).abs() + m.abs())
    check_norm_grads(got, to64(dy), h, r, to64(w), dtype, d_h)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_layer_norm_backward_from_checkpoint(ns, shape, dtype):
    x = rand(13, *shape, dtype=dtype)
    dy = rand(14, *shape, scale=0.1, dtype=dtype)
    w, b = rand(15, shape[1]), rand(16, shape[1])
    _, rstd, saved = ns.layer_norm_checkpoint(x, w, b)
    got = ns.layer_norm_backward(dy, saved, None, rstd, w, b)
    h = O.decode(saved.q, saved.e, shape[1])
    check_norm_grads(got, to64(dy), h, to64(rstd), to64(w), dtype, torch.zeros((), dtype=D))


def test_layer_norm_gradient_against_differences(ns):
    rows, cols, step = 5, 96, 1e-4
    x, w, b = rand(17, rows, cols), rand(18, cols), rand(19, cols)
    dy, dirx, dirw, dirb = (rand(20 + i, *s) for i, s in
                            enumerate(((rows, cols), (rows, cols), (cols,), (cols,))))
    _, mean, rstd = ns.layer_norm(x, w, b)
    dx, dw, db = ns.layer_norm_backward(dy, x, mean, rstd, w, b)

    def objective(s, t, u):
        y = O.layer_norm(to64(x) + s * to64(dirx), to64(w) + t * to64(dirw), to64(b) + u * to64(dirb), 1e-5)[0]
        return (to64(dy) * y).sum().item()

    # the differences are off by about step^2 times a third derivative of the objective's size
    for got, d, args in ((dx, dirx, (1, 0, 0)), (dw, dirw, (0, 1, 0)), (db, dirb, (0, 0, 1))):
        diff = (objective(*(step * a for a in args)) - objective(*(-step * a for a in args))) / (2 * step)
        terms = to64(got) * to64(d)
        assert abs(terms.sum().item() - diff) <= 1e-5 * terms.abs().sum().item()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [200, 203])
def test_layer_norm_of_views_in_place_and_broadcast(ns, cols, dtype):
    x, dy = rand(24, 37, cols, dtype=dtype), rand(25, 37, cols, dtype=dtype)
    w, b = rand(26, cols), rand(27, cols)
    y, mean, rstd = ns.layer_norm(x, w, b)
    grads = ns.layer_norm_backward(dy, x, mean, rstd, w, b)
    _, _, saved = ns.layer_norm_checkpoint(x, w, b)
    grads8 = ns.layer_norm_backward(dy, saved, None, rstd, w, b)
    for lead, pad in ((1, 0), (3, 5), (8, 8), (0, 1)):
        xv, dyv = strided(x, lead, pad), strided(dy, lead, pad)
        out = strided(torch.zeros_like(x), lead, pad)
        assert torch.equal(ns.layer_norm(xv, w, b, out=out)[0], y)
        yv, _, sv = ns.layer_norm_checkpoint(xv, w, b)
        assert torch.equal(yv, y) and torch.equal(sv.q, saved.q) and torch.equal(sv.e, saved.e)
        for a, c in zip(ns.layer_norm_backward(dyv, xv, mean, rstd, w, b), grads):
            assert torch.equal(a, c)
        for a, c in zip(ns.layer_norm_backward(dyv, saved, None, rstd, w, b), grads8):
            assert torch.equal(a, c)
        wv, bv = torch.cat([w[:lead], w])[lead:], torch.cat([b[:pad], b])[pad:]
        assert torch.equal(ns.layer_norm(x, wv, bv)[0], y)
    xi, di = x.clone(), dy.clone()
    assert torch.equal(ns.layer_norm(xi, w, b, out=xi)[0], y)
    for a, c in zip(ns.layer_norm_backward(di, x, mean, rstd, w, b, out=di), grads):
        assert torch.equal(a, c)
    # one row for all: its gradient sums over the rows that it was spread to
    row = dy[:1].expand(37, -1)
    for a, c in zip(ns.layer_norm_backward(row, x, mean, rstd, w, b),
                    ns.layer_norm_backward(row.contiguous(), x, mean, rstd, w, b)):
        assert torch.equal(a, c)
    xr = x[:1].expand(37, -1)
    assert torch.equal(ns.layer_norm(xr, w, b)[0], y[:1].expand(37, -1))


def test_layer_norm_no_rows_constant_rows_and_bad_values(ns):
    w, b = rand(28, 64), rand(29, 64)
    none = torch.empty(0, 64, device=DEV)
    y, mean, rstd = ns.layer_norm(none, w, b)
    dx, dw, db = ns.layer_norm_backward(none, none, mean, rstd, w, b)
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()
    x = rand(30, 6, 64)
    x[0] = 3.25                      # no variance: h = 0, rstd = 1 / sqrt(eps)
    x[1] += 30000.0                  # a mean far above the deviation
    x[2, 5], x[3, 6], x[4, 7] = math.inf, -math.inf, math.nan
    y, mean, rstd = ns.layer_norm(x, w, b)
    assert torch.equal(y[0], b) and abs(rstd[0].item() - 1e5 ** 0.5) < 1e-4
    y64, mean64, rstd64, h = O.layer_norm(to64(x), to64(w), to64(b), 1e-5)
    _, d_rel, d_h = norm_bounds(to64(x), mean64, rstd64, h)
    for r in (1, 5):
        close(y[r], y64[r], to64(w).abs() * d_h[r] + 1e-5, "y")
    assert torch.isnan(y[2:5]).all() and not torch.isnan(y[[0, 1, 5]]).any()
    _, _, saved = ns.layer_norm_checkpoint(x, w, b)
    assert bool((saved.e[2:5] == 255).all()) and not saved.q[0].any()


# --------------------------------------------------------------- weight grad

def saved_of(ns, seed, t, k, scale=1.0):
    return ns.checkpoint8(rand(seed, t, k, scale=scale, dtype=BF)) if t else \
        ns.Checkpoint8.empty(0, k, DEV)


def check_weight_grad(got, dy, saved, w=None, b=None, c=None, offsets=None):
    h = O.decode(saved.q, saved.e, saved.cols)
    want = O.weight_grad(to64(dy), h, to64(w), to64(b), to64(c),
                         None if offsets is None else offsets.cpu())
    mag = O.weight_grad(to64(dy).abs(), h.abs(), None if w is None else to64(w).abs(),
                        None if b is None else to64(b).abs(), None,
                        None if offsets is None else offsets.cpu())
    t = dy.shape[0]
    bound = (t / 16 + 32) * 2.0 ** -23 * mag + OUT_ROUND[got.dtype] * want.abs() + 1e-38
    if c is not None:
        bound = bound + 2 * U32 * (mag + to64(c).abs())
    close(got, want, bound, "gradient")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (1, 8, 32), (2, 64, 64), (16, 256, 256), (64, 256, 256),
                                   (63, 40, 72), (65, 264, 520), (300, 512, 2048), (129, 257, 130),
                                   (1000, 33, 65), (4097, 128, 96), (700, 300, 1000), (2111, 768, 776)])
def test_weight_grad(ns, t, n, k, dtype):
    dy, saved = rand(40, t, n, scale=0.1, dtype=BF), saved_of(ns, 41, t, k)
    check_weight_grad(ns.weight_grad(dy, saved, dtype=dtype), dy, saved)
    w, b, c = rand(42, k), rand(43, k), rand(44, n, k, dtype=dtype)
    check_weight_grad(ns.weight_grad(dy, saved, weight=w, bias=b, add=c, dtype=dtype),
                      dy, saved, w, b, c)
    check_weight_grad(ns.weight_grad(dy, saved, weight=w, dtype=dtype), dy, saved, w)
    check_weight_grad(ns.weight_grad(dy, saved, bias=b, dtype=dtype), dy, saved, None, b)
    # accumulated in place
    g = c.clone()
    assert ns.weight_grad(dy, saved, add=g, out=g) is g
    check_weight_grad(g, dy, saved, None, None, c)


@pytest.mark.parametrize("counts", [[5], [0], [0, 0, 0], [1, 0, 2, 63, 64, 65, 0, 200, 1],
                                    [300, 0, 0, 0], [0, 0, 17], [128, 128, 128], [7] * 40,
                                    [2500, 3]])
@pytest.mark.parametrize("n,k,dtype", [(64, 96, BF), (264, 520, F32), (100, 33, BF)])
def test_weight_grad_of_experts(ns, counts, n, k, dtype):
    t = sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    dy, saved = rand(45, t, n, scale=0.1, dtype=BF), saved_of(ns, 46, t, k)
    got = ns.weight_grad(dy, saved, offsets=offsets, dtype=dtype)
    assert got.shape == (len(counts), n, k)
    check_weight_grad(got, dy, saved, offsets=offsets)
    w, b, c = rand(47, k), rand(48, k), rand(49, len(counts), n, k, dtype=dtype)
    got = ns.weight_grad(dy, saved, weight=w, bias=b, add=c, offsets=offsets, dtype=dtype)
    check_weight_grad(got, dy, saved, w, b, c, offsets)


def test_weight_grad_experts_do_not_see_each_other(ns):
    """An expert whose tokens hold NaN and infinities leaves the others as
    they are, whatever tile their rows share."""
    counts = [30, 3, 61, 2, 100]
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    t = sum(counts)
    dy, x = rand(50, t, 96, dtype=BF), rand(51, t, 160, dtype=BF)
    clean = ns.weight_grad(dy, ns.checkpoint8(x), offsets=offsets)
    for bad in (1, 3):
        d2, x2 = dy.clone(), x.clone()
        d2[offsets[bad]:offsets[bad + 1]] = math.nan
        x2[offsets[bad]:offsets[bad + 1]] = math.inf
        got = ns.weight_grad(d2, ns.checkpoint8(x2), offsets=offsets)
        for e in range(5):
            if e == bad:
                assert torch.isnan(got[e]).all()
            else:
                assert torch.equal(got[e], clean[e]), e


def test_weight_grad_offsets_out_of_order_are_limited(ns):
    dy, saved = rand(52, 50, 64, dtype=BF), saved_of(ns, 53, 50, 64)
    offsets = torch.tensor([-5, 20, 10, 2000000000], dtype=torch.int32, device=DEV)
    got = ns.weight_grad(dy, saved, offsets=offsets)
    for e, (a, b) in enumerate(((0, 20), (20, 20), (10, 50))):
        part = ns.Checkpoint8(saved.q[a:b], saved.e[a:b], 64)
        check_weight_grad(got[e], dy[a:b], part)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_grad_of_views(ns, dtype):
    t, n, k = 150, 72, 104
    dy, saved = rand(54, t, n, dtype=BF), saved_of(ns, 55, t, k)
    c = rand(56, n, k, dtype=dtype)
    want = ns.weight_grad(dy, saved, add=c, dtype=dtype)
    for lead, pad in ((1, 0), (3, 5), (8, 8), (0, 1), (2, 2)):
        out = strided(torch.zeros(n, k, dtype=dtype, device=DEV), lead, pad)
        base = out._base.clone()
        got = ns.weight_grad(strided(dy, lead, pad), saved, add=strided(c, lead, pad), out=out)
        assert torch.equal(got, want)
        rest = out._base.clone()
        rest[lead:lead + n * (k + pad)].view(n, k + pad)[:, :k] = 0
        assert torch.equal(rest, base)                      # nothing outside the view
    wide = ns.Checkpoint8(torch.zeros(t, 256, dtype=torch.int8, device=DEV),
                          torch.zeros(t, 9, dtype=torch.uint8, device=DEV), k)
    ns.checkpoint8(saved.values(), out=wide)
    assert torch.equal(ns.weight_grad(dy, wide, add=c, dtype=dtype), want)
    row = dy[:1].expand(t, -1)
    assert torch.equal(ns.weight_grad(row, saved), ns.weight_grad(row.contiguous(), saved))
    three = torch.zeros(5, n + 3, k + 8, dtype=dtype, device=DEV)[1:4, :n, :k]
    offsets = torch.tensor([0, 20, 20, t], dtype=torch.int32, device=DEV)
    assert torch.equal(ns.weight_grad(dy, saved, offsets=offsets, out=three),
                       ns.weight_grad(dy, saved, offsets=offsets, dtype=dtype))


@pytest.mark.parametrize("t,n,k", [(1000, 2300, 2100), (1100, 6000, 6400), (961, 2304, 2304),
                                   (1025, 2049, 2305)])
def test_weight_grad_of_many_tiles(ns, t, n, k):
    """Long sums and enough tiles for several a pair: bf16 takes tiles of 512
    rows there (sizes with whole ones, with half of one, with a ragged end)."""
    dy, saved = rand(57, t, n, scale=0.1, dtype=BF), saved_of(ns, 58, t, k)
    got = ns.weight_grad(dy, saved)
    check_weight_grad(got, dy, saved)
    for lead, pad in ((8, 8), (1, 3)):
        out = strided(torch.zeros(n, k, dtype=BF, device=DEV), lead, pad)
        base = out._base.clone()
        assert torch.equal(ns.weight_grad(dy, saved, out=out), got)
        rest = out._base.clone()
        rest[lead:lead + n * (k + pad)].view(n, k + pad)[:, :k] = 0
        assert torch.equal(rest, base)                      # nothing outside the view
    w, b, c = rand(59, k), rand(60, k), rand(61, n, k, dtype=BF)
    check_weight_grad(ns.weight_grad(dy, saved, weight=w, bias=b, add=c), dy, saved, w, b, c)


def test_weight_grad_of_long_sums(ns):
    """Hundreds of steps a tile with all stages in flight; the same every
    time."""
    dy, saved = rand(67, 16384, 4096, scale=0.1, dtype=BF), saved_of(ns, 68, 16384, 4096)
    got = ns.weight_grad(dy, saved)
    check_weight_grad(got, dy, saved)
    for _ in range(5):
        assert torch.equal(ns.weight_grad(dy, saved), got)


@pytest.mark.parametrize("counts,n,k", [([3000, 0, 1, 4000, 63, 2900], 1024, 1500),
                                        ([2000, 2111, 0, 1900], 1100, 2050)])
def test_weight_grad_of_experts_with_many_tokens(ns, counts, n, k):
    t = sum(counts)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
    dy, saved = rand(62, t, n, scale=0.1, dtype=BF), saved_of(ns, 63, t, k)
    check_weight_grad(ns.weight_grad(dy, saved, offsets=offsets), dy, saved, offsets=offsets)
    w, b, c = rand(64, k), rand(65, k), rand(66, len(counts), n, k, dtype=BF)
    got = ns.weight_grad(dy, saved, weight=w, bias=b, add=c, offsets=offsets)
    check_weight_grad(got, dy, saved, w, b, c, offsets)


def test_weight_grad_scales_over_their_whole_range(ns):
    """Blocks from the smallest scale to the largest: powers of two pass
    through exactly; a block that held a NaN makes its columns NaN."""
    p = torch.tensor([-126, -100, -60, -7, 0, 3, 60, 100, 120])
    x = torch.ldexp(torch.ones(9, 1), p[:, None]).expand(9, 288).clone()
    for i in range(9):
        keep = torch.zeros(288)
        keep[32 * i:32 * i + 32] = 1
        x[i] = x[i] * keep
    dy = torch.zeros(9, 16, dtype=BF)
    dy[:, :9] = torch.eye(9, dtype=BF)
    got = ns.weight_grad(dy.to(DEV), ns.checkpoint8(x.to(DEV)), dtype=F32)
    assert torch.equal(got.cpu()[:9], x)
    x[4, 130] = math.nan
    got = ns.weight_grad(dy.to(DEV), ns.checkpoint8(x.to(DEV)), dtype=F32).cpu()
    assert torch.isnan(got[:, 128:160]).all() and not torch.isnan(got[:, :128]).any()


def test_weight_grad_feeds_the_step(ns):
    """The gradient written into a Muon set's own G is the one its step reads."""
    n, k, t = 256, 512, 200
    W, M = rand(57, n, k, scale=0.02, dtype=BF), torch.zeros(n, k, device=DEV)
    G = torch.zeros(n, k, dtype=BF, device=DEV)
    opt = ns.Muon([(W, G, M)])
    dy, saved = rand(58, t, n, dtype=BF), saved_of(ns, 59, t, k)
    ns.weight_grad(dy, saved, out=G)
    opt.step(lr=0.02, beta=0.95)
    opt.sync()
    assert torch.equal(M, G.float())
    opt.close()


# -------------------------------------------------------------------- router

ROUTE_SHAPES = [(1, 1, 1), (5, 4, 2), (200, 128, 8), (33, 7, 7), (64, 32, 1), (17, 33, 3),
                (9, 384, 8), (3, 1000, 32), (4, 1024, 5), (100, 64, 6), (1000, 12, 2)]


def check_route(r, z, k, mask, coef, renormalise):
    idx, w, counts, offsets, loss, kept, p = O.route(to64(z), k, None if mask is None else mask.cpu(),
                                                     coef, renormalise)
    assert torch.equal(r.indices.cpu().long(), idx)
    assert torch.equal(r.counts.cpu().long(), counts) and int(r.kept) == kept
    assert torch.equal(r.offsets.cpu().long(), offsets)
    # exp is good to 2^-22, its argument to 2^-24 of its magnitude
    zz = to64(z)
    spread = torch.where(torch.isfinite(zz), zz, torch.zeros((), dtype=D)).abs().max().item()
    rel = (2 * spread + 8 + 96) * U32 + 2.0 ** -22
    close(r.weights, w, 3 * rel * w + 1e-38, "weights")
    assert abs(r.loss.item() - loss) <= (2 * rel + COL) * abs(loss)
    return idx, counts, kept, rel


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tokens,experts,k", ROUTE_SHAPES)
def test_route_and_its_gradient(ns, tokens, experts, k, dtype, renormalise):
    z = rand(60, tokens, experts, scale=2.0, dtype=dtype)
    r = ns.route(z, k, coef=0.1, renormalise=renormalise)
    idx, counts, kept, rel = check_route(r, z, k, None, 0.1, renormalise)
    dw = rand(61, tokens, k)
    dloss = torch.tensor(0.7, device=DEV)
    for a, d in ((None, dw), (dloss, None), (dloss, dw)):
        got = ns.route_backward(z, r, dloss=a, dweights=d)
        assert got.dtype == dtype
        want = O.route_grad(to64(z), idx, counts, kept, 0.1, renormalise,
                            0.0 if a is None else float(a), to64(d))
        p = torch.softmax(to64(z), -1)
        up = torch.zeros_like(p)
        if d is not None:
            s = p.gather(1, idx).sum(-1, keepdim=True) if renormalise else 1.0
            up.scatter_(1, idx, (to64(d).abs() + to64(d).abs().amax(-1, keepdim=True)) / s)
        if a is not None:
            up = up + float(a) * 0.1 * experts / (k * kept * kept) * counts.to(D)
        close(got, want, 6 * rel * p * (up + (p * up).sum(-1, keepdim=True))
              + OUT_ROUND[dtype] * want.abs() + 1e-38, "dlogits")


@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient_against_differences(ns, renormalise):
    z = rand(62, 7, 20)
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1], dtype=torch.bool, device=DEV)
    r = ns.route(z, 3, mask=mask, coef=0.5, renormalise=renormalise)
    dw, dloss = rand(63, 7, 3), torch.tensor(1.3, device=DEV)
    got = to64(ns.route_backward(z, r, dloss=dloss, dweights=dw))
    step = 1e-5
    for seed in (64, 65):
        d = to64(rand(seed, 7, 20))
        args = (to64(r.indices).long(), to64(r.counts), int(r.kept), 0.5, renormalise, 1.3, to64(dw))
        diff = (O.route_objective(to64(z) + step * d, *args)
                - O.route_objective(to64(z) - step * d, *args)).item() / (2 * step)
        terms = got * d
        assert abs(terms.sum().item() - diff) <= 1e-5 * terms.abs().sum().item()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_ties_go_to_the_lowest_index(ns, dtype):
    z = torch.zeros(6, 100, dtype=dtype, device=DEV)
    z[1, 50:] = 1.0
    z[2, ::2] = -1.0
    z[3, 99] = z[3, 0] = 2.0
    z[4] = -0.0
    z[4, ::3] = 0.0                                  # the two zeros are equal
    z[5] = torch.finfo(dtype).min                    # the type's lowest value is a value
    r = ns.route(z, 5, coef=0.1)
    check_route(r, z, 5, None, 0.1, True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_masks_and_empty_rows(ns, dtype, renormalise):
    z = rand(66, 40, 12, dtype=dtype)
    z[3] = -math.inf                                 # nothing left
    z[4, 1:] = -math.inf                             # one expert for three places
    z[5, :10] = -math.inf
    z[6, 2:5] = torch.finfo(dtype).min
    mask = torch.ones(40, dtype=torch.uint8, device=DEV)
    mask[7:9] = 0
    z[7], z[8, 3] = math.nan, math.inf               # behind the mask anything may stand
    r = ns.route(z, 3, mask=mask, coef=0.1, renormalise=renormalise)
    clean = z.clone()
    clean[7:9] = 0
    idx, counts, kept, rel = check_route(r, clean, 3, mask, 0.1, renormalise)
    assert kept == 37
    dw = rand(67, 40, 3)
    dw[3], dw[7], dw[4, 1:] = math.nan, math.inf, math.nan      # places that hold nothing
    dloss = torch.tensor(1.0, device=DEV)
    got = ns.route_backward(z, r, dloss=dloss, dweights=dw)
    assert not got[[3, 7, 8]].any()
    want = O.route_grad(to64(clean), idx, counts, kept, 0.1, renormalise, 1.0, to64(dw))
    close(got, want, 40 * rel * to64(dw)[idx >= 0].abs().max().item()
          + OUT_ROUND[dtype] * want.abs(), "dlogits")
    # all tokens masked, and no tokens at all
    r = ns.route(z, 3, mask=torch.zeros_like(mask), coef=0.1, renormalise=renormalise)
    assert float(r.loss) == 0.0 and int(r.kept) == 0 and not r.counts.any() and not r.offsets.any()
    assert bool((r.indices == -1).all()) and not r.weights.any()
    assert not ns.route_backward(z, r, dloss=dloss, dweights=dw).any()
    r = ns.route(z[:0], 3)
    assert float(r.loss) == 0.0 and int(r.kept) == 0 and not r.offsets.any()
    assert ns.route_backward(z[:0], r, dloss=dloss).shape == (0, 12)


def test_route_nan_and_infinity_show(ns):
    z = rand(68, 4, 40)
    z[1, 30], z[2, 5] = math.nan, math.inf
    r = ns.route(z, 2)
    assert torch.isnan(r.weights[1:3]).all() and not torch.isnan(r.weights[[0, 3]]).any()
    assert math.isnan(float(r.loss)) and int(r.kept) == 4
    assert int(r.indices[1, 0]) == 30 and int(r.indices[2, 0]) == 5
    dz = ns.route_backward(z, r, dloss=torch.tensor(1.0, device=DEV))
    assert torch.isnan(dz[1:3]).all() and not torch.isnan(dz[[0, 3]]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_of_views(ns, dtype):
    z, dw = rand(69, 21, 48, dtype=dtype), rand(70, 21, 4)
    r = ns.route(z, 4)
    dz = ns.route_backward(z, r, dweights=dw)
    for lead, pad in ((1, 0), (3, 5), (8, 8), (0, 1)):
        zv = strided(z, lead, pad)
        rv = ns.route(zv, 4)
        for name in ("indices", "weights", "counts", "offsets", "loss", "kept"):
            assert torch.equal(getattr(rv, name), getattr(r, name))
        out = strided(torch.zeros_like(z), lead, pad)
        assert torch.equal(ns.route_backward(zv, r, dweights=strided(dw, lead, pad), out=out), dz)
    zi = z.clone()
    assert torch.equal(ns.route_backward(zi, r, dweights=dw, out=zi), dz)
    row = dw[:1].expand(21, -1)
    assert torch.equal(ns.route_backward(z, r, dweights=row),
                       ns.route_backward(z, r, dweights=row.contiguous()))


# ------------------------------------------------------- streams, repeats, sets

def test_operators_on_another_stream_and_again(ns):
    """Queued on a side stream behind its inputs' producer, every operator
    gives the bits that it gives on the default stream; and again each time."""
    x, dy, w, b = rand(71, 300, 264, dtype=BF), rand(72, 300, 264, dtype=BF), rand(73, 264), rand(74, 264)

    def everything(x, dy):
        y, rstd, saved = ns.layer_norm_checkpoint(x, w, b)
        r = ns.route(y, 4)
        return [y, rstd, saved.q, saved.e, *ns.layer_norm_backward(dy, saved, None, rstd, w, b),
                ns.weight_grad(dy, saved, weight=w, bias=b, dtype=F32), r.indices, r.weights,
                r.loss, ns.route_backward(y, r, dloss=torch.ones((), device=DEV))]

    want = everything(x, dy)
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            x2, dy2 = x * 1, dy * 1
            got = everything(x2, dy2)
        torch.cuda.default_stream().wait_stream(side)
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    ns.ops_sync()
    with torch.cuda.stream(side):
        ns.ops_sync()


def test_operators_in_a_captured_graph(ns):
    x, dy, w = rand(75, 130, 520, dtype=BF), rand(76, 130, 520, dtype=BF), rand(77, 520)

    def everything():
        y, rstd, saved = ns.layer_norm_checkpoint(x, w)
        r = ns.route(y, 4)
        return [y, *ns.layer_norm_backward(dy, saved, None, rstd, w)[:2],
                ns.weight_grad(dy, saved, weight=w), r.indices, r.loss,
                ns.route_backward(y, r, dloss=torch.ones((), device=DEV))]

    everything()
    torch.cuda.synchronize()
    one = torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        got = everything()
    for seed in (78, 79):
        x.copy_(rand(seed, 130, 520, dtype=BF))
        one.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, everything()):
            assert torch.equal(a, c)


# ------------------------------------------------------ together, and far out

def test_example_block_trains():
    """The operators together, as a training step uses them: the block's
    gradients are those of the same block with autograd in fp64, within what
    bf16 and 8-bit activations cost, and its loss falls."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_moe_block.py")
    spec = importlib.util.spec_from_file_location("train_moe_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.Block(64, 32, 8, 2)
    x = rand(80, 128, 64, dtype=BF)
    out = block.forward(x)
    dout = rand(81, 128, 64)
    dx = block.backward(dout)
    r = block.kept[3]
    leaves = [t.to("cpu", D).requires_grad_() for t in (x, block.router, block.w1, block.w2, block.gain,
                                                        block.shift)]
    xr, router, w1, w2, gain, shift = leaves
    y = torch.nn.functional.layer_norm(xr, (64,), gain, shift)
    p = torch.softmax(y @ router.t(), -1)
    idx = r.indices.cpu().long()
    w = p.gather(1, idx)
    w = w / w.sum(-1, keepdim=True)
    # which units are active is the block's choice, as the experts taken are: a ReLU that
    # switches by a rounding is no error of a gradient
    order, active = block.kept[4].cpu(), block.kept[8].cpu()
    on = torch.empty(128 * 2, 32, dtype=torch.bool)
    on[order] = active
    u = torch.einsum("tkih,th->tki", w1[idx], y) * on.view(128, 2, 32)
    ref = xr + (w[..., None] * torch.einsum("tkhi,tki->tkh", w2[idx], u)).sum(1)
    counts = torch.bincount(idx.flatten(), minlength=8).to(D)
    balance = 0.01 * 8 / (2 * 128) * (counts * p.mean(0)).sum()
    ((ref * to64(dout)).sum() + balance).backward()
    # every value has passed about six roundings to bf16 (2^-9 each) and one to 8 bits (2^-7 of
    # its block's largest, to nearest): a few percent of the norm
    for got, want in ((out, ref), (dx, xr.grad), (block.g_router, router.grad), (block.g_w1, w1.grad),
                      (block.g_w2, w2.grad), (block.d_gain, gain.grad), (block.d_shift, shift.grad)):
        want = want.detach()
        assert (to64(got) - want).norm() <= 0.06 * want.norm()
    block.muon.close()
    losses = ex.train(steps=25, tokens=512, hidden=128, inner=64, experts=8)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5]), losses


def _needs(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_layer_norm_past_32_bits(ns):
    """Rows whose elements lie past 2^31, forward, checkpoint and backward: the
    same bits as the same rows on their own."""
    _needs(32)
    rows, cols, n = 270000, 8192, 40
    x = torch.empty(rows, cols, dtype=BF, device=DEV)
    x.view(-1).view(torch.int16).random_(0x3c00, 0x4000)        # bf16 between 2^-7 and 2
    w, b = rand(82, cols), rand(83, cols)
    y, rstd, saved = ns.layer_norm_checkpoint(x, w, b)
    tail = x[-n:].clone()
    y1, rstd1, saved1 = ns.layer_norm_checkpoint(tail, w, b)
    assert torch.equal(rstd[-n:], rstd1)
    close(y[-n:], y1, 2.0 ** -7 * to64(y1).abs() + 1e-5, "y")
    assert (saved.q[-n:].int() - saved1.q.int()).abs().max() <= 1
    dx, dw, db = ns.layer_norm_backward(x, saved, None, rstd, w, b)
    dx1, _, _ = ns.layer_norm_backward(tail, ns.Checkpoint8(saved.q[-n:], saved.e[-n:], cols), None,
                                       rstd[-n:], w, b)
    close(dx[-n:], dx1, 2.0 ** -7 * to64(dx1).abs() + 1e-4, "dx")
    want = x[:, :8].sum(0, dtype=D)
    close(db[:8], want, 1e-4 * to64(want).abs(), "dbias")       # rows of one part add up in chains of 900
    del y, dx
    v = saved.values()
    assert torch.equal(v[-n:], ns.Checkpoint8(saved.q[-n:], saved.e[-n:], cols).values())
    c = ns.checkpoint8(x)
    assert torch.equal(c.q[-n:], ns.checkpoint8(tail).q)


def test_weight_grad_past_32_bits(ns):
    """Tokens whose elements lie past 2^31, and a result that passes it."""
    _needs(32)
    t, n, k = 560000, 4096, 256
    dy = torch.empty(t, n, dtype=BF, device=DEV)
    dy.view(-1).view(torch.int16).random_(0x3c00, 0x4000)
    saved = ns.checkpoint8(rand(84, 200, k, dtype=BF))
    q = torch.zeros(t, k, dtype=torch.int8, device=DEV)
    e = torch.zeros(t, k // 32, dtype=torch.uint8, device=DEV)
    q[-200:], e[-200:] = saved.q, saved.e
    offsets = torch.tensor([0, 3, t - 200, t], dtype=torch.int32, device=DEV)
    got = ns.weight_grad(dy, ns.Checkpoint8(q, e, k), offsets=offsets, dtype=F32)
    check_weight_grad(got[2], dy[-200:], saved)
    assert not got[:2].any()
    del dy, q, e, got
    torch.cuda.empty_cache()
    dy = rand(85, 6, 300, dtype=BF)
    saved = ns.checkpoint8(rand(86, 6, 512, dtype=BF))
    big = torch.empty(15000, 300, 512, dtype=BF, device=DEV)
    offsets = torch.zeros(15001, dtype=torch.int32, device=DEV)
    offsets[14000:] = 6
    ns.weight_grad(dy, saved, offsets=offsets, out=big)
    check_weight_grad(big[13999], dy, saved)
    assert not big[14000:].any() and not big[:13999:700].any()


def test_route_past_32_bits(ns):
    _needs(24)
    t, experts, k = 2200000, 1024, 4
    z = torch.empty(t, experts, dtype=BF, device=DEV)
    z.view(-1).view(torch.int16).random_(0x3c00, 0x4080)
    r = ns.route(z, k, coef=1.0)
    n = 50
    r1 = ns.route(z[-n:].clone(), k)
    assert torch.equal(r.indices[-n:], r1.indices) and torch.equal(r.weights[-n:], r1.weights)
    assert int(r.kept) == t and int(r.offsets[-1]) == t * k == int(r.counts.sum())
    assert abs(float(r.loss) - 1.0) < 0.01                      # an even load: E * sum of f P is about 1
    dz = ns.route_backward(z, r, dloss=torch.ones((), device=DEV), dweights=torch.ones_like(r.weights))
    assert bool(torch.isfinite(dz[-n:].float()).all())
