"""The operators inside a block against their 64-bit forms.  Bounds are those
of block_oracle: every rounding to bf16 is off by at most half a step, sums as
the tensor cores make them, and each error is carried through what follows."""
import math

import pytest
import torch

import block_oracle as O
from block_oracle import D, HALF, U32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def rand(seed, *shape, scale=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


def strided(t, lead, pad):
    """t as a view: `lead` elements into a buffer whose rows are `pad` longer."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + lead + 8,), 7.0, dtype=t.dtype, device=t.device)
    v = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def near(got, want, bound, what):
    """|got - want| <= bound where want is finite; NaN and infinities alike."""
    got = got.to(D)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    over = fine & ((got - want).abs() > bound)
    if bool(over.any()):
        at = tuple(over.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} off, first at {at}: "
                             f"{got[at].item()} for {want[at].item()}, bound {bound[at].item():.3e}")


def close_norm(got, want, what, most=4e-3):
    """The whole is as near as roundings of random signs leave it: error and
    value of an output are sums over the same random terms, so that their squares'
    ratio is the roundings' (below 2^-8.5 each, a few of them) for many outputs.
    That of a few, where the terms may cancel, has only its bound (near)."""
    if want.numel() < 1000:
        return
    off, size = (got.to(D) - want).norm().item(), want.norm().item()
    assert off <= most * size + 1e-30, (what, off, size)


# ----------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,p", [(1, 1, 0.5), (1, 7, 0.3), (3, 8, 0.5), (64, 40, 0.1), (5, 33, 0.25),
                                         (2, 2047, 0.9), (33, 264, 0.0), (4, 16, 1.0), (3, 100, 1e-6)])
def test_dropout(ns, rows, cols, p, dtype):
    x, r = rand(1, rows, cols, dtype=dtype), rand(2, rows, cols, dtype=dtype)
    for seed, offset in ((0, 0), (123456789012345678, 987654321987), (2 ** 64 - 1, 2 ** 64 - 1)):
        for res in (None, r):
            want = O.dropout(x, p, seed, offset, res)
            got = ns.dropout(x, p, seed, offset, residual=res)
            assert got.dtype == dtype
            # the scale, the product and the sum are rounded once each
            size = want.abs() + (0 if res is None else 2 * res.cpu().to(D).abs())
            near(got.cpu(), want, (3 * U32 + HALF[dtype]) * size + 1e-38, "y")
    assert torch.equal(ns.dropout_backward(x, p, 5, 6), ns.dropout(x, p, 5, 6))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [40, 41, 2048])
def test_dropout_goes_by_the_element_not_its_address(ns, cols, dtype):
    x, r = rand(3, 29, cols, dtype=dtype), rand(4, 29, cols, dtype=dtype)
    want = ns.dropout(x, 0.4, 11, 12, residual=r)
    for lead, pad in ((0, 8), (1, 0), (3, 5), (8, 16), (0, 1)):
        out = strided(torch.zeros_like(x), lead, pad)
        base = out._base.clone()
        got = ns.dropout(strided(x, lead, pad), 0.4, 11, 12, residual=strided(r, pad, lead), out=out)
        assert got is out and torch.equal(got, want)
        rest = out._base.clone()
        rest[lead:lead + 29 * (cols + pad)].view(29, cols + pad)[:, :cols] = 0
        base[lead:lead + 29 * (cols + pad)].view(29, cols + pad)[:, :cols] = 0
        assert torch.equal(rest, base)                      # nothing outside the view
    for into in (0, 1):
        a, b = x.clone(), r.clone()
        assert torch.equal(ns.dropout(a, 0.4, 11, 12, residual=b, out=(a, b)[into]), want)
    row = ns.dropout(x[:1].expand(29, -1), 0.4, 11, 12)
    assert torch.equal(row, ns.dropout(x[:1].expand(29, -1).contiguous(), 0.4, 11, 12))


def test_dropout_of_what_is_not_finite(ns):
    """A dropped element is 0 whatever it holds; p = 1 drops all."""
    x = torch.full((8, 64), math.nan, device=DEV)
    x[4:] = math.inf
    y = ns.dropout(x, 0.5, 3, 4)
    keep = torch.tensor(O.kept(512, 0.5, 3, 4)).view(8, 64).to(DEV)
    assert bool((y[~keep] == 0).all()) and bool(torch.isnan(y[:4][keep[:4]]).all())
    assert bool(torch.isinf(y[4:][keep[4:]]).all())
    assert not ns.dropout(x, 1.0, 3, 4).any()
    r = rand(5, 8, 64)
    assert torch.equal(ns.dropout(x, 1.0, 3, 4, residual=r), r)


def test_dropout_counter_is_read_by_the_kernel(ns):
    """A captured graph whose counter moves drops other elements each time, and
    its backward pass the same ones."""
    x = rand(6, 64, 256)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    ns.dropout(x, 0.3, 9, 100, counter=step)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ns.dropout(x, 0.3, 9, 100, counter=step)
        dx = ns.dropout_backward(x, 0.3, 9, 100, counter=step)
        step += 1
    seen = []
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ns.dropout(x, 0.3, 9, 100 + i)) and torch.equal(dx, y)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    # offsets add up modulo 2^64
    step.fill_(-1)
    assert torch.equal(ns.dropout(x, 0.3, 9, 0, counter=step), ns.dropout(x, 0.3, 9, 2 ** 64 - 1))


def test_dropout_share_and_mean(ns):
    """Of 2^24 elements the kept share is p's to six deviations, in every place
    of a block and across blocks."""
    n, p = 1 << 24, 0.1
    y = ns.dropout(torch.ones(4096, 4096, device=DEV), p, 77, 88)
    keep = (y != 0).view(-1, 8)
    limit = math.floor(p * 65536 + 0.5)
    q = 1 - limit / 65536
    dev = math.sqrt(q * (1 - q) / (n / 8))
    assert ((keep.double().mean(0) - q).abs() < 6 * dev).all()
    assert abs(keep.double().mean().item() - q) < 6 * dev / math.sqrt(8)
    assert abs((keep[1:] & keep[:-1]).double().mean().item() - q * q) < 6 * math.sqrt(q * q * 2 / n)
    assert (y[y != 0] == torch.tensor(65536 / (65536 - limit), dtype=F32)).all()


def test_dropout_past_32_bits(ns):
    """The last rows of more than 2^32 elements get the numbers of their place."""
    rows, cols = (1 << 22) + 5, 1040
    x = torch.ones(rows, cols, dtype=BF, device=DEV)
    y = ns.dropout(x, 0.5, 21, 22, out=x)
    for r in (0, 4130000, rows - 1):
        first = r * cols // 8
        keep = []
        for b in range(first, first + cols // 8):
            for w in O.philox((b & 0xFFFFFFFF, b >> 32, 22, 0), (21, 0)):
                keep += [(w & 0xFFFF) >= 32768, (w >> 16) >= 32768]
        assert torch.equal(y[r].cpu() != 0, torch.tensor(keep))
    del x, y
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ rotary

def positions_of(batch, seq, positions, offset):
    at = torch.arange(seq, device=DEV)[None] if positions is None else positions.long().view(-1, seq)
    return at.expand(batch, seq) + offset


def check_rotary(ns, x, got, plan_args, layout, positions, offset, inverse, what):
    batched = x if x.dim() == 4 else x[None]
    freq, scale = O.frequencies(**plan_args)
    want, bound = O.rotary(batched, positions_of(batched.shape[0], batched.shape[1], positions, offset),
                           plan_args["dim"], freq, scale, layout, inverse)
    near(got if x.dim() == 4 else got[None], want, bound, what)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("batch,seq,heads,kheads,head,dim", [
    (1, 1, 1, 1, 2, 2), (1, 3, 32, 4, 128, 128), (2, 37, 3, 1, 192, 64), (3, 5, 2, 2, 100, 74),
    (1, 130, 1, 7, 64, 64), (2, 9, 16, 16, 66, 66), (1, 1, 128, 1, 512, 512), (1, 700, 2, 1, 96, 32),
    (5, 1, 5, 3, 130, 6), (1, 7, 3, 2, 131, 6), (2, 11, 2, 1, 17, 16), (1, 9, 4, 2, 40, 24)])
def test_rotary(ns, batch, seq, heads, kheads, head, dim, layout, dtype):
    q, k = rand(10, batch, seq, heads, head, dtype=dtype), rand(11, batch, seq, kheads, head, dtype=dtype)
    plan = ns.RotaryPlan(dim, layout=layout)
    args = dict(dim=dim)
    for inverse, turn in ((False, ns.rotary), (True, ns.rotary_backward)):
        yq, yk = turn(q, k, plan)
        check_rotary(ns, q, yq, args, layout, None, 0, inverse, "q")
        check_rotary(ns, k, yk, args, layout, None, 0, inverse, "k")
    one, none = ns.rotary(q, None, plan, offset=77)
    assert none is None
    check_rotary(ns, q, one, args, layout, None, 77, False, "q alone")
    a, b = q.clone(), k.clone()
    ya, yb = ns.rotary(a, b, plan, offset=77, out_q=a, out_k=b)
    assert ya is a and torch.equal(a, one)
    if batch == 1:
        assert torch.equal(ns.rotary(q[0], k[0], plan, offset=77)[1], yb[0])


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 32.0),
                                            ("yarn", 1.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_far_positions(ns, layout, scaling, factor):
    """Positions up to 2^31 and below zero, in both widths."""
    args = dict(dim=64, base=500000.0, scaling=scaling, factor=factor, original=8192)
    plan = ns.RotaryPlan(layout=layout, **args)
    q, k = rand(12, 2, 50, 4, 64), rand(13, 2, 50, 2, 64, dtype=F32)
    g = torch.Generator().manual_seed(14)
    far = torch.randint(0, 1 << 31, (2, 50), generator=g)
    far[0, :5] = torch.tensor([0, 1, (1 << 31) - 1, -1, -(1 << 31)])
    for positions in (far.to(DEV), far.to(torch.int32).to(DEV), far[1].to(DEV), far[:1].to(torch.int32).to(DEV)):
        yq, yk = ns.rotary(q, k, plan, positions=positions)
        check_rotary(ns, q, yq, args, layout, positions, 0, False, "q")
        check_rotary(ns, k, yk, args, layout, positions, 0, False, "k")
    # what is added to a position is added in 64 bits
    moved = ns.rotary(q, k, plan, positions=far.to(torch.int32).to(DEV), offset=1 << 20)[0]
    check_rotary(ns, q, moved, args, layout, far.to(DEV), 1 << 20, False, "offset")


def test_rotary_frequencies(ns):
    for args in (dict(dim=128), dict(dim=2), dict(dim=64, scaling="linear", factor=3.0),
                 dict(dim=96, scaling="ntk", factor=16.0, base=1e6),
                 dict(dim=128, scaling="yarn", factor=40.0, original=4096, fast=16.0, slow=2.0)):
        plan = ns.RotaryPlan(**args)
        freq, scale = O.frequencies(**args)
        assert abs(plan.scale - scale) <= U32 * scale
        for a, b in zip(plan.frequencies, freq):
            assert abs(a - b) <= 2.0 ** -50 * b + 2 * math.pi * 2.0 ** -64


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_of_views(ns, layout, dtype):
    """Transposed batches, the last values of longer heads, odd addresses, one
    head for all, in place and not: the same bits as dense tensors, nothing
    outside the views."""
    plan = ns.RotaryPlan(32, layout=layout)
    x, k = rand(15, 2, 21, 6, 32, dtype=dtype), rand(16, 2, 21, 1, 32, dtype=dtype)
    wq, wk = ns.rotary(x, k, plan, offset=3)
    # batch x heads x seq x head
    t = x.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty(2, 6, 21, 32, dtype=dtype, device=DEV).transpose(1, 2)
    assert torch.equal(ns.rotary(t, k, plan, offset=3, out_q=out)[0], wq) and torch.equal(out, wq)
    # the last 32 of 96, in place
    for lead in (0, 1, 2):
        buf = torch.full((2 * 21 * 6 * 96 + 8,), 5.0, dtype=dtype, device=DEV)
        long = buf[lead:lead + 2 * 21 * 6 * 96].view(2, 21, 6, 96)
        part = long[..., 64:]
        part.copy_(x)
        ns.rotary(part, k, plan, offset=3, out_q=part)
        assert torch.equal(part, wq)
        part.fill_(5.0)
        assert bool((buf == 5.0).all())
    # the keys' values beside others in a wider row
    row = torch.full((2, 21, 71), 5.0, dtype=dtype, device=DEV)
    kv = row[..., 39:].unflatten(-1, (1, 32))
    kv.copy_(k)
    assert torch.equal(ns.rotary(x, kv, plan, offset=3, out_k=kv)[1], wk)
    assert bool((row[..., :39] == 5.0).all())
    same = k.expand(2, 21, 4, 32)
    assert torch.equal(ns.rotary(same, None, plan, offset=3)[0], wk.expand(2, 21, 4, 32))


def test_rotary_gradient_is_that_of_the_rotation(ns):
    """<dy, R x> = <R^T dy, x>, and turning back gives x where the scale is 1."""
    for layout in ("half", "interleaved"):
        plan = ns.RotaryPlan(64, layout=layout, scaling="yarn", factor=16.0)
        x, dy = rand(17, 40, 3, 80), rand(18, 40, 3, 80)
        y, dx = ns.rotary(x, None, plan)[0], ns.rotary_backward(dy, None, plan)[0]
        a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
        # each of the 9600 terms is off by at most 2^-20 of its size
        assert abs((a - b).item()) <= 2.0 ** -20 * 2 * (dy.double().abs() * y.double().abs()).sum().item() + 1e-3
        plain = ns.RotaryPlan(64, layout=layout)
        there = ns.rotary(x, None, plain, offset=123456)[0]
        back = ns.rotary_backward(there, None, plain, offset=123456)[0]
        assert (back - x).abs().max().item() <= 2.0 ** -18 * x.abs().max().item()


def test_rotary_of_nothing(ns):
    plan = ns.RotaryPlan(16)
    for shape in ((0, 3, 16), (2, 0, 3, 16), (5, 0, 16)):
        q = torch.empty(shape, device=DEV)
        y, k = ns.rotary(q, q, plan)
        assert y.shape == shape and k.shape == shape


# ------------------------------------------------------- gated feed-forward

def weights(seed, hidden, inner, experts=0):
    lead = (experts,) if experts else ()
    return (rand(seed, *lead, inner, hidden, scale=hidden ** -0.5, dtype=BF),
            rand(seed + 1, *lead, inner, hidden, scale=hidden ** -0.5, dtype=BF),
            rand(seed + 2, *lead, hidden, inner, scale=inner ** -0.5, dtype=BF))


def bounds_of(counts, device=DEV):
    return torch.tensor([0, *counts]).cumsum(0).to(torch.int32).to(device)


def check_forward(x, w, y, saved, offsets=None, name="silu"):
    (y64, g64, u64), (by, bg, bu) = O.ffn(x, *w, offsets, name)
    live = ~torch.isnan(y64[:, 0])
    for got, want, bound, what in ((y, y64, by, "y"), (saved[0], g64, bg, "g"), (saved[1], u64, bu, "u")):
        near(got[live], want[live], bound[live], what)
        close_norm(got[live], want[live], what)


def check_backward(dy, x, saved, w, got, offsets=None, name="silu", before=None):
    dtype = next(g.dtype for g in got[1:] if g is not None)
    want, bounds = O.ffn_grad(dy, x, *saved, *w, offsets, name, dtype, before)
    live = ~torch.isnan(want[0][:, 0])
    near(got[0][live], want[0][live], bounds[0][live], "dx")
    close_norm(got[0][live], want[0][live], "dx")
    for i, what in ((1, "dw_gate"), (2, "dw_up"), (3, "dw_down")):
        if got[i] is not None:
            near(got[i], want[i], bounds[i], what)
            close_norm(got[i], want[i], what)


DENSE = [(1, 8, 8), (1, 64, 32), (5, 2048, 768), (2, 72, 136), (31, 100, 33), (33, 33, 100), (64, 256, 128),
         (127, 264, 520), (257, 128, 256), (300, 1, 1), (1000, 520, 264), (513, 1000, 7), (700, 2056, 1032)]


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,hidden,inner", DENSE)
def test_gated_ffn(ns, tokens, hidden, inner, name):
    x, w = rand(20, tokens, hidden, dtype=BF), weights(21, hidden, inner)
    y, saved = ns.gated_ffn(x, *w, activation=name)
    check_forward(x, w, y, saved, None, name)
    again, none = ns.gated_ffn(x, *w, activation=name, keep=False)
    assert none is None and torch.equal(again, y)
    dy = rand(24, tokens, hidden, scale=0.1, dtype=BF)
    got = ns.gated_ffn_backward(dy, x, saved, *w, activation=name)
    check_backward(dy, x, saved, w, got, None, name)
    ns.ops_sync()


@pytest.mark.parametrize("tokens,hidden,inner,dtype", [(3, 4096, 520, BF), (40, 7168, 256, BF), (1, 520, 4100, BF),
                                                       (70, 2049, 2050, BF), (3000, 264, 136, BF),
                                                       (4100, 264, 136, BF), (4100, 100, 72, F32),
                                                       (4500, 513, 31, F32)])
def test_gated_ffn_of_few_tiles(ns, tokens, hidden, inner, dtype):
    """Long sums of few outputs, which are cut into parts and joined."""
    x, w = rand(25, tokens, hidden, dtype=BF), weights(26, hidden, inner)
    y, saved = ns.gated_ffn(x, *w)
    check_forward(x, w, y, saved)
    dy = rand(29, tokens, hidden, scale=0.1, dtype=BF)
    got = ns.gated_ffn_backward(dy, x, saved, *w, dtype=dtype)
    check_backward(dy, x, saved, w, got)
    base = [rand(30 + i, *v.shape, dtype=dtype) for i, v in enumerate(w)]
    more = ns.gated_ffn_backward(dy, x, saved, *w, grads=[b.clone() for b in base], accumulate=True)
    check_backward(dy, x, saved, w, more, before=base)
    again = ns.gated_ffn_backward(dy, x, saved, *w, dtype=dtype)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    ns.ops_sync()


@pytest.mark.parametrize("counts", [[5], [0], [0, 0, 0], [1, 0, 2, 63, 64, 65, 0, 200, 1], [300, 0, 0, 0],
                                    [0, 0, 17], [128, 128, 128], [7] * 40, [600, 3], [31, 33, 255, 257]])
@pytest.mark.parametrize("hidden,inner,dtype", [(64, 96, BF), (264, 520, F32), (100, 33, BF)])
def test_gated_ffn_of_experts(ns, counts, hidden, inner, dtype):
    t = sum(counts)
    offsets = bounds_of(counts)
    x, w = rand(30, t, hidden, dtype=BF), weights(31, hidden, inner, len(counts))
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    check_forward(x, w, y, saved, offsets)
    dy = rand(34, t, hidden, scale=0.1, dtype=BF)
    got = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets, dtype=dtype)
    check_backward(dy, x, saved, w, got, offsets)
    for e, c in enumerate(counts):
        if c == 0:
            assert not any(g[e].any() for g in got[1:])
    # added to what is there
    base = [rand(35 + i, *v.shape, dtype=dtype) for i, v in enumerate(w)]
    into = [b.clone() for b in base]
    more = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets, grads=into, accumulate=True)
    assert all(a is b for a, b in zip(more[1:], into))
    assert torch.equal(more[0], got[0])
    check_backward(dy, x, saved, w, more, offsets, before=base)
    ns.ops_sync()


def test_gated_ffn_rows_of_no_expert_stay(ns):
    """Rows before the first and behind the last expert are not written."""
    x, w = rand(40, 100, 64, dtype=BF), weights(41, 64, 40, 3)
    offsets = torch.tensor([10, 40, 40, 77], dtype=torch.int32, device=DEV)
    out = torch.full((100, 64), 3.0, dtype=BF, device=DEV)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets, out=out)
    assert bool((y[:10] == 3).all()) and bool((y[77:] == 3).all())
    check_forward(x, w, y, saved, offsets)
    dy = rand(44, 100, 64, dtype=BF)
    dx = torch.full((100, 64), 3.0, dtype=BF, device=DEV)
    # what the rows of no expert hold is read nowhere
    for v in (x, dy, *saved):
        v[:10] = math.nan
        v[77:] = math.nan
    got = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets, out=dx)
    assert bool((dx[:10] == 3).all()) and bool((dx[77:] == 3).all())
    check_backward(dy, x, saved, w, got, offsets)


@pytest.mark.parametrize("bad", [1, 3])
def test_gated_ffn_experts_do_not_see_each_other(ns, bad):
    """An expert whose rows and matrices hold NaN and infinities leaves the
    others as they are, whatever tile or step their rows share."""
    counts = [30, 3, 61, 2, 100]
    offsets = bounds_of(counts)
    t, hidden, inner = sum(counts), 100, 72
    x, w, dy = rand(50, t, hidden, dtype=BF), weights(51, hidden, inner, 5), rand(54, t, hidden, dtype=BF)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    clean = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets)
    a, b = offsets[bad].item(), offsets[bad + 1].item()
    x2, dy2, w2 = x.clone(), dy.clone(), [v.clone() for v in w]
    x2[a:b], dy2[a:b] = math.nan, math.inf
    for v in w2:
        v[bad] = math.nan
    y2, saved2 = ns.gated_ffn(x2, *w2, offsets=offsets)
    got = ns.gated_ffn_backward(dy2, x2, saved2, *w2, offsets=offsets)
    mine = torch.zeros(t, dtype=torch.bool, device=DEV)
    mine[a:b] = True
    for one, two in ((y2, y), (saved2[0], saved[0]), (got[0], clean[0])):
        assert torch.equal(one[~mine], two[~mine]) and bool(torch.isnan(one[mine]).all())
    for one, two in zip(got[1:], clean[1:]):
        for e in range(5):
            assert bool(torch.isnan(one[e]).all()) if e == bad else torch.equal(one[e], two[e])


def test_gated_ffn_offsets_out_of_order_are_limited(ns):
    x, w = rand(60, 50, 64, dtype=BF), weights(61, 64, 40, 4)
    offsets = torch.tensor([-5, 20, 10, 30, 2000000000], dtype=torch.int32, device=DEV)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    check_forward(x, w, y, saved, offsets)
    dy = rand(64, 50, 64, dtype=BF)
    check_backward(dy, x, saved, w, ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets), offsets)


def test_gated_ffn_many_experts(ns):
    """As many experts as a router may have, most without rows."""
    g = torch.Generator().manual_seed(70)
    counts = torch.randint(0, 4, (1024,), generator=g).tolist()
    offsets = bounds_of(counts)
    x, w = rand(71, sum(counts), 64, dtype=BF), weights(72, 64, 32, 1024)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    check_forward(x, w, y, saved, offsets)
    dy = rand(75, sum(counts), 64, dtype=BF)
    check_backward(dy, x, saved, w, ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets), offsets)


@pytest.mark.parametrize("experts", [0, 3])
def test_gated_ffn_of_views(ns, experts):
    """Rows and matrices at any address and stride give the same bits, and
    nothing is written outside the views."""
    t, hidden, inner = 150, 104, 72
    offsets = bounds_of([50, 0, 100]) if experts else None
    x, dy, w = rand(80, t, hidden, dtype=BF), rand(81, t, hidden, dtype=BF), weights(82, hidden, inner, experts)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    want = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets)

    def wide(v, lead, pad):
        if v.dim() == 2:
            return strided(v, lead, pad)
        e, r, c = v.shape
        buf = torch.full((lead + e * (r + 1) * (c + pad) + 8,), 7.0, dtype=v.dtype, device=DEV)
        out = buf[lead:lead + e * (r + 1) * (c + pad)].view(e, r + 1, c + pad)[:, :r, :c]
        out.copy_(v)
        return out

    for lead, pad in ((1, 0), (3, 5), (8, 8), (0, 1)):
        x2, dy2, w2 = wide(x, lead, pad), wide(dy, lead, pad), [wide(v, lead, pad) for v in w]
        s2 = [wide(v, lead, pad) for v in saved]
        out, dx = wide(torch.zeros_like(x), lead, pad), wide(torch.zeros_like(x), lead, pad)
        grads = [wide(torch.zeros_like(v), lead, pad) for v in w]
        before = [v._base.clone() for v in (out, dx, *grads)]
        got, _ = ns.gated_ffn(x2, *w2, offsets=offsets, out=out)
        assert torch.equal(got, y)
        got = ns.gated_ffn_backward(dy2, x2, s2, *w2, offsets=offsets, out=dx, grads=grads)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for v, b in zip((out, dx, *grads), before):
            v.zero_()
            assert torch.equal(v._base, b)
    # rows and matrices that are one for all
    row = ns.gated_ffn(x[:1].expand(t, -1), *w, offsets=offsets, keep=False)[0]
    assert torch.equal(row, ns.gated_ffn(x[:1].expand(t, -1).contiguous(), *w, offsets=offsets, keep=False)[0])
    if experts:
        same = [v[:1].expand(3, -1, -1) for v in w]
        full = [v.contiguous() for v in same]
        a, sa = ns.gated_ffn(x, *same, offsets=offsets)
        b, sb = ns.gated_ffn(x, *full, offsets=offsets)
        assert torch.equal(a, b)
        for one, two in zip(ns.gated_ffn_backward(dy, x, sa, *same, offsets=offsets),
                            ns.gated_ffn_backward(dy, x, sb, *full, offsets=offsets)):
            assert torch.equal(one, two)


def test_gated_ffn_of_no_rows(ns):
    w = weights(90, 64, 40)
    x = torch.empty(0, 64, dtype=BF, device=DEV)
    y, saved = ns.gated_ffn(x, *w)
    assert y.shape == (0, 64) and saved[0].shape == (0, 40)
    base = [torch.ones_like(v) for v in w]
    got = ns.gated_ffn_backward(x, x, saved, *w, grads=[b.clone() for b in base])
    assert not any(g.any() for g in got[1:])
    got = ns.gated_ffn_backward(x, x, saved, *w, grads=[b.clone() for b in base], accumulate=True)
    assert all(torch.equal(g, b) for g, b in zip(got[1:], base))


@pytest.mark.parametrize("inner", [72, 45])
@pytest.mark.parametrize("counts", [None, [40, 0, 1, 159]])
def test_gated_ffn_from_a_checkpoint(ns, counts, inner):
    """x kept in 8 bits, with a norm's weight and bias: the gradients of w_gate
    and w_up are those of what the checkpoint stands for."""
    t, hidden = 200, 136
    offsets = None if counts is None else bounds_of(counts)
    w = weights(91, hidden, inner, 0 if counts is None else 4)
    h, dy = ns.checkpoint8(rand(94, t, hidden)), rand(95, t, hidden, scale=0.1, dtype=BF)
    gain, shift = rand(96, hidden), rand(97, hidden)
    x64 = h.values(F32).to(D) * gain.to(D) + shift.to(D)
    _, saved = ns.gated_ffn(x64.to(BF), *w, offsets=offsets)
    for dtype in (BF, F32):
        got = ns.gated_ffn_backward(dy, h, saved, *w, offsets=offsets, weight=gain, bias=shift, dtype=dtype)
        want, bounds = O.ffn_grad(dy, x64, *saved, *w, offsets, "silu", dtype)
        # the weight and the bias act on sums: their terms' sizes add up
        for i in (1, 2):
            close_norm(got[i], want[i], i)
        near(got[0], want[0], bounds[0], "dx")
        near(got[3], want[3], bounds[3], "dw_down")
        into = [g.clone() for g in got[1:]]
        twice = ns.gated_ffn_backward(dy, h, saved, *w, offsets=offsets, weight=gain, bias=shift, grads=into,
                                      accumulate=True)
        for a, b in zip(twice[1:], got[1:]):
            close_norm(a, 2 * b.to(D), "added")
    none = ns.gated_ffn_backward(dy, None, saved, *w, offsets=offsets, dtype=F32)
    assert none[1] is None and none[2] is None and torch.equal(none[3], got[3]) and torch.equal(none[0], got[0])


def test_gated_ffn_some_gradients_and_in_place(ns):
    """Any of the weights' gradients alone, what is made on the way in tensors
    of the caller's (through the C entry), and y in x's place."""
    import ctypes

    from newton_schulz_06_gb300 import _lib
    t, hidden, inner = 150, 104, 45
    x, w, dy = rand(120, t, hidden, dtype=BF), weights(121, hidden, inner), rand(124, t, hidden, dtype=BF)
    y, saved = ns.gated_ffn(x, *w)
    want = ns.gated_ffn_backward(dy, x, saved, *w)
    for i in range(3):
        grads = [None, None, None]
        grads[i] = torch.empty_like(w[i])
        got = ns.gated_ffn_backward(dy, x, saved, *w, grads=grads)
        assert torch.equal(got[0], want[0])
        assert all((g is None) if j != i else torch.equal(g, want[j + 1]) for j, g in enumerate(got[1:]))
    made = [torch.empty(t, inner, dtype=BF, device=DEV) for _ in range(3)]
    a = _lib.GatedFfnGradArgs(dy=dy.data_ptr(), gate=saved[0].data_ptr(), up=saved[1].data_ptr(),
                              w_down=w[2].data_ptr(), dgate=made[0].data_ptr(), dup=made[1].data_ptr(),
                              h=made[2].data_ptr(), rows=t, hidden=hidden, inner=inner, experts=1, ld_dy=hidden,
                              ld_kept=inner, ld_down=inner, ld_d=inner)
    size = ctypes.c_size_t()
    L = _lib.lib()
    assert L.muon_gated_ffn_grad_workspace(ctypes.byref(a), ctypes.byref(size)) == 0
    ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device=DEV)
    assert L.muon_gated_ffn_grad(ctypes.byref(a), ws.data_ptr(), size.value,
                                 torch.cuda.current_stream().cuda_stream, None, 0) == 0
    f, df, _ = O.act("silu", saved[0].to(D))
    dh = dy.to(D) @ w[2].to(D)
    for got, exact in zip(made, (dh * saved[1].to(D) * df, dh * f, f * saved[1].to(D))):
        close_norm(got, exact, "made")
    z = x.clone()
    assert ns.gated_ffn(z, *w, out=z)[0] is z and torch.equal(z, y)


def test_gated_ffn_past_32_bits(ns):
    """Rows whose kept values lie past 2^31 elements."""
    rows, hidden, inner, n = 270000, 64, 8192, 40
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of device memory")
    x, w = torch.zeros(rows, hidden, dtype=BF, device=DEV), weights(130, hidden, inner)
    x[-n:] = rand(133, n, hidden, dtype=BF)
    y, saved = ns.gated_ffn(x, *w)
    assert not y[:-n].any() and not saved[0][:-n].any()
    tail = [v[-n:].clone() for v in saved]
    check_forward(x[-n:], w, y[-n:], tail)
    dy = torch.zeros_like(x)
    dy[-n:] = rand(134, n, hidden, scale=0.1, dtype=BF)
    got = ns.gated_ffn_backward(dy, x, saved, *w)
    assert not got[0][:-n].any()
    want, bounds = O.ffn_grad(dy[-n:], x[-n:], *tail, *w)
    for i, what in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        near(got[i][-n:] if i == 0 else got[i], want[i], bounds[i], what)
    del saved, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_ffn_gradient_is_that_of_differences(ns, name):
    """Along a direction, the 64-bit form's difference quotient is the inner
    product with the kernel's gradients."""
    t, hidden, inner = 64, 48, 40
    x, w = rand(100, t, hidden, dtype=BF), weights(101, hidden, inner)
    dy = rand(104, t, hidden, dtype=BF)
    g64, u64 = x.to(D) @ w[0].to(D).t(), x.to(D) @ w[1].to(D).t()
    got = ns.gated_ffn_backward(dy, x, (g64.to(BF), u64.to(BF)), *w, activation=name, dtype=F32)
    args = [v.to(D) for v in (x, *w)]
    for i in range(4):
        way = rand(105 + i, *args[i].shape).to(D)

        def value(step):
            a = list(args)
            a[i] = a[i] + step * way
            h = O.act(name, a[0] @ a[1].t())[0] * (a[0] @ a[2].t())
            return ((h @ a[3].t()) * dy.to(D)).sum()

        want = ((value(1e-5) - value(-1e-5)) / 2e-5).item()
        have = (got[i].to(D) * way).sum().item()
        # a norm-wise error of 1e-2 in the gradient, against a random direction
        assert abs(have - want) <= 1e-2 * got[i].to(D).norm().item() * 6, (i, have, want)


def test_gated_ffn_saturates(ns):
    """Gates far on both sides: act(g) is g or 0 and its derivative 1 or 0."""
    hidden, inner = 64, 32
    x = torch.zeros(4, hidden, dtype=BF, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = 1e4, -1e4, 1e30
    w = [torch.zeros(inner, hidden, dtype=BF, device=DEV) for _ in range(2)]
    w[0][:, 0], w[1][:, 0] = 1.0, 1e-3
    wd = torch.eye(hidden, inner, dtype=BF, device=DEV)
    for name in ("silu", "gelu", "gelu_tanh"):
        y, saved = ns.gated_ffn(x, *w, wd, activation=name)
        (y64, _, _), (by, _, _) = O.ffn(x, *w, wd, None, name)
        near(y, y64, by, name)
        got = ns.gated_ffn_backward(x, x, saved, *w, wd, activation=name)
        assert all(bool(torch.isfinite(g.float()[:2]).all()) for g in got[:1])


def test_run_of_a_block(ns):
    """The operators as a block's step uses them, in eager order and captured:
    norm, rotary, dropout with a residual, router, experts, and back."""
    T, H, E, K, inner = 96, 64, 8, 2, 48
    plan = ns.RotaryPlan(32)
    w = weights(110, H, inner, E)
    x, dout = rand(113, T, H, dtype=BF), rand(114, T, H, scale=0.1, dtype=BF)
    router = rand(115, E, H, scale=0.1)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)

    def run():
        y, rstd, saved8 = ns.layer_norm_checkpoint(x)
        q, _ = ns.rotary(y.view(T, 2, 32), None, plan)
        a = ns.dropout(q.reshape(T, H), 0.2, 1, counter=step, residual=x)
        r = ns.route(a.float() @ router.t(), K)
        order = torch.argsort(r.indices.flatten(), stable=True)
        token = order // K
        rows = a[token]
        f, kept = ns.gated_ffn(rows, *w, offsets=r.offsets)
        df = dout[token]
        drows, *dw = ns.gated_ffn_backward(df, rows, kept, *w, offsets=r.offsets)
        da = torch.zeros(T, H, device=DEV).index_add_(0, token, drows.float()).to(BF)
        dq = ns.dropout_backward(da, 0.2, 1, counter=step)
        dy = ns.rotary_backward(dq.view(T, 2, 32), None, plan)[0].reshape(T, H)
        dx, _, _ = ns.layer_norm_backward(dy, saved8, None, rstd)
        return f, dx + da, *dw

    eager = [v.clone() for v in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = run()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        second = run()
    for graph, outs in ((g, captured), (g2, second), (g, captured)):
        for v in outs:
            v.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b)
    ns.ops_sync()


def one_sign(tokens, size, seed):
    """Operands whose dgate, dup and h are exact and whose weight gradients are
    sums of one sign: silu(64) = 64 and silu'(64) = 1 in fp32, up is a power of
    two and w_down the identity."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dy, x = (torch.randn(tokens, size, generator=g, device=DEV).abs_().to(BF) for _ in range(2))
    up = (2.0 ** (torch.arange(size, device=DEV) % 3)).to(BF)
    saved = torch.full((tokens, size), 64.0, dtype=BF, device=DEV), up.expand(tokens, -1).contiguous()
    return dy, x, saved, up.to(D), torch.eye(size, dtype=BF, device=DEV)


def one_sign_grads(dy, x, up, a, b):
    of_x = torch.zeros(dy.shape[1], x.shape[1], dtype=D, device=DEV)
    of_h = torch.zeros(dy.shape[1], dtype=D, device=DEV)
    for t in range(a, b, 16384):
        part = dy[t:min(b, t + 16384)].to(D)
        of_x += part.t() @ x[t:min(b, t + 16384)].to(D)
        of_h += part.sum(0)
    return up[:, None] * of_x, 64 * of_x, 64 * of_h[:, None] * up


LONG = 200003


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("size,counts", [(1024, None), (256, None), (256, [LONG]), (264, [40, 0, LONG - 4200, 4097])])
def test_gated_ffn_long_sums(ns, size, counts, accumulate):
    """fp32 gradients: running sums of 4096 tokens at most (256 products of
    two cuts of 2^-23 at most each), added up with one rounding each.  One running
    sum loses 0.4 * 2^-23 a product on average, ten times as much."""
    dy, x, saved, up, eye = one_sign(LONG, size, 1)
    lead = () if counts is None else (len(counts),)
    w = [eye.expand(*lead, -1, -1).contiguous()] * 3
    ends = [0, LONG] if counts is None else [0, *torch.tensor(counts).cumsum(0).tolist()]
    before = rand(2, *lead, size, size).abs() * 1e6
    grads = [before.clone() for _ in range(3)]
    ns.gated_ffn_backward(dy, x, saved, *w, grads=grads, accumulate=accumulate,
                          offsets=None if counts is None else bounds_of(counts))
    bound = 256 * 2 * 2.0 ** -23 + (LONG / 4096 + 30) * U32
    assert bound < 0.12 * 0.4 * 2.0 ** -23 * LONG / 16
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        for got, want, name in zip(grads, one_sign_grads(dy, x, up, a, b), ("gate", "up", "down")):
            old = before.view(-1, size, size)[e].to(D) * accumulate
            got = got.view(-1, size, size)[e]
            near(got, want + old, bound * want + U32 * (want + old), f"dw_{name} of {e}")


@pytest.mark.parametrize("size,counts", [(1024, None), (256, [LONG]), (264, [40, 0, LONG - 4200, 4160])])
def test_gated_ffn_long_sums_of_bf16(ns, size, counts):
    """What a sum has lost shows in the mean difference of many results from
    the exact values' roundings.  8192 tokens (512 products of two cuts of a
    place each at most, 2^-23 of a sum that is on average 0.375 of its end's place)
    lose 4.6e-5 at most, one running sum over all of them more than ten times that.
    The difference is 0 or a step, 2^-7 of a value at most, at the few values that the
    loss carries over a rounding's border: a share of 2^-7 or so of them, the
    deviation of one's relative difference is 7e-4 and of the mean of 65536 values
    3e-6; up to five of those count."""
    dy, x, saved, up, eye = one_sign(LONG, size, 3)
    lead = () if counts is None else (len(counts),)
    w = [eye.expand(*lead, -1, -1).contiguous()] * 3
    ends = [0, LONG] if counts is None else [0, *torch.tensor(counts).cumsum(0).tolist()]
    _, *grads = ns.gated_ffn_backward(dy, x, saved, *w, offsets=None if counts is None else bounds_of(counts))
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        for got, want, name in zip(grads[:2], one_sign_grads(dy, x, up, a, b), ("gate", "up")):
            got = got.view(-1, size, size)[e].to(D)
            near(got, want, (HALF[BF] + 512 * 2 * 2.0 ** -23) * want, f"dw_{name} of {e}")
            if b > a:
                off = ((got - want.to(BF).to(D)) / want).mean().item()
                assert abs(off) <= 4.9e-5 + 1.5e-5, (name, e, off)


def test_two_calls_at_once(ns):
    """Calls on two streams and from two threads have workspaces of their own."""
    import threading
    w = weights(150, 256, 512)
    we, offsets = weights(153, 256, 96, 5), bounds_of([100, 0, 300, 7, 93])
    x, dy = rand(156, 500, 256, dtype=BF), rand(157, 500, 256, dtype=BF)

    def dense():
        y, s = ns.gated_ffn(x, *w)
        return y, *ns.gated_ffn_backward(dy, x, s, *w)

    def experts():
        y, s = ns.gated_ffn(x, *we, offsets=offsets)
        return y, *ns.gated_ffn_backward(dy, x, s, *we, offsets=offsets)

    want = dense(), experts()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(20):
                got[i].append((dense, experts)[i]())

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 20
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
    ns.ops_sync()


def test_example_block(ns):
    """The example's block: its gradients are those of the same block with
    autograd in 64 bits, within what bf16 and 8-bit activations cost."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_gated_block.py")
    spec = importlib.util.spec_from_file_location("train_gated_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    T, H = 96, 64
    block = ex.Block(hidden=H, heads=4, kv_heads=2, head=16, inner=48, experts=8, k=2, p=0.2)
    x, dout = rand(140, T, H, dtype=BF), rand(141, T, H, dtype=BF)
    out = block.forward(x, step=3)
    dx = block.backward(dout)
    names = ("wq", "wk", "wv", "wo", "router", "w_gate", "w_up", "w_down", "gain1", "shift1", "gain2", "shift2")
    leaf = {n: getattr(block, n).to("cpu", D).requires_grad_() for n in names}
    xr = x.to("cpu", D).requires_grad_()
    kept = block.kept
    freq, _ = O.frequencies(16)
    angle = torch.arange(T, dtype=D)[:, None] * torch.tensor(freq, dtype=D)

    def turn(v):
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        a, b = v[..., :8], v[..., 8:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def drop(v, offset):
        keep = torch.tensor(O.kept(T * H, 0.2, block.seed, offset)).view(T, H)
        return v * keep * (65536 / (65536 - math.floor(0.2 * 65536 + 0.5)))

    norm = torch.nn.functional.layer_norm
    y1 = norm(xr, (H,), leaf["gain1"], leaf["shift1"])
    q, k, v = (y1 @ leaf[n].t() for n in ("wq", "wk", "wv"))
    q, k, v = turn(q.view(T, 4, 16)), turn(k.view(T, 2, 16)), v.view(T, 2, 16)
    k, v = k.repeat_interleave(2, 1), v.repeat_interleave(2, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) / 4
    s = s.masked_fill(torch.ones(T, T).triu(1).bool(), -math.inf)
    a = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v).reshape(T, -1)
    x1 = xr + drop(a @ leaf["wo"].t(), 6)
    y2 = norm(x1, (H,), leaf["gain2"], leaf["shift2"])
    p = torch.softmax(y2 @ leaf["router"].t(), -1)
    idx = kept["routing"].indices.cpu().long()
    w = p.gather(1, idx)
    w = w / w.sum(-1, keepdim=True)
    g = torch.einsum("tkih,th->tki", leaf["w_gate"][idx], y2)
    u = torch.einsum("tkih,th->tki", leaf["w_up"][idx], y2)
    f = torch.einsum("tkhi,tki->tkh", leaf["w_down"][idx], torch.nn.functional.silu(g) * u)
    ref = x1 + drop((w[..., None] * f).sum(1), 7)
    counts = torch.bincount(idx.flatten(), minlength=8).to(D)
    balance = 0.01 * 8 / (2 * T) * (counts * p.mean(0)).sum()
    ((ref * dout.to("cpu", D)).sum() + balance).backward()
    got = {n: block.grads[n] for n in names}
    # a value has passed about ten roundings to bf16 and one to 8 bits on its
    # way: a few percent of the norm
    for name, have, want in (("out", out, ref.detach()), ("dx", dx, xr.grad),
                             *((n, got[n], leaf[n].grad) for n in names)):
        off = (have.to("cpu", D) - want).norm() / want.norm()
        assert off <= 0.08, (name, off.item())
    block.muon.close()
    losses = ex.train(steps=3, tokens=128, hidden=64, inner=32, experts=4)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


@pytest.mark.parametrize("hidden,inner", [(264, 96), (40, 200)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_ffn_every_last_step(ns, hidden, inner, dtype):
    """Experts of 1 to 64 tokens and of 65 to 128, each beside one of a single
    token whose rows are NaN: whatever a last step of 64 holds of them, their
    gradients are those of their own tokens."""
    counts = []
    for n in range(1, 65):
        counts += [n, 1, n + 64, 1]
    offsets = bounds_of(counts)
    t, experts = sum(counts), len(counts)
    x, dy = rand(160, t, hidden, dtype=BF), rand(161, t, hidden, scale=0.1, dtype=BF)
    w = [v[:1].expand(experts, -1, -1) for v in weights(162, hidden, inner, 1)]
    _, saved = ns.gated_ffn(x, *w, offsets=offsets)
    for e in range(1, experts, 2):
        at = int(offsets[e])
        x[at], dy[at] = math.nan, math.nan
    got = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets, dtype=dtype)
    for e in range(0, experts, 2):
        a, b = int(offsets[e]), int(offsets[e + 1])
        s = [v[a:b] for v in saved]
        want, bounds = O.ffn_grad(dy[a:b], x[a:b], *s, *[v[0] for v in w], None, "silu", dtype)
        for i, what in ((1, "dw_gate"), (2, "dw_up"), (3, "dw_down")):
            near(got[i][e], want[i], bounds[i], f"{what} of {b - a}")
            assert bool(torch.isnan(got[i][e + 1]).any())


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_ffn_small_activations_keep_their_digits(ns, name):
    """Gates of -9 to -3, where act(g) falls to 1e-18 and less: h, dup and y are
    off by a rounding of their own size, not of the gate's.

    Relative errors of act(g), in units of 2^-23.  gelu: exp(-g^2 / 2), whose
    argument is off by half a unit of itself, g^2 / 4, and which is itself off by 2 +
    1.2 g^2 / 2; what it is multiplied by: the fit 1, the reciprocal 2, the sum and
    the products 5.  The logistic function of z, for the others: the argument's
    roundings 2 |z|, the exponential 2 + 1.2 |z|, the sum, the quotient and the
    products 5."""
    gates = -torch.linspace(3, 9, 256).to(BF)
    n = gates.numel()
    g64 = gates.to(D)
    z = g64 if name == "silu" else 2 * math.sqrt(2 / math.pi) * (g64 + 0.044715 * g64 ** 3)
    off = (0.85 * g64 * g64 + 10 if name == "gelu" else 3.2 * z.abs() + 7) * 2.0 ** -23
    # (ndtr, even in 64 bits, is 0 below -8.3)
    f64 = g64 / 2 * torch.special.erfc(-g64 / math.sqrt(2)) if name == "gelu" else O.act(name, g64)[0]
    assert bool((f64.abs() > 1e-30).all())
    bound = ((HALF[BF] + 1.01 * off) * f64.abs())[:, None].to(DEV)
    want = f64[:, None].to(DEV)
    # forward: rows whose gates are one of these, and whose u is 1
    hidden = inner = 64
    x = torch.zeros(n, hidden, dtype=BF, device=DEV)
    x[:, 0], x[:, 1] = gates.to(DEV), 1.0
    wg, wu = (torch.zeros(inner, hidden, dtype=BF, device=DEV) for _ in range(2))
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    eye = torch.eye(hidden, dtype=BF, device=DEV)
    y, saved = ns.gated_ffn(x, wg, wu, eye, activation=name)
    assert torch.equal(saved[0], x[:, :1].expand(-1, inner)) and bool((saved[1] == 1).all())
    near(y, want.expand(n, hidden), bound.expand(n, hidden), "y")
    # backward, with dh = 1: dw_up = dup^T x and dw_down = dy^T h of one row each
    one = torch.ones(1, hidden, dtype=BF, device=DEV)
    wide = torch.ones(hidden, n, dtype=BF, device=DEV)
    wide[1:] = 0
    row = gates.to(DEV)[None]
    dx, _, dup, ddown = ns.gated_ffn_backward(one, one, (row, torch.ones_like(row)), *[wide.t().contiguous()] * 2,
                                              wide, activation=name, dtype=F32)
    near(dup, want.expand(n, hidden), bound.expand(n, hidden), "dw_up")
    near(ddown, want.t().expand(hidden, n), bound.t().expand(hidden, n), "dw_down")


def test_rotary_offset_of_64_bits(ns):
    """Position and offset add up modulo 2^64, and an offset past 64 bits is
    refused."""
    plan, q = ns.RotaryPlan(32), rand(170, 3, 2, 32)
    top = torch.full((3,), 2 ** 63 - 1, dtype=torch.int64, device=DEV)
    low = torch.full((3,), -2 ** 63, dtype=torch.int64, device=DEV)
    assert torch.equal(ns.rotary(q, None, plan, positions=top, offset=1)[0], ns.rotary(q, None, plan, positions=low)[0])
    back = torch.zeros(3, dtype=torch.int64, device=DEV)
    assert torch.equal(ns.rotary(q, None, plan, positions=low, offset=-2 ** 63)[0],
                       ns.rotary(q, None, plan, positions=back)[0])
    for offset in (2 ** 63, -2 ** 63 - 1, 10 ** 30):
        with pytest.raises(ValueError, match="offset"):
            ns.rotary(q, None, plan, offset=offset)


def test_gated_ffn_long_sums_added_to_bf16(ns):
    """bf16 gradients over several chunks, added to what is there, of rows that
    do not lie on 16 bytes: 8192 tokens in one running sum at most (512 products
    of two cuts of 2^-23), the chunks' sums and the old value added up in fp32,
    one rounding to bf16."""
    size, tokens = 257, 30000
    dy, x, saved, up, eye = one_sign(tokens, size, 5)
    # (the tiles of an expert are not split into parts, whose sums end before a chunk does)
    before = [rand(180 + i, 1, size, size).abs().to(BF) * 4096 for i in range(3)]
    grads = [b.clone() for b in before]
    ns.gated_ffn_backward(dy, x, saved, *[eye[None]] * 3, grads=grads, accumulate=True, offsets=bounds_of([tokens]))
    bound = 512 * 2 * 2.0 ** -23 + 40 * U32
    for got, want, old, name in zip(grads, one_sign_grads(dy, x, up, 0, tokens), before, ("gate", "up", "down")):
        total = want + old[0].to(D)
        near(got[0], total, bound * want + 4 * U32 * total + HALF[BF] * (1 + bound) * total, f"dw_{name}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gated_ffn_chunks_inside_parts(ns, dtype):
    """Few tiles and many tokens: the sums are cut into parts (here 25), and a
    part into chunks, of 10000 tokens two of bf16 (or three of fp32) results."""
    size, tokens = 256, 250000
    dy, x, saved, up, eye = one_sign(tokens, size, 6)
    _, *grads = ns.gated_ffn_backward(dy, x, saved, eye, eye, eye, dtype=dtype)
    bound = (512 if dtype == BF else 256) * 2 * 2.0 ** -23 + 100 * U32
    for got, want, name in zip(grads, one_sign_grads(dy, x, up, 0, tokens), ("gate", "up", "down")):
        near(got, want, (bound + HALF[dtype] * (1 + bound)) * want, f"dw_{name}")


@pytest.mark.parametrize("tokens,hidden,inner", [(300, 264, 20000), (2500, 20000, 128)])
def test_gated_ffn_long_sums_between_the_products(ns, tokens, hidden, inner):
    """Sums of one sign over a wide inner (y, and dx, whose sum is twice as
    long) or a wide hidden (g, u and dhidden): each product of 16 terms may cut
    twice 2^-23 of the running sum (the oracle's sums())."""
    g = torch.Generator().manual_seed(190)
    x, dy = (torch.rand(tokens, hidden, generator=g).to(BF).to(DEV) for _ in range(2))
    w = [(torch.rand(*s, generator=g) * 2 / s[1]).to(BF).to(DEV) for s in ((inner, hidden), (inner, hidden), (hidden, inner))]
    y, saved = ns.gated_ffn(x, *w)
    check_forward(x, w, y, saved)
    check_backward(dy, x, saved, w, ns.gated_ffn_backward(dy, x, saved, *w))
    ns.ops_sync()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gated_ffn_closed_gates_stay_closed(ns, name):
    """Where act'(g) is 0, dg is 0 however large dh and u are; where it is 1, dg is
    dh u.  (dh and du come through matrices of 0 and 1.)"""
    hidden = inner = 64
    gates = torch.tensor([-200.0, -200.0, 200.0, 200.0], device=DEV).to(BF)[:, None].expand(-1, inner).contiguous()
    up = torch.tensor([1e20, -1e30, 1e10, 1e-20], device=DEV).to(BF)[:, None].expand(-1, inner).contiguous()
    dy = torch.tensor([1e20, 1e30, 1e20, 1e20], device=DEV).to(BF)[:, None].expand(-1, hidden).contiguous()
    eye = torch.eye(hidden, dtype=BF, device=DEV)
    none = torch.zeros(inner, hidden, dtype=BF, device=DEV)
    dx = ns.gated_ffn_backward(dy, None, (gates, up), eye, none, eye, activation=name)[0].to(D)
    assert not dx[:2].any()
    # dh is exact, dg and dx are rounded
    want = dy[2:].to(D) * up[2:].to(D)
    near(dx[2:], want, 2.1 * HALF[BF] * want, "dx")
