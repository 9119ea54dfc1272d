"""Outputs that share memory with what is still read, or with each other: found
from addresses and strides before any CUDA call (overlap.h), and refused."""
import ctypes
import os
import subprocess
from ctypes import byref

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
M = 1 << 20            # addresses that no refused call looks behind, far from each other
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from newton_schulz_06_gb300 import build as b
    b.build()
    from newton_schulz_06_gb300 import _lib
    return _lib


def refused(L, name, struct, base, *rest, **kw):
    a = struct()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    buf = ctypes.create_string_buffer(256)
    rc = getattr(L.lib(), name)(byref(a), *rest, None, buf, 256)
    assert rc == L.MUON_ERR_INVALID_ARG, rc
    return buf.value.decode()


def test_areas_are_told_apart_as_their_bytes_are(tmp_path):
    """No two that share memory are taken for separate, and parts of one buffer
    (columns, rows, matrices, an expert's matrices beside each other) that share
    nothing are taken for what they are."""
    exe = str(tmp_path / "overlap")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "newton_schulz_06_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "overlap.cpp"), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split() == ["0", "0", "0"]


# 4 rows of 64 values are 512 bytes, of 32 values 256; the weights 4096
FFN = dict(x=1 * M, w_gate=2 * M, w_up=3 * M, w_down=4 * M, y=5 * M, gate=6 * M, up=7 * M, rows=4, hidden=64, inner=32,
           experts=1, ld_x=64, ld_gate=64, ld_up=64, ld_down=32, ld_y=64, ld_kept=32)


@pytest.mark.parametrize("kw,names", [
    (dict(y=2 * M + 4094), "y w_gate"), (dict(y=3 * M - 510), "y w_up"), (dict(y=4 * M), "y w_down"),
    (dict(gate=2 * M), "gate w_gate"), (dict(up=4 * M + 2), "up w_down"), (dict(up=6 * M + 254), "gate up"),
    (dict(gate=1 * M + 256), "gate x"), (dict(up=5 * M + 16), "up y"), (dict(gate=5 * M - 254), "gate y"),
    # columns of one matrix that have one in common
    (dict(gate=6 * M, up=6 * M + 62, ld_kept=72), "gate up"),
    (dict(offsets=64 * M, experts=3, stride_gate=4096, stride_up=4096, stride_down=4096, y=2 * M + 2 * 8192), "y w_gate")])
def test_gated_ffn_refuses_what_shares_memory(L, kw, names):
    msg = refused(L, "muon_gated_ffn", L.GatedFfnArgs, FFN, 256 * M, 1 << 30, **kw)
    assert "share memory" in msg and all(n in msg.split() for n in names.split()), msg


GRAD = dict(dy=1 * M, x=2 * M, gate=3 * M, up=4 * M, w_gate=5 * M, w_up=6 * M, w_down=7 * M, dx=8 * M, dw_gate=9 * M,
            dw_up=10 * M, dw_down=11 * M, rows=4, hidden=64, inner=32, experts=1, ld_dy=64, ld_x=64, ld_kept=32,
            ld_gate=64, ld_up=64, ld_down=32, ld_dx=64, ld_dw_gate=64, ld_dw_up=64, ld_dw_down=32, ld_d=32, g_dtype=1)


@pytest.mark.parametrize("kw,names", [
    (dict(dx=1 * M + 128), "dx dy"), (dict(dx=1 * M - 2), "dx dy"), (dict(dx=2 * M + 510), "dx x"),
    (dict(dx=1 * M + 64, ld_dx=96, ld_dy=96), "dx dy"), (dict(dx=5 * M), "dx w_gate"), (dict(dx=6 * M + 4000), "dx w_up"),
    (dict(dw_gate=1 * M), "dw_gate dy"), (dict(dw_up=2 * M - 4000), "dw_up x"), (dict(dw_down=8 * M), "dw_down dx"),
    (dict(dw_up=9 * M + 4094), "dw_gate dw_up"), (dict(dw_down=10 * M), "dw_up dw_down"),
    (dict(dgate=1 * M), "dgate dy"), (dict(dup=3 * M + 2), "dup gate"), (dict(h=7 * M), "h w_down"),
    (dict(dgate=12 * M, dup=12 * M), "dgate dup"), (dict(dgate=8 * M), "dgate dx"), (dict(h=9 * M), "h dw_gate"),
    (dict(dgate=3 * M, ld_kept=0), "dgate gate"), (dict(dgate=2 * M), "dgate x"), (dict(dup=5 * M), "dup w_gate"),
    (dict(offsets=64 * M, experts=3, stride_gate=2048, stride_up=2048, stride_down=2048, stride_dw_gate=4096,
          stride_dw_up=4096, stride_dw_down=4096, dw_gate=9 * M, dw_up=9 * M + 4094), "dw_gate dw_up")])
def test_gated_ffn_grad_refuses_what_shares_memory(L, kw, names):
    msg = refused(L, "muon_gated_ffn_grad", L.GatedFfnGradArgs, GRAD, 256 * M, 1 << 30, **kw)
    assert "share memory" in msg and all(n in msg.split() for n in names.split()), msg


TURNS = (ctypes.c_uint64 * 8)()
# 2 batches of 3 positions of 2 heads of 16 bf16 values, dense: 384 bytes
ROTARY = dict(turns=ctypes.addressof(TURNS), batch=2, seq=3, head=16, pairs=8, x_dtype=1, scale=1.0)
HEADS = dict(heads=2, x_batch=96, x_seq=32, x_head=16, y_batch=96, y_seq=32, y_head=16)


@pytest.mark.parametrize("q,k,word", [
    (dict(y=1 * M + 32), {}, "q"), (dict(y=1 * M - 382), {}, "q"), ({}, dict(y=2 * M + 2), "k"),
    (dict(y=2 * M), {}, "q"), ({}, dict(y=1 * M + 352), "k"), (dict(y=4 * M + 382), {}, "q"),
    # the same tensor for both, in place
    (dict(y=1 * M), dict(x=1 * M, y=1 * M), "q"),
    # heads, positions and batches over one another
    (dict(y_head=15), {}, "q"), ({}, dict(y_seq=31), "k"), ({}, dict(y_batch=95), "k"), (dict(y_seq=16), {}, "q"),
    # columns of one row that have a head in common
    (dict(x_seq=64, x_batch=192, y=1 * M + 32, y_seq=64, y_batch=192), {}, "q")])
def test_rotary_refuses_what_shares_memory(L, q, k, word):
    a = {**ROTARY, "q": L.RotaryTensor(**{**HEADS, "x": 1 * M, "y": 3 * M, **q}),
         "k": L.RotaryTensor(**{**HEADS, "x": 2 * M, "y": 4 * M, **k})}
    msg = refused(L, "muon_rotary", L.RotaryArgs, a)
    assert msg.startswith(word + " is written to") and "share" in msg, msg


DROP = dict(x=1 * M, residual=2 * M, y=3 * M, rows=4, cols=64, ld_x=64, ld_r=64, ld_y=64, p=0.1, x_dtype=1)


@pytest.mark.parametrize("kw,names", [
    (dict(y=1 * M + 2), "y x"), (dict(y=1 * M - 510), "y x"), (dict(y=2 * M + 128), "y residual"),
    (dict(y=1 * M, residual=1 * M + 128), "y residual"), (dict(y=1 * M + 4, x_dtype=0), "y x"),
    (dict(y=1 * M + 100, ld_x=100, ld_y=100), "y x")])
def test_dropout_refuses_what_shares_memory(L, kw, names):
    msg = refused(L, "muon_dropout", L.DropoutArgs, DROP, **kw)
    assert "share memory" in msg and all(n in msg.split() for n in names.split()), msg


# ------------------------------------------------------------- on the GPU

@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * 0.1).to(BF).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("experts", [0, 3])
def test_gated_ffn_takes_views_that_interleave(ns, experts):
    """Inputs, outputs and gradients that are parts of one buffer beside each
    other give what separate tensors give."""
    t, hidden, inner = 70, 64, 40
    lead = (experts,) if experts else ()
    offsets = torch.tensor([0, 30, 30, 70], dtype=torch.int32, device="cuda") if experts else None
    x, dy = rand(1, t, hidden), rand(2, t, hidden)
    w = rand(3, *lead, inner, hidden), rand(4, *lead, inner, hidden), rand(5, *lead, hidden, inner)
    y, saved = ns.gated_ffn(x, *w, offsets=offsets)
    want = ns.gated_ffn_backward(dy, x, saved, *w, offsets=offsets)
    wide = torch.zeros(t, 4 * hidden + 8, dtype=BF, device="cuda")
    parts = [wide[:, i * hidden + 8:(i + 1) * hidden + 8] for i in range(4)]
    parts[0].copy_(x)
    parts[1].copy_(dy)
    got, _ = ns.gated_ffn(parts[0], *w, offsets=offsets, out=parts[2])
    assert torch.equal(got, y)
    size = inner * hidden
    for split in range(3):
        flat = torch.zeros(*lead, 3 * size + (8 if split == 2 else 0), dtype=BF, device="cuda")
        if split == 0:           # one after the other
            gate, up = (flat[..., i * size:(i + 1) * size].unflatten(-1, (inner, hidden)) for i in range(2))
        elif split == 1:         # row by row
            gate, up = flat[..., :2 * size].unflatten(-1, (inner, 2, hidden)).unbind(-2)
        else:                    # columns of one matrix, with a gap behind it
            both = flat[..., :2 * size].unflatten(-1, (inner, 2 * hidden))
            gate, up = both[..., :hidden], both[..., hidden:]
        down = flat[..., 2 * size:3 * size].unflatten(-1, (hidden, inner))
        got = ns.gated_ffn_backward(parts[1], parts[0], saved, *w, offsets=offsets, out=parts[3], grads=(gate, up, down))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ns.ops_sync()


@pytest.mark.gpu
def test_gated_ffn_refuses_shifted_rows(ns):
    t, hidden, inner = 70, 64, 40
    buf = rand(1, t + 1, hidden)
    x = rand(2, t, hidden)
    w = rand(3, inner, hidden), rand(4, inner, hidden), rand(5, hidden, inner)
    _, saved = ns.gated_ffn(x, *w)
    with pytest.raises(ns.MuonError, match="share memory"):
        ns.gated_ffn_backward(buf[:-1], x, saved, *w, out=buf[1:])
    with pytest.raises(ns.MuonError, match="share memory"):
        ns.gated_ffn_backward(x, buf[1:], saved, *w, out=buf[:-1])
    # where nothing reads them again, they may
    none = (None, None, None)
    want = ns.gated_ffn_backward(buf[:-1].clone(), None, saved, *w, grads=none)[0]
    assert torch.equal(ns.gated_ffn_backward(buf[:-1], None, saved, *w, grads=none, out=buf[1:])[0], want)
    rows = rand(6, t + 1, hidden)
    want = ns.gated_ffn(rows[:-1].clone(), *w, keep=False)[0]
    assert torch.equal(ns.gated_ffn(rows[:-1], *w, keep=False, out=rows[1:])[0], want)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_takes_views_that_interleave(ns, layout):
    """Queries and keys beside each other in one row, in place and to another
    part of it; heads of which only some values turn."""
    plan = ns.RotaryPlan(32, layout=layout)
    row = rand(1, 2, 21, 6 + 2 + 6, 48)
    q, k, other = row.split([6, 2, 6], 2)
    want_q, want_k = ns.rotary(q.clone(), k.clone(), plan, offset=5)
    first = row.clone()
    a, b, c = first.split([6, 2, 6], 2)
    ns.rotary(a, b, plan, offset=5, out_q=c, out_k=b)
    assert torch.equal(c, want_q) and torch.equal(b, want_k) and torch.equal(a, q)
    ns.rotary(a, None, plan, offset=5, out_q=a)
    assert torch.equal(a, want_q)
    # batch x heads x seq x head, written to the other order
    turned = torch.zeros(2, 6, 21, 48, dtype=BF, device="cuda").transpose(1, 2)
    assert torch.equal(ns.rotary(q, None, plan, offset=5, out_q=turned)[0], want_q)
    with pytest.raises(ns.MuonError, match="shares"):
        ns.rotary(row[:, :, :6], None, plan, out_q=row[:, :, 1:7])
    with pytest.raises(ns.MuonError, match="shares"):
        ns.rotary(q, k, plan, out_q=row[:, :, 4:10])


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [64, 33])
def test_dropout_takes_views_that_interleave(ns, cols):
    buf = rand(1, 40, 3 * cols)
    x, r, out = buf.split(cols, 1)
    want = ns.dropout(x.clone(), 0.3, 1, 2, residual=r.clone())
    assert torch.equal(ns.dropout(x, 0.3, 1, 2, residual=r, out=out), want)
    assert torch.equal(ns.dropout(x, 0.3, 1, 2, residual=r, out=r), want)
    row = buf[:1]
    assert torch.equal(ns.dropout(row, 0.0, 1, 2, out=row), row)
    for a, b in ((buf[:-1], buf[1:]), (buf[:, 1:], buf[:, :-1])):
        with pytest.raises(ns.MuonError, match="share memory"):
            ns.dropout(a, 0.3, 1, 2, out=b)
        with pytest.raises(ns.MuonError, match="share memory"):
            ns.dropout(torch.zeros_like(a), 0.3, 1, 2, residual=a, out=b)
