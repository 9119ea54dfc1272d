"""Argument checks of the operators of a block's training step, without a
GPU: every refusal comes before any CUDA call, with its code and a message."""
import ctypes
from ctypes import byref

import pytest
import torch

import ops_oracle as O


@pytest.fixture(scope="module")
def L():
    from newton_schulz_06_gb300 import build as b
    b.build()
    from newton_schulz_06_gb300 import _lib
    return _lib


P = 0x10000            # a pointer that no refused call looks behind


def call(L, name, *args):
    buf = ctypes.create_string_buffer(256)
    rc = getattr(L.lib(), name)(*args, None, buf, 256)
    return rc, buf.value.decode()


def fields(struct, base, **kw):
    a = struct()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def ckpt(L, **kw):
    return fields(L.Ckpt8, dict(q=P, e=P, ld_q=64, ld_e=2), **kw)


NORM = dict(x=P, weight=P, bias=P, y=P + 64, mean=P, rstd=P, rows=4, cols=64, ld_x=64, ld_y=64,
            x_dtype=1, w_dtype=0, eps=1e-5)
NORM_GRAD = dict(dy=P, x=P, mean=P, rstd=P, weight=P, dx=P + 64, dweight=P, dbias=P, rows=4, cols=64,
                 ld_dy=64, ld_x=64, ld_dx=64, x_dtype=1, w_dtype=0)
WGRAD = dict(dy=P, g=P, rows=4, n=64, k=64, experts=1, ld_dy=64, ld_g=64, g_dtype=1)
ROUTE = dict(logits=P, indices=P, weights=P, counts=P, offsets=P, loss=P, kept=P, tokens=4, experts=8,
             k=2, ld_z=8, z_dtype=0, renormalise=1, coef=0.1)
ROUTE_GRAD = dict(logits=P, indices=P, weights=P, counts=P, kept=P, dloss=P, dweights=P,
                  dlogits=P + 64, tokens=4, experts=8, k=2, ld_z=8, ld_dw=2, ld_dz=8, z_dtype=0,
                  renormalise=1, coef=0.1)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(cols=0), "cols"),
    (dict(cols=(1 << 20) + 1), "cols"), (dict(x_dtype=2), "type"), (dict(w_dtype=-1), "type"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(x=None), "x is NULL"),
    (dict(y=None), "y is NULL"), (dict(ld_x=63), "leading dimension"), (dict(ld_y=63), "leading dimension"),
    (dict(ld_y=0), "leading dimension"), (dict(x=P + 1), "aligned"), (dict(weight=P + 2), "aligned"),
    (dict(bias=P + 1), "aligned"), (dict(mean=P + 2), "aligned"), (dict(y=P, ld_x=72), "another leading")])
def test_layer_norm_refuses(L, kw, word):
    rc, msg = call(L, "muon_layer_norm", byref(fields(L.LayerNormArgs, NORM, **kw)))
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


@pytest.mark.parametrize("kw", [dict(e=None), dict(q=P + 8), dict(ld_q=72), dict(ld_q=32), dict(ld_e=1)])
def test_checkpoints_refused(L, kw):
    a = fields(L.LayerNormArgs, NORM)
    a.saved = ckpt(L, **kw)
    for rc, msg in (call(L, "muon_layer_norm", byref(a)),
                    call(L, "muon_ckpt8_pack", P, 1, 4, 64, 64, byref(ckpt(L, **kw))),
                    call(L, "muon_ckpt8_unpack", byref(ckpt(L, **kw)), 4, 64, P, 1, 64)):
        assert rc == L.MUON_ERR_INVALID_ARG and "saved" in msg


def test_pack_and_unpack_refuse(L):
    ok = byref(ckpt(L))
    for args, word in (((P, 1, 4, 64, 64, None), "saved"), ((None, 1, 4, 64, 64, ok), "x is NULL"),
                       ((P, 3, 4, 64, 64, ok), "type"), ((P, 1, 4, 64, 60, ok), "leading"),
                       ((P, 1, -4, 64, 64, ok), "rows"), ((P + 1, 0, 4, 64, 64, ok), "aligned")):
        rc, msg = call(L, "muon_ckpt8_pack", *args)
        assert rc == L.MUON_ERR_INVALID_ARG and word in msg
    # written rows need room of their own
    rc, msg = call(L, "muon_ckpt8_unpack", ok, 4, 64, P, 1, 0)
    assert rc == L.MUON_ERR_INVALID_ARG and "leading" in msg


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(x_dtype=9), "type"), (dict(dy=None), "dy is NULL"),
    (dict(dx=None), "dx is NULL"), (dict(rstd=None), "rstd is NULL"), (dict(mean=None), "mean is NULL"),
    (dict(x=None), "x is NULL"), (dict(ld_dx=8), "leading"), (dict(dx=P), "dx"),
    (dict(dy=P + 1), "aligned"), (dict(dweight=P + 2), "aligned"),
    (dict(dy=P + 64, ld_dy=72), "another leading")])
def test_layer_norm_grad_refuses(L, kw, word):
    a = fields(L.LayerNormGradArgs, NORM_GRAD, **kw)
    rc, msg = call(L, "muon_layer_norm_grad", byref(a), P, 1 << 30)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


def test_layer_norm_grad_refuses_x_beside_a_checkpoint(L):
    a = fields(L.LayerNormGradArgs, NORM_GRAD)
    a.saved = ckpt(L)
    rc, msg = call(L, "muon_layer_norm_grad", byref(a), P, 1 << 30)
    assert rc == L.MUON_ERR_INVALID_ARG and "both" in msg


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(n=0), "cols"), (dict(k=0), "cols"), (dict(g_dtype=5), "type"),
    (dict(experts=0), "experts"), (dict(experts=65537), "experts"), (dict(experts=2), "offsets"),
    (dict(dy=None), "dy is NULL"), (dict(g=None), "g is NULL"), (dict(ld_g=63), "leading"),
    (dict(ld_dy=63), "leading"), (dict(weight=P + 1), "aligned"), (dict(offsets=P + 2), "aligned"),
    (dict(c=P + 64, ld_c=3), "leading"), (dict(c=P, ld_c=128), "other strides"),
    (dict(experts=2, offsets=P, stride_g=64 * 64 - 1), "stride_g"),
    (dict(experts=2, offsets=P, stride_g=4096, c=P + 64, ld_c=64, stride_c=-1), "stride_c")])
def test_weight_grad_refuses(L, kw, word):
    a = fields(L.WeightGradArgs, WGRAD, **kw)
    a.saved = ckpt(L)
    rc, msg = call(L, "muon_weight_grad", byref(a), P, 1 << 40)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(experts=0), "experts"), (dict(experts=1025), "experts"), (dict(k=0), "k out"), (dict(k=9), "k out"),
    (dict(experts=64, ld_z=64, k=33), "k out"), (dict(tokens=-1), "tokens"),
    (dict(tokens=1 << 30, k=2), "tokens"), (dict(z_dtype=2), "type"), (dict(logits=None), "logits"),
    (dict(indices=None), "indices"), (dict(weights=None), "weights"), (dict(counts=None), "counts"),
    (dict(offsets=None), "offsets"), (dict(loss=None), "loss"), (dict(kept=None), "kept"),
    (dict(ld_z=7), "leading"), (dict(logits=P + 2), "aligned")])
def test_route_refuses(L, kw, word):
    rc, msg = call(L, "muon_route", byref(fields(L.RouteArgs, ROUTE, **kw)), P, 1 << 30)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


@pytest.mark.parametrize("kw,word", [
    (dict(experts=1025), "experts"), (dict(k=9), "k out"), (dict(dlogits=None), "dlogits"),
    (dict(indices=None), "indices"), (dict(counts=None), "counts"), (dict(kept=None), "kept"),
    (dict(ld_dw=1), "leading"), (dict(ld_dz=7), "leading"), (dict(dloss=P + 1), "aligned"),
    (dict(dlogits=P, ld_dz=9), "another leading")])
def test_route_grad_refuses(L, kw, word):
    rc, msg = call(L, "muon_route_grad", byref(fields(L.RouteGradArgs, ROUTE_GRAD, **kw)))
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg


def test_no_arguments_and_no_workspace(L):
    n = ctypes.c_size_t()
    for name, struct, base in (("muon_layer_norm_grad", L.LayerNormGradArgs, NORM_GRAD),
                               ("muon_weight_grad", L.WeightGradArgs, WGRAD),
                               ("muon_route", L.RouteArgs, ROUTE)):
        assert call(L, name, None, None, 0)[0] == L.MUON_ERR_INVALID_ARG
        assert getattr(L.lib(), name + "_workspace")(None, byref(n)) == L.MUON_ERR_INVALID_ARG
        a = fields(struct, base)
        if "saved" in dict(struct._fields_) and name == "muon_weight_grad":
            a.saved = ckpt(L)
        assert getattr(L.lib(), name + "_workspace")(byref(a), None) == L.MUON_ERR_INVALID_ARG
        assert getattr(L.lib(), name + "_workspace")(byref(a), byref(n)) == 0
        if n.value:
            rc, msg = call(L, name, byref(a), P, n.value - 1)
            assert rc == L.MUON_ERR_NO_WORKSPACE and "workspace" in msg
            assert call(L, name, byref(a), None, n.value)[0] == L.MUON_ERR_NO_WORKSPACE
            assert call(L, name, byref(a), P + 16, n.value)[0] == L.MUON_ERR_INVALID_ARG
    for name in ("muon_layer_norm", "muon_route_grad"):
        assert call(L, name, None)[0] == L.MUON_ERR_INVALID_ARG


def test_messages_fit_any_buffer(L):
    a = fields(L.LayerNormArgs, NORM, rows=-1)
    assert L.lib().muon_layer_norm(byref(a), None, None, 0) == L.MUON_ERR_INVALID_ARG
    buf = ctypes.create_string_buffer(b"x" * 8, 8)
    assert L.lib().muon_layer_norm(byref(a), None, buf, 4) == L.MUON_ERR_INVALID_ARG
    assert buf.raw[:4] == b"row\0" and buf.raw[4:7] == b"xxx"


def test_tensors_are_checked():
    """The Python face refuses what it cannot pass on (CPU tensors among it)."""
    import newton_schulz_06_gb300 as ns
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ns.layer_norm(x)
    with pytest.raises(ValueError, match="2-D"):
        ns.layer_norm(x[0])
    with pytest.raises(ValueError, match="int8"):
        ns.Checkpoint8(x, x, 64)
    q, e = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)
    for bad in ((q[:, :63], e, 64), (q, e[:, :1], 64), (q[:3], e, 64), (q, e, 0), (q, e, 65),
                (q.t(), e, 4)):
        with pytest.raises(ValueError):
            ns.Checkpoint8(*bad)
    with pytest.raises(ValueError, match="CUDA"):
        ns.weight_grad(x.bfloat16(), ns.Checkpoint8(q, e, 64))
    with pytest.raises(ValueError, match="CUDA"):
        ns.route(x, 2)


# the 64-bit forms themselves, against differences and by hand

def test_oracle_code_by_hand():
    v = torch.tensor([[1.0, -2.0, 0.5, 1.99, 127.0 / 64, 3.0] + [0.0] * 26], dtype=torch.float64)
    q, e = O.encode(v)
    assert e.tolist() == [[128]]                       # floor(log2 3) = 1: steps of 2^-5
    assert q[0, :6].tolist() == [32, -64, 16, 64, 64, 96]
    assert O.decode(q, e, 6)[0, :3].tolist() == [1.0, -2.0, 0.5]
    q, e = O.encode(torch.tensor([[1.999, 2.5 / 64, 3.5 / 64] + [0.0] * 29], dtype=torch.float64))
    assert q[0, :3].tolist() == [127, 2, 4]            # limited; ties to even


@pytest.mark.parametrize("renormalise", [True, False])
def test_oracle_router_gradient_is_that_of_its_objective(renormalise):
    g = torch.Generator().manual_seed(3)
    z = torch.randn(6, 9, generator=g, dtype=torch.float64)
    z[1, 3:] = float("-inf")
    mask = [1, 1, 0, 1, 1, 1]
    idx, w, counts, offsets, loss, kept, p = O.route(z, 4, mask, 0.3, renormalise)
    assert kept == 5 and idx[1].tolist()[3] == -1 and offsets[-1] == counts.sum() == 19
    dw = torch.randn(6, 4, generator=g, dtype=torch.float64)
    zr = z.clone().requires_grad_()
    O.route_objective(zr, idx, counts, kept, 0.3, renormalise, 0.9, dw).backward()
    got = O.route_grad(z, idx, counts, kept, 0.3, renormalise, 0.9, dw)
    assert torch.allclose(torch.nan_to_num(zr.grad), got, rtol=1e-12, atol=1e-14)
    assert abs(O.route_objective(z, idx, counts, kept, 0.3, renormalise, 1.0, None).item() - loss) < 1e-14


def test_packed_arguments_have_the_structures_layout(L):
    for cls in (L.Ckpt8, L.LayerNormArgs, L.LayerNormGradArgs, L.WeightGradArgs, L.RouteArgs,
                L.RouteGradArgs):
        pack = L.packer(cls)
        assert pack.size == ctypes.sizeof(cls)
        n = len(pack.unpack(bytes(pack.size)))
        a = cls.from_buffer_copy(pack.pack(*range(1, n + 1)))
        flat = []

        def walk(v):
            for f, _ in v._fields_:
                x = getattr(v, f)
                if isinstance(x, ctypes.Structure):
                    walk(x)
                else:
                    flat.append(x)

        walk(a)
        assert flat == list(range(1, n + 1))
