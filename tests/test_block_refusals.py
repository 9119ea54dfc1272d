"""Argument checks of the operators inside a block, without a GPU: every
refusal comes before any CUDA call, with its code and a message; and the
64-bit forms that the GPU tests compare against."""
import ctypes
import math
from ctypes import byref

import pytest
import torch

import block_oracle as O


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


FFN = dict(x=P, w_gate=P, w_up=P, w_down=P, y=P, gate=P, up=P, rows=4, hidden=64, inner=32, experts=1,
           ld_x=64, ld_gate=64, ld_up=64, ld_down=32, ld_y=64, ld_kept=32)
GRAD = dict(dy=P, x=P, gate=P, up=P, w_gate=P, w_up=P, w_down=P, dx=P + 1024, dw_gate=P, dw_up=P, dw_down=P, rows=4,
            hidden=64, inner=32, experts=1, ld_dy=64, ld_x=64, ld_kept=32, ld_gate=64, ld_up=64, ld_down=32,
            ld_dx=64, ld_dw_gate=64, ld_dw_up=64, ld_dw_down=32, g_dtype=1)
EXPERTS = dict(offsets=P, experts=3, stride_gate=2048, stride_up=2048, stride_down=2048, stride_dw_gate=2048,
               stride_dw_up=2048, stride_dw_down=2048)
FORWARD_EXPERTS = {k: v for k, v in EXPERTS.items() if "dw" not in k}


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 31) - 1), "rows"), (dict(hidden=0), "hidden"),
    (dict(hidden=262145), "hidden"), (dict(inner=0), "inner"), (dict(inner=262145), "inner"),
    (dict(experts=2), "offsets"), (dict(experts=0), "experts"), (dict(experts=1025, offsets=P), "experts"),
    (dict(activation=3), "activation"), (dict(activation=-1), "activation"), (dict(offsets=P + 2), "offsets"),
    (dict(x=None), "x is NULL"), (dict(x=P + 1), "aligned"), (dict(ld_x=63), "x has too small"),
    (dict(w_gate=None), "w_gate is NULL"), (dict(ld_up=63), "w_up"), (dict(ld_down=31), "w_down"),
    (dict(w_up=P + 1), "aligned"), (dict(y=None), "y is NULL"), (dict(ld_y=0), "y has too small"),
    (dict(gate=None), "without"), (dict(up=None), "without"), (dict(ld_kept=31), "gate"),
    ({**FORWARD_EXPERTS, "stride_gate": -1}, "negative")])
def test_gated_ffn_refuses(L, kw, word):
    a = fields(L.GatedFfnArgs, FFN, **kw)
    rc, msg = call(L, "muon_gated_ffn", byref(a), P, 1 << 30)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg, msg


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(hidden=0), "hidden"), (dict(inner=0), "inner"), (dict(g_dtype=2), "type"),
    (dict(experts=2), "offsets"), (dict(activation=9), "activation"), (dict(dy=None), "dy is NULL"),
    (dict(x=None), "x is NULL"), (dict(ld_x=1), "x has too small"), (dict(gate=None), "gate is NULL"),
    (dict(up=P + 1), "up is not aligned"), (dict(ld_kept=8), "gate"), (dict(w_gate=None), "w_gate"),
    (dict(w_down=None), "w_down"), (dict(ld_dx=63), "dx"), (dict(ld_dw_gate=0), "dw_gate"),
    (dict(dw_up=P + 2, g_dtype=0), "dw_up"), (dict(ld_dw_down=31), "dw_down"), (dict(h=P, ld_d=31), "dgate, dup or h"),
    (dict(dgate=P + 1, ld_d=32), "dgate, dup or h"), (dict(dx=P, dy=P, x=P + 64), "dx is dy or x"),
    (dict(dx=P, x=P, dy=P + 64), "dx is dy or x"), ({**EXPERTS, "stride_dw_down": 2047}, "dw_down"),
    ({**EXPERTS, "stride_up": -8}, "w_up")])
def test_gated_ffn_grad_refuses(L, kw, word):
    a = fields(L.GatedFfnGradArgs, GRAD, **kw)
    rc, msg = call(L, "muon_gated_ffn_grad", byref(a), P, 1 << 30)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg, msg


def test_gated_ffn_workspace(L):
    size = ctypes.c_size_t()
    for name, struct, base in (("muon_gated_ffn", L.GatedFfnArgs, FFN), ("muon_gated_ffn_grad", L.GatedFfnGradArgs, GRAD)):
        query = getattr(L.lib(), name + "_workspace")
        a = fields(struct, base)
        assert query(byref(a), byref(size)) == 0 and size.value >= 4 * 32 * 2
        need = size.value
        assert call(L, name, byref(a), P, need - 1)[0] == L.MUON_ERR_NO_WORKSPACE
        assert call(L, name, byref(a), None, need)[0] == L.MUON_ERR_NO_WORKSPACE
        assert call(L, name, byref(a), P + 128, need)[0] == L.MUON_ERR_INVALID_ARG
        # rows that TMA cannot read are copied there
        assert query(byref(fields(struct, base, ld_x=65)), byref(size)) == 0 and size.value > need
        assert query(None, byref(size)) == L.MUON_ERR_INVALID_ARG
        assert query(byref(fields(struct, base, rows=-1)), byref(size)) == L.MUON_ERR_INVALID_ARG
        assert query(byref(a), None) == L.MUON_ERR_INVALID_ARG
        # more tiles than the kernels count
        big = dict(rows=(1 << 31) - 300, hidden=262144, inner=262144)
        assert query(byref(fields(struct, base, **big)), byref(size)) == L.MUON_ERR_UNSUPPORTED


TURNS = (ctypes.c_uint64 * 8)()


def rotary(L, q=None, k=None, **kw):
    a = fields(L.RotaryArgs, dict(turns=ctypes.addressof(TURNS), batch=2, seq=3, head=16, pairs=8, x_dtype=1,
                                  scale=1.0), **kw)
    one = dict(x=P, y=P, heads=2, x_batch=96, x_seq=32, x_head=16, y_batch=96, y_seq=32, y_head=16)
    a.q = fields(L.RotaryTensor, one, **(q or {}))
    a.k = fields(L.RotaryTensor, one, **(k or {}))
    return call(L, "muon_rotary", byref(a))


@pytest.mark.parametrize("kw,word", [
    (dict(x_dtype=2), "type"), (dict(layout=2), "layout"), (dict(pairs=0), "pairs"), (dict(pairs=257), "pairs"),
    (dict(head=15), "head"), (dict(head=65537), "head"), (dict(batch=-1), "batch"), (dict(seq=-1), "seq"),
    (dict(batch=1 << 20, seq=1 << 20), "batch"), (dict(turns=None), "turns"), (dict(scale=math.inf), "scale"),
    (dict(scale=math.nan), "scale"), (dict(positions=P + 4, positions_64=1), "positions"),
    (dict(positions=P + 2), "positions"), (dict(positions=P, stride_positions=-1), "positions"),
    (dict(q=dict(x=None)), "q is NULL"), (dict(k=dict(y=None)), "k is NULL"), (dict(q=dict(x=P + 1)), "aligned"),
    (dict(k=dict(heads=-1)), "heads"), (dict(q=dict(heads=65537)), "heads"),
    (dict(q=dict(heads=65536), head=4096), "heads"),
    (dict(q=dict(x_seq=-16)), "negative"), (dict(q=dict(y_head=0)), "share memory"),
    (dict(k=dict(y_seq=0)), "share memory"), (dict(k=dict(y_batch=0)), "share memory"), (dict(k=dict(y_head=32)), "in place")])
def test_rotary_refuses(L, kw, word):
    rc, msg = rotary(L, **kw)
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg, msg


@pytest.mark.parametrize("kw,word", [
    (dict(pairs=0), "pairs"), (dict(pairs=257), "pairs"), (dict(base=1.0), "base"), (dict(base=math.nan), "base"),
    (dict(base=math.inf), "base"), (dict(scaling=4), "scaling"), (dict(factor=0.5), "factor"),
    (dict(factor=math.nan), "factor"), (dict(pairs=1, scaling=2), "pairs"),
    (dict(scaling=3, original=0.0), "original"), (dict(scaling=3, fast=1.0), "slow"),
    (dict(scaling=3, slow=0.0), "slow"), (dict(turns=None), "NULL"), (dict(scale=None), "NULL")])
def test_rotary_frequencies_refuse(L, kw, word):
    a = dict(pairs=8, base=1e4, scaling=0, factor=1.0, original=4096.0, fast=32.0, slow=1.0, turns=TURNS,
             scale=byref(ctypes.c_float()))
    a.update(kw)
    buf = ctypes.create_string_buffer(256)
    rc = L.lib().muon_rotary_frequencies(*a.values(), buf, 256)
    assert rc == L.MUON_ERR_INVALID_ARG and word in buf.value.decode()


def test_rotary_frequencies(L):
    import newton_schulz_06_gb300 as ns
    for args in (dict(dim=128), dict(dim=2), dict(dim=512, base=1e6), dict(dim=64, scaling="linear", factor=3.0),
                 dict(dim=96, scaling="ntk", factor=16.0), dict(dim=64, scaling="yarn", factor=1.0),
                 dict(dim=128, scaling="yarn", factor=40.0, fast=16.0, slow=2.0)):
        plan = ns.RotaryPlan(**args)
        freq, scale = O.frequencies(**args)
        assert abs(plan.scale - scale) <= O.U32 * scale and len(plan.frequencies) == args["dim"] // 2
        for a, b in zip(plan.frequencies, freq):
            assert abs(a - b) <= 2.0 ** -50 * b + 2 * math.pi * 2.0 ** -64
    import copy
    import pickle
    for twin in (copy.deepcopy(plan), pickle.loads(pickle.dumps(plan))):
        assert twin.frequencies == plan.frequencies and (twin.dim, twin.layout, twin.scale) == (
            plan.dim, plan.layout, plan.scale)
    for bad in (dict(dim=3), dict(dim=0), dict(dim=514), dict(dim=8, layout="both"), dict(dim=8, scaling="more")):
        with pytest.raises(ValueError):
            ns.RotaryPlan(**bad)
    with pytest.raises(L.MuonError):
        ns.RotaryPlan(8, base=0.5)


DROP = dict(x=P, residual=P, y=P + 64, rows=4, cols=64, ld_x=64, ld_r=64, ld_y=64, p=0.1, x_dtype=1)


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(rows=1 << 31), "rows"), (dict(cols=0), "cols"), (dict(cols=(1 << 20) + 1), "cols"),
    (dict(x_dtype=2), "type"), (dict(p=-0.1), "p out"), (dict(p=1.1), "p out"), (dict(p=math.nan), "p out"),
    (dict(x=None), "x is NULL"), (dict(y=None), "y is NULL"), (dict(ld_x=63), "x has"), (dict(ld_y=0), "y has"),
    (dict(ld_r=63), "residual has"), (dict(x=P + 1), "aligned"), (dict(residual=P + 1), "aligned"),
    (dict(counter=P + 4), "counter"), (dict(y=P, ld_x=72), "y is x"),
    (dict(y=P, x=P + 64, ld_r=72), "y is residual")])
def test_dropout_refuses(L, kw, word):
    rc, msg = call(L, "muon_dropout", byref(fields(L.DropoutArgs, DROP, **kw)))
    assert rc == L.MUON_ERR_INVALID_ARG and word in msg, msg


def test_calls_with_nothing_to_do(L):
    assert call(L, "muon_dropout", byref(fields(L.DropoutArgs, DROP, rows=0, x=None, y=None, residual=None)))[0] == 0
    assert rotary(L, batch=0, q=dict(x=None))[0] == 0 and rotary(L, q=dict(heads=0), k=dict(heads=0))[0] == 0
    for name in ("muon_rotary", "muon_dropout"):
        assert call(L, name, None)[0] == L.MUON_ERR_INVALID_ARG
    for name in ("muon_gated_ffn", "muon_gated_ffn_grad"):
        assert call(L, name, None, None, 0)[0] == L.MUON_ERR_INVALID_ARG


def test_python_face_refuses_cpu_tensors_and_wrong_shapes(L):
    import newton_schulz_06_gb300 as ns
    x, w, d = torch.zeros(4, 64).bfloat16(), torch.zeros(32, 64).bfloat16(), torch.zeros(64, 32).bfloat16()
    with pytest.raises(ValueError, match="CUDA"):
        ns.gated_ffn(x, w, w, d)
    with pytest.raises(ValueError, match="CUDA"):
        ns.gated_ffn_backward(x, x, (w, w), w, w, d)
    with pytest.raises(ValueError, match="2-D"):
        ns.dropout(x[0], 0.1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ns.dropout(x, 0.1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        ns.rotary(x.view(4, 1, 64), None, ns.RotaryPlan(64))


def test_packed_arguments_have_the_structures_layout(L):
    for cls in (L.GatedFfnArgs, L.GatedFfnGradArgs, L.RotaryArgs, L.DropoutArgs):
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


# --------------------------------------------------------- the 64-bit forms

def test_oracle_generator_has_its_published_answers():
    """The known answers that the generator's authors give."""
    low = 0xFFFFFFFF
    assert O.philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert O.philox((low,) * 4, (low,) * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert O.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_oracle_gradient_is_autograds(name):
    g = torch.Generator().manual_seed(1)
    offsets = torch.tensor([0, 3, 3, 8])
    x = torch.randn(8, 6, generator=g, dtype=torch.float64, requires_grad=True)
    w = [torch.randn(3, *s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((5, 6), (5, 6), (6, 5))]
    dy = torch.randn(8, 6, generator=g, dtype=torch.float64)
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    y = torch.cat([(act(x[a:b] @ w[0][e].t()) * (x[a:b] @ w[1][e].t())) @ w[2][e].t()
                   for e, (a, b) in enumerate(O.spans(offsets, 8))])
    y.backward(dy)
    (y64, g64, u64), _ = O.ffn(x.detach(), *[v.detach() for v in w], offsets, name)
    assert torch.allclose(y64, y.detach(), rtol=1e-12, atol=1e-13)
    got, _ = O.ffn_grad(dy, x.detach(), g64, u64, *[v.detach() for v in w], offsets, name)
    for a, b in zip(got, (x.grad, *[v.grad for v in w])):
        assert torch.allclose(a, b, rtol=1e-11, atol=1e-13)


def test_oracle_rotation_keeps_lengths_and_differences():
    """A rotation; and the product of a query and a key goes by the distance of
    their positions."""
    g = torch.Generator().manual_seed(2)
    q, k = torch.randn(1, 1, 1, 16, generator=g).double(), torch.randn(1, 1, 1, 16, generator=g).double()
    O.HALF[torch.float64] = 2.0 ** -53
    freq, scale = O.frequencies(16)
    for layout in ("half", "interleaved"):
        def at(x, p):
            return O.rotary(x, torch.tensor([[p]]), 16, freq, scale, layout)[0]
        assert abs(at(q, 9).norm() - q.norm()) < 1e-12
        a, b = (at(q, 100) * at(k, 93)).sum(), (at(q, 7) * at(k, 0)).sum()
        assert abs(a - b) < 1e-11 and (at(q, 0) - q).abs().max() == 0
