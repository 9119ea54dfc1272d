"""The norm's weight and bias go to every operator that takes them in the type
that they have."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def rand(seed, *shape, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("wdtype", [BF, F32])
def test_one_weight_and_bias_for_all(ns, wdtype):
    """The calls of the README, with the same w and b."""
    t, n, k = 300, 264, 520
    x, dy, w, b = rand(1, t, k), rand(2, t, n), rand(3, k, dtype=wdtype), rand(4, k, dtype=wdtype)
    y, rstd, saved = ns.layer_norm_checkpoint(x, w, b)
    G = torch.empty(n, k, dtype=BF, device=DEV)
    ns.weight_grad(dy, saved, weight=w, bias=b, out=G)
    dx, dw, db = ns.layer_norm_backward(y, saved, None, rstd, w, b)
    assert dw.dtype == db.dtype == wdtype
    assert torch.equal(G, ns.weight_grad(dy, saved, weight=w.float(), bias=b.float()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (300, 264, 521), (2111, 768, 776), (4097, 128, 96),
                                   (1025, 2049, 2305)])
def test_bf16_weight_and_bias_are_what_they_stand_for(ns, t, n, k, dtype):
    """A bf16 number is an fp32 number: the same bits as from fp32 copies, with
    either and with both, split and not, one matrix and several."""
    dy, saved = rand(5, t, n), ns.checkpoint8(rand(6, t, k))
    w, b = rand(7, k + 3)[3:], rand(8, k + 1)[1:]
    offsets = torch.tensor([0, t // 3, t // 3, t], dtype=torch.int32, device=DEV)
    for o in (None, offsets):
        for kw in (dict(weight=w), dict(bias=b), dict(weight=w, bias=b)):
            wide = {name: v.float() for name, v in kw.items()}
            assert torch.equal(ns.weight_grad(dy, saved, offsets=o, dtype=dtype, **kw),
                               ns.weight_grad(dy, saved, offsets=o, dtype=dtype, **wide))


def test_weights_of_two_types_are_refused(ns):
    dy, saved = rand(9, 4, 8), ns.checkpoint8(rand(10, 4, 32))
    with pytest.raises(ValueError, match="differ in type"):
        ns.weight_grad(dy, saved, weight=rand(11, 32), bias=rand(12, 32, dtype=F32))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ns.weight_grad(dy, saved, weight=rand(11, 32).half())


@pytest.mark.parametrize("wdtype", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("t,n,k", [(0, 40, 65), (300, 264, 520), (3000, 64, 64)])
def test_a_matrix_without_tokens_is_zero_whatever_its_weights(ns, t, n, k, dtype, wdtype):
    """An infinity or a NaN among the norm's weights shows where there are
    tokens, and nowhere else; C passes through."""
    dy = rand(13, t, n)
    saved = ns.checkpoint8(rand(14, t, k)) if t else ns.Checkpoint8.empty(0, k, DEV)
    w, b = rand(15, k, dtype=wdtype), rand(16, k, dtype=wdtype)
    w[3], b[5] = float("inf"), float("nan")
    offsets = torch.tensor([0, 0, t, t], dtype=torch.int32, device=DEV)
    got = ns.weight_grad(dy, saved, weight=w, bias=b, offsets=offsets, dtype=dtype)
    assert not got[[0, 2]].any()
    if t:
        assert torch.isnan(got[1, :, 5]).all() and not torch.isfinite(got[1, :, 3]).any()
        assert torch.isfinite(got[1, :, 6:].float()).all()
    c = rand(17, 3, n, k, dtype=dtype)
    got = ns.weight_grad(dy, saved, weight=w, bias=b, offsets=offsets, add=c, dtype=dtype)
    assert torch.equal(got[[0, 2]], c[[0, 2]])
    if not t:
        assert not ns.weight_grad(dy, saved, weight=w, bias=b, dtype=dtype).any()
