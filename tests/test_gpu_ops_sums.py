"""Long sums of the weight gradient: how much of a sum the tensor cores' running
sums may lose.

Sums of one sign, where what is cut off adds up.  A product of 16 tokens cuts
the running sum off at its last place (2^-23 of it at most) up to twice; on
average each cut takes half a place, and a sum that grows evenly has 0.4 of its
final places on the way: 0.4 * 2^-23 a product on average."""
import pytest
import torch

from ops_oracle import D, U32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TOKENS = 200003


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def one_sign(ns, tokens, n, k, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dy = torch.randn(tokens, n, generator=g, device=DEV).abs_().to(BF)
    return dy, ns.checkpoint8(torch.randn(tokens, k, generator=g, device=DEV).abs_())


def columns(dy, saved, a, b, step):
    """Every step-th column of the gradient over tokens a .. b, in 64 bits."""
    h = saved.values(F32)[:, ::step]
    want = torch.zeros(dy.shape[1], h.shape[1], dtype=D, device=DEV)
    for t in range(a, b, 16384):
        end = min(b, t + 16384)
        want += dy[t:end].to(D).t() @ h[t:end].to(D)
    return want


def test_fp32_sums_are_added_up_to_nearest(ns):
    """Chunks of 1024 tokens (64 products of two cuts), added up with one
    rounding each.  One running sum over all the tokens would lose ten times
    as much on average."""
    dy, saved = one_sign(ns, TOKENS, 2048, 2560, 1)
    got = ns.weight_grad(dy, saved, dtype=F32)[:, ::40].to(D)
    want = columns(dy, saved, 0, TOKENS, 40)
    bound = 64 * 2 * 2.0 ** -23 + (TOKENS / 1024 + 1) * U32
    assert bound < 0.1 * 0.4 * 2.0 ** -23 * TOKENS / 16 * 2
    assert ((got - want).abs() <= bound * want).all()


@pytest.mark.parametrize("experts", [1, 4])
@pytest.mark.parametrize("n,k", [(4096, 5120), (512, 512)])
def test_bf16_sums_lose_no_more_than_their_chunks(ns, n, k, experts):
    """bf16 results hide what a sum has lost in their own rounding; over many
    of them it shows in the mean difference from the exact values' roundings.
    Chunks of 16384 tokens (1024 products) lose 4.9e-5 on average at most, one
    running sum over all the tokens up to twelve times that.  The mean over 50000
    values and more is good to 5e-6."""
    tokens = TOKENS if experts == 1 else TOKENS + 100
    dy, saved = one_sign(ns, tokens, n, k, 2)
    ends, offsets = [0, tokens], None
    if experts > 1:
        # one expert has nearly all tokens; the others' sums are short
        ends = [0, 40, TOKENS + 40, TOKENS + 40, tokens]
        offsets = torch.tensor(ends, dtype=torch.int32, device=DEV)
    got = ns.weight_grad(dy, saved, offsets=offsets).view(experts, n, k)[:, :, ::5].to(D)
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        want = columns(dy, saved, a, b, 5)
        if a == b:
            assert not got[e].any()
            continue
        products = min(b - a, 16384) / 16
        assert ((got[e] - want).abs() <= (2.0 ** -8 + products * 2.0 ** -22) * want).all()
        lost = ((want.to(BF).to(D) - got[e]) / want).mean().item()
        assert abs(lost) <= 0.4 * 2.0 ** -23 * products + 5e-6
