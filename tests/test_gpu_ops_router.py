"""The router where logits lie far apart."""
import pytest
import torch

import ops_oracle as O
from ops_oracle import D, U32, close, to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
# an exponential: 2^-22 for its power of two and a rounding, in the numerator
# and in the sum; the sum's chain of at most 40 additions; three more roundings
REL = (2 * 5 + 40 + 3) * U32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("experts,k", [(8, 4), (12, 12), (128, 8), (384, 8), (1000, 6)])
def test_weights_of_far_logits_are_as_exact_as_those_of_near_ones(ns, experts, k, dtype):
    """One logit far above the others, on a grid on which differences are
    exact: the others' weights are e^-86 to e^-40 of its own."""
    g = torch.Generator().manual_seed(1)
    z = torch.randint(-40 * 4, -10 * 4, (50, experts), generator=g).double() / 4
    z[torch.arange(50), torch.randint(0, experts, (50,), generator=g)] = \
        torch.randint(30 * 4, 46 * 4, (50,), generator=g).double() / 4
    z = z.to(dtype).to(DEV)
    r = ns.route(z, k, renormalise=False)
    idx, w, counts, _, _, kept, p = O.route(to64(z), k, None, 0.01, False)
    assert torch.equal(r.indices.cpu().long(), idx)
    assert p.min() < 1e-30                       # of the inputs: some are far
    close(r.weights, w, REL * w, "weights")
    dw = torch.randn(50, k, generator=g).to(DEV)
    got = ns.route_backward(z, r, dweights=dw)
    want = O.route_grad(to64(z), idx, counts, kept, 0.01, False, 0.0, to64(dw))
    up = torch.zeros_like(p).scatter_(1, idx, to64(dw).abs())
    out = 2.0 ** -8 if dtype == BF else 2.0 ** -23
    close(got, want, 2 * REL * p * (up + (p * up).sum(-1, keepdim=True)) + out * want.abs(), "dlogits")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_exponentials_past_their_range_are_zero(ns, dtype):
    """e^-200 and e^-infinity are 0, one infinity or NaN makes its row NaN."""
    z = torch.full((5, 40), -150.0, dtype=dtype)
    z[:, 3] = 50.0
    z[1, 7:] = -float("inf")
    z[2, 9], z[3, 9] = float("inf"), float("nan")
    z[4] = 3e38
    r = ns.route(z.to(DEV), 3)
    assert torch.equal(r.weights[:2].cpu(), torch.tensor([[1.0, 0.0, 0.0]] * 2))
    assert torch.isnan(r.weights[2:4]).all()
    close(r.weights[4], torch.full((3,), 1 / 3), 4 * U32, "weights")
    dz = ns.route_backward(z.to(DEV), r, dweights=torch.ones(5, 3, device=DEV))
    assert not dz[:2].any() and torch.isnan(dz[2:4]).all() and torch.isfinite(dz[4].float()).all()
