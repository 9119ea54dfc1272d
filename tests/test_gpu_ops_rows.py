"""Layer norm over rows that are hard: means far above the deviation, rows without
any, means far below it."""
import pytest
import torch

import ops_oracle as O
from ops_oracle import D, U32, to64
from test_gpu_ops import check_norm_grads

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ns():
    import newton_schulz_06_gb300 as ns
    return ns


def rand(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("rows,cols,dtype", [(40, 200, F32), (40, 203, BF), (33, 2048, F32), (20, 7168, BF),
                                             (9, 4099, F32), (3, 33000, F32)])
def test_the_gradient_differentiates_the_forward_pass(ns, rows, cols, dtype):
    """h is (x - mean) * rstd, rounded twice, whatever the mean: rows with a
    mean 1000 times the deviation, and rows of one value, whose h is 0."""
    x = rand(1, rows, cols) + 1000.0
    x[::3] = 1000.0 * (1 + torch.arange(0, rows, 3, device=DEV)[:, None] % 7)
    x = x.to(dtype)
    dy, w, b = rand(2, rows, cols, dtype=dtype), rand(3, cols), rand(4, cols)
    _, mean, rstd = ns.layer_norm(x, w, b)
    got = ns.layer_norm_backward(dy, x, mean, rstd, w, b)
    h = (to64(x) - to64(mean)[:, None]) * to64(rstd)[:, None]
    assert not h[::3].any()
    check_norm_grads(got, to64(dy), h, to64(rstd), to64(w), dtype, 2.01 * U32 * h.abs())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(40, 200), (33, 2048), (20, 7168), (9, 4099), (3000, 7168), (3, 70000),
                                       (10000, 1024)])
def test_a_mean_that_can_be_exact_is(ns, rows, cols, dtype):
    """Values on a grid, whose sums fp32 holds exactly: the mean is off by the
    rounding of 1 / cols and of one product, however small it is beside the
    deviation."""
    g = torch.Generator().manual_seed(5)
    most = min(255, (1 << 24) // cols)
    whole = torch.randint(-most, most + 1, (rows, cols), generator=g)
    x = (whole.to(F32) / 64).to(dtype).to(DEV)
    assert torch.equal(x.double().cpu() * 64, whole.double())
    want = whole.to(DEV).sum(-1).double() / 64 / cols
    y, mean, rstd = ns.layer_norm(x)
    assert ((mean.double() - want).abs() <= 2.01 * U32 * want.abs()).all()
    saved_rstd = ns.layer_norm_checkpoint(x)[1]
    assert torch.equal(saved_rstd, rstd)


@pytest.mark.parametrize("rows,cols", [(40, 200), (20, 7168), (3000, 7168), (3, 70000)])
def test_a_mean_above_the_deviation_is_corrected(ns, rows, cols):
    """A sum in chains of L terms is off by up to L / 2 places; its correction
    leaves the mean within a place or so (and the rounding of the deviations)."""
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(rows, cols, generator=g) + 1000.7).to(DEV)
    want = x.double().mean(-1)
    mean = ns.layer_norm(x)[1].double()
    assert ((mean - want).abs() <= 2 * U32 * want).all()
