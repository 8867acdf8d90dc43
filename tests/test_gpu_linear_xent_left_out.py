"""GPU tests of the linear head's cross entropy: rows that are left out have
zero gradients whatever the upstream gradient and w hold."""
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


# Whole products, sliced ones (a join kernel), odd widths, one and two CTAs' rows.
@pytest.mark.parametrize("N,V,D", [(5, 700, 64), (40, 20000, 65), (300, 9001, 200), (300, 500, 72), (2000, 300, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("upstream", [float("inf"), float("nan")])
def test_upstream_overflow(N, V, D, dtype, upstream):
    """An overflowed loss scale reaches the rows that take part, and no other."""
    g = torch.Generator("cuda").manual_seed(N)
    x = torch.randn(N, D, generator=g, device="cuda").to(dtype)
    w = torch.randn(V, D, generator=g, device="cuda").to(dtype)
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    y[::3] = -100
    for reduction in ("mean", "sum", "none"):
        grad = torch.full((N,) if reduction == "none" else (), upstream, device="cuda")
        _, lse = zr.zr_linear_xent_fwd(x, w, y, reduction)
        gx, _ = zr.zr_linear_xent_bwd(grad, x, w, y, lse, reduction)
        assert not gx[::3].any(), reduction
        assert not torch.isfinite(gx[y >= 0]).all(1).any(), reduction


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 300])
def test_infinite_weights(N, dtype):
    """A class whose weights overflowed: rows left out stay 0."""
    x, w = torch.ones(N, 64, device="cuda", dtype=dtype), torch.ones(500, 64, device="cuda", dtype=dtype)
    w[17, 3] = float("inf")
    y = torch.zeros(N, dtype=torch.int64, device="cuda")
    y[1] = -100
    _, lse = zr.zr_linear_xent_fwd(x, w, y)
    gx, _ = zr.zr_linear_xent_bwd(torch.ones((), device="cuda"), x, w, y, lse)
    assert not gx[1].any() and torch.isnan(gx[0]).any()
