"""GPU tests of layer norm's backward on many rows of more than 8192 columns."""
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


@pytest.mark.parametrize("R,D", [(40000, 8200), (40000, 8193), (9000, 40001), (300000, 8193)])
def test_many_long_rows(R, D):
    """A lane adds 128 rows at most, the warps 8 more, and the second pass is
    compensated with a tree of 8: (128 + 40) u of the sum.  The gradient is a
    constant just below half a unit in the last place of sums of 512 to 1024,
    so that one long run of additions would lose it every time."""
    t = 1 + 2.0 ** -15 - 2.0 ** -21
    g = torch.full((1, 1), t, device="cuda").expand(R, D)
    x = torch.linspace(-1.5, 2.5, D, device="cuda")[None].expand(R, D)
    mean, rstd = torch.full((R,), 0.5, device="cuda"), torch.full((R,), 2.0, device="cuda")
    _, gg, gb = zr.zr_layer_norm_bwd(g, x, None, mean, rstd, want=(False, True, True))
    want = R * t
    assert float((gb.double() - want).abs().max()) <= (128 + 40) * U * want
    xh = (x[0].double() - 0.5) * 2
    # xh is within 2u of itself, and so is its product.
    assert bool(((gg.double() - want * xh).abs() <= (128 + 44) * U * want * xh.abs() + 1e-30).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_with_a_mean(dtype):
    g0 = torch.Generator("cuda").manual_seed(1)
    R, D = 5000, 9001
    x = torch.randn(R, D, generator=g0, device="cuda").to(dtype)
    g = (torch.randn(R, D, generator=g0, device="cuda") + 3).to(dtype)
    _, mean, rstd = zr.zr_layer_norm_fwd(x)
    _, gg, gb = zr.zr_layer_norm_bwd(g, x, None, mean, rstd)
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    us = 2.0 ** -8 if dtype == torch.bfloat16 else U
    for got, terms in ((gb, g.double()), (gg, g.double() * xh)):
        want, size = terms.sum(0), terms.abs().sum(0)
        bound = (128 + 44) * U * size
        assert bool(((got.double() - want).abs() <= bound + us * (want.abs() + bound)).all())
