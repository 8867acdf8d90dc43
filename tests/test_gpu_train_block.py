"""The example that runs the training operators together learns its batch, and
the chain's gradients are those of 64-bit autograd."""
import importlib.util
import math
import os

import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_loss_falls(example, dtype):
    losses = example.train(steps=60, dtype=dtype)
    assert all(math.isfinite(v) for v in losses)
    assert abs(losses[0] - math.log(301)) < 0.5       # an untrained model is near uniform
    assert losses[-1] < 0.6 * losses[0]


def test_chain_of_operators_against_autograd():
    """h = r + dropout(f), y = norm(h), loss = xent(y E^T): the operators'
    gradients in binary32 against 64-bit autograd on the same mask.  Each
    gradient passes three operators whose relative errors are below 1e-5 at
    these sizes; the bound is 1e-4 of the gradient's largest element."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator("cuda").manual_seed(2)

    def normal(*s):
        return torch.randn(s, generator=gen, device="cuda")

    N, D, V = 150, 96, 333
    f, r, E = normal(N, D), normal(N, D), normal(V, D) * 0.2
    gamma, beta = normal(D) * 0.1 + 1, normal(D) * 0.1
    y = torch.randint(0, V, (N,), generator=gen, device="cuda")
    y[::7] = -100
    h = zr.zr_dropout_fwd(f, 0.3, 9, 4, residual=r)
    n, mu, rs = zr.zr_layer_norm_fwd(h, gamma, beta)
    loss, lse = zr.zr_linear_xent_fwd(n, E, y)
    gn, gE = zr.zr_linear_xent_bwd(torch.ones((), device="cuda"), n, E, y, lse)
    gh, gg, gb = zr.zr_layer_norm_bwd(gn, h, gamma, mu, rs)
    gf = zr.zr_dropout_bwd(gh, 0.3, 9, 4)
    keep = (zr.zr_dropout_fwd(torch.ones_like(f), 0.3, 9, 4) != 0).double()
    leaves = [t.double().requires_grad_() for t in (f, r, E, gamma, beta)]
    f6, r6, E6, g6, b6 = leaves
    h6 = r6 + keep * f6 / 0.7
    c = h6 - h6.mean(1, keepdim=True)
    n6 = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * g6 + b6
    l6 = torch.nn.functional.cross_entropy(n6 @ E6.t(), y, ignore_index=-100)
    l6.backward()
    l6 = float(l6.detach())
    assert abs(float(loss) - l6) < 1e-5 * l6
    for got, leaf in zip((gf, gh, gE, gg, gb), leaves):
        want = leaf.grad
        assert (got.double() - want).abs().max() <= 1e-4 * want.abs().max()
