"""GPU tests of the linear head's cross entropy: labels and upstream gradients
that are views give what their copies give, bit for bit."""
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


def views(itype):
    """(labels, a name) of shapes whose rows few- and many-row paths take."""
    g = torch.Generator("cuda").manual_seed(2)
    ids = torch.randint(0, 500, (7, 41), generator=g, device="cuda").to(itype)
    ids[2, 3:9] = -100
    yield ids[:, 1:], "the next token's"
    yield ids[:3, 1:2], "one per row"
    yield ids[1:3, ::3][:, :2], "a pitch and a step"
    yield ids[:, 5].contiguous()[:, None].expand(7, 40), "expanded inside"
    yield ids[3, :30].expand(11, 30), "expanded outside"
    yield torch.randint(0, 500, (4, 6, 9), generator=g, device="cuda").to(itype)[1:, 1:5, 2:], "two pitches"
    yield torch.randint(0, 500, (300, 18), generator=g, device="cuda").to(itype)[:, 1:], "many rows"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("itype", [torch.int64, torch.int32])
def test_labels_are_views(dtype, itype):
    g = torch.Generator("cuda").manual_seed(3)
    for y, what in views(itype):
        for D in (64, 72):
            x = torch.randn(*y.shape, D, generator=g, device="cuda").to(dtype)
            w = torch.randn(500, D, generator=g, device="cuda").to(dtype)
            for reduction in ("mean", "none"):
                grad = torch.rand(y.shape if reduction == "none" else (), generator=g, device="cuda")
                both = []
                for labels in (y, y.contiguous()):
                    loss, lse = zr.zr_linear_xent_fwd(x, w, labels, reduction)
                    both.append((loss, lse, *zr.zr_linear_xent_bwd(grad, x, w, labels, lse, reduction)))
                assert all(torch.equal(a, b) for a, b in zip(*both)), (what, D, reduction)


@pytest.mark.parametrize("N", [3, 200])
def test_upstream_gradient_is_a_view(N):
    """loss.sum()'s gradient is an expanded one; others have a step."""
    g = torch.Generator("cuda").manual_seed(4)
    x, w = torch.randn(N, 64, generator=g, device="cuda"), torch.randn(300, 64, generator=g, device="cuda")
    y = torch.randint(0, 300, (N,), generator=g, device="cuda")
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    for grad in (torch.tensor(0.5, device="cuda").expand(N), torch.rand(2 * N, generator=g, device="cuda")[::2]):
        got = zr.zr_linear_xent_bwd(grad, x, w, y, lse, "none")
        want = zr.zr_linear_xent_bwd(grad.contiguous(), x, w, y, lse, "none")
        assert all(torch.equal(a, b) for a, b in zip(got, want))
