"""GPU tests of the linear head's cross entropy on rows that are learnt: the
label's probability p is within 1e-3 of 1, so its element of G = p - [label]
is a small difference, through the C ABI against the definition in 64 bits.

``learnt`` builds rows of positive terms (the worst case for sums that
truncate) whose label logit is 20 and whose other logits are 6 to 8, and ends
each row in a marker column that is 1 in that row alone and 0 in every row of
w: the logits do not see it, and column n of grad_w is row n of G itself.
"""
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


def learnt(N, D, dtype, V=64):
    """x [N, D + 256], w [V, D + 256], labels, and G [N, V] in 64 bits."""
    g = torch.Generator("cuda").manual_seed(D + N)
    x = torch.zeros(N, D + 256, device="cuda")
    x[:, :D] = torch.rand(N, D, generator=g, device="cuda") / 2 + 0.5
    level = torch.rand(V, generator=g, device="cuda") * 2 + 6
    level[1] = 20
    w = torch.zeros(V, D + 256, device="cuda")
    w[:, :D] = (level / x[:, :D].sum(1).mean())[:, None] * (torch.rand(V, D, generator=g, device="cuda") + 0.5)
    x[torch.arange(N), D + torch.arange(N)] = 1
    x, w = x.to(dtype), w.to(dtype)
    G = torch.softmax(x.double() @ w.double().t(), 1)
    G[:, 1] = -(G[:, :1].sum(1) + G[:, 2:].sum(1))
    assert float(G[:, 1].min()) > -1e-3
    return x, w, torch.ones(N, dtype=torch.int64, device="cuda"), G


def gradient(x, w, y):
    """Row n of G as the backward has it, from the marker columns."""
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    _, gw = zr.zr_linear_xent_bwd(torch.ones(len(x), device="cuda"), x, w, y, lse, "none")
    D = x.shape[1] - 256
    return gw[:, D:D + len(x)].t().double()


@pytest.mark.parametrize("D", [1024, 2048, 4096, 8192, 16384 - 256])
def test_long_rows_match_the_forward(D):
    """bfloat16 rows on the tensor cores, whatever their length.  An error
    that logits and lse share scales G; what they do not share is added to p:
    lse's rounding and those of the exponentials' arguments, 4u (|l| + |lse|),
    the exponentials themselves, 2^-20, and 64 additions of positive terms.
    Two roundings to bfloat16, of G and of the result."""
    x, w, y, G = learnt(200, D, torch.bfloat16)
    shared = 20 * (64 * 2 + D / 1024 + 16) * U      # 64 truncating steps to an accumulation
    bound = (2.0 ** -8 + 2 ** -16 + shared) * G.abs() + 2.0 ** -20 + (4 * 40 + 64) * U
    err = (gradient(x, w, y) - G).abs()
    assert (err[:, 1] <= bound[:, 1]).all(), (D, float((err[:, 1] / bound[:, 1]).max()))
