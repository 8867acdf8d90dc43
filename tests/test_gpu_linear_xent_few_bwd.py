"""GPU tests of the linear head's cross entropy: the bfloat16 backward of up to
128 rows rounds nothing but its results to bfloat16.

u = 2^-24.  A logit of D terms is off by (D / 16 + 16) 2u of the sum of its
terms' sizes, lse by the row's largest such error and 2^-21 + 2u (|l| + |lse|)
+ 64u, G by p times both and the exponential's 2^-21 + 2u (|l| + |lse|), and by
2^-16 of itself for the parts it is held in.  The products over K terms add
(K / 16 + 80) 2u of the sum of sizes, and the result is rounded once, 2^-8.
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


@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("N,V,D", [(1, 5000, 512), (1, 33, 72), (2, 700, 1000), (7, 3000, 264), (64, 1501, 1280),
                                   (100, 20000, 128), (128, 257, 768), (128, 2048, 64)])
def test_only_the_results_are_rounded(N, V, D, reduction):
    g = torch.Generator("cuda").manual_seed(N + V + D)
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = (torch.randn(N, D, generator=g, device="cuda") +
         torch.rand(N, 1, generator=g, device="cuda") * 8 * w[y].float()).bfloat16()
    grad = torch.rand(N if reduction == "none" else (), generator=g, device="cuda") + 0.5
    _, lse = zr.zr_linear_xent_fwd(x, w, y, reduction)
    got = zr.zr_linear_xent_bwd(grad, x, w, y, lse, reduction)
    X, W = x.double(), w.double()
    l = X @ W.t()
    lerr = (D / 16 + 16) * 2 * U * (X.abs() @ W.abs().t())
    z = torch.logsumexp(l, 1, keepdim=True)
    turn = 2.0 ** -21 + 2 * U * (l.abs().max(1, keepdim=True).values + z.abs())
    c = (grad.double() if reduction == "none" else (grad.double() / N).expand(N))[:, None]
    p = torch.exp(l - z)
    G = p.clone()
    G[torch.arange(N), y] -= 1
    gerr = c * (p * (lerr + lerr.max(1, keepdim=True).values + 2 * turn + 64 * U) + 2.0 ** -16 * G.abs())
    G *= c
    for name, a, want, e in (
            ("grad_x", got[0], G @ W, gerr @ W.abs() + (V / 16 + 80) * 2 * U * (G.abs() @ W.abs())),
            ("grad_w", got[1], G.t() @ X, gerr.t() @ X.abs() + (N / 16 + 80) * 2 * U * (G.abs().t() @ X.abs()))):
        bound = e + 2.0 ** -8 * (want.abs() + e) + 1e-38
        bad = (a.double() - want).abs() > bound
        assert not bad.any(), (name, int(bad.sum()), float(((a.double() - want).abs() / bound).max()))
