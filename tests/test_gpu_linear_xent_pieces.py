"""GPU tests of the linear head's cross entropy: binary32 gradients whose G
comes in several pieces of the vocabulary, against the definition in 64 bits.

u = 2^-24.  A logit is off by lerr = (48 + D / 64 + 8) u of the sum of its terms'
sizes (chunks of 64 terms, 24 steps of 2u), lse by the row's largest such error,
2^-21, 2u (|l| + |lse|) and 64u; an element of G by |G| times what both add up
to, the label's by the row's sum of such errors over p and 200u.  Products over K
terms add (48 + K / 64 + 16) u of the sum of sizes, the pieces and the label's
part 8u.
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
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")
    zr.build()
    zr.lib()


def check(x, w, y, reduction="mean", want=(True, True)):
    N, D = x.shape
    V = w.shape[0]
    g = torch.Generator("cuda").manual_seed(1)
    grad = torch.rand(N if reduction == "none" else (), generator=g, device="cuda") + 0.5
    _, lse = zr.zr_linear_xent_fwd(x, w, y, reduction)
    got = zr.zr_linear_xent_bwd(grad, x, w, y, lse, reduction, want=want)
    used = y >= 0
    safe = y.clamp(min=0)[:, None]
    c = (grad.double().expand(N) / (max(int(used.sum()), 1) if reduction == "mean" else 1)) * used
    X, W = x.double(), w.double()
    refs = [torch.empty(N, D, dtype=torch.float64, device="cuda"), torch.zeros(V, D, dtype=torch.float64, device="cuda")]
    errs = [torch.empty_like(refs[0]), torch.zeros_like(refs[1])]
    for at in range(0, N, 512):
        s = slice(at, at + 512)
        l = X[s] @ W.t()
        z = torch.logsumexp(l, 1, keepdim=True)
        e = (48 + D / 64 + 8) * U * (X[s].abs() @ W.abs().t())
        e += e.max(1, keepdim=True).values + 2.0 ** -20 + 4 * U * (l.abs().max(1, keepdim=True).values + z.abs()) + 128 * U
        G = torch.exp(l - z)
        G.scatter_(1, safe[s], 0)
        e *= G
        rest = G.sum(1, keepdim=True)
        e.scatter_(1, safe[s], 2 * e.sum(1, keepdim=True) + 200 * U * rest)
        G.scatter_(1, safe[s], -rest)
        G *= c[s, None]
        e *= c[s, None]
        refs[0][s], errs[0][s] = G @ W, e @ W.abs() + (48 + V / 64 + 24) * U * (G.abs() @ W.abs())
        refs[1] += G.t() @ X[s]
        errs[1] += e.t() @ X[s].abs() + (48 + N / 64 + 24) * U * (G.abs().t() @ X[s].abs())
    for k, name in enumerate(("grad_x", "grad_w")):
        assert (got[k] is not None) == want[k]
        if want[k]:
            bad = ~((got[k].double() - refs[k]).abs() <= errs[k] + U * refs[k].abs() + 1e-38)
            assert not bad.any(), (name, int(bad.sum()), float(((got[k].double() - refs[k]).abs() / errs[k]).max()))
    if want[0]:
        assert not got[0][~used].any()


def make(N, V, D, seed=2):
    g = torch.Generator("cuda").manual_seed(seed)
    w = torch.randn(V, D, generator=g, device="cuda") / D ** 0.5
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = torch.randn(N, D, generator=g, device="cuda") + torch.rand(N, 1, generator=g, device="cuda") * 12 * w[y]
    y[torch.rand(N, generator=g, device="cuda") < 0.1] = -100
    return x, w, y


@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("want", [(True, True), (True, False), (False, True)])
def test_each_gradient(reduction, want):
    check(*make(3001, 70001, 72), reduction, want)


def test_sizes_and_layouts():
    check(*make(1500, 130001, 300))                       # two blocks of columns, odd rows
    x, w, y = make(4099, 50000, 65)
    check(x, w.t().contiguous().t(), y)                   # transposed weights
    wide = torch.randn(4099, 130, device="cuda")
    check(wide[:, ::2], w, y)                             # strided rows


def test_few_classes_take_all_rows():
    """Every row of one class, or of eight that alternate: long lists to one block."""
    x, w, y = make(4000, 50000, 64)
    check(x, w, torch.full_like(y, 49999))
    check(x, w, torch.arange(4000, device="cuda") % 8 * 3 + 31)
    check(x, w, torch.full_like(y, -100))


def test_repeats_itself():
    x, w, y = make(4000, 50000, 64)
    y = y % 97
    _, lse = zr.zr_linear_xent_fwd(x, w, y)
    one = torch.ones((), device="cuda")
    a = zr.zr_linear_xent_bwd(one, x, w, y, lse)
    b = zr.zr_linear_xent_bwd(one, x, w, y, lse)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_infinite_upstream_gradient():
    """One row's upstream gradient overflowed: its label's row of grad_w is
    infinite with the sign of -x, and rows it has no part in stay finite."""
    x, w, y = make(300, 700001, 8)
    y[5] = 17
    y[torch.arange(300, device="cuda") != 5] = 700000
    grad = torch.ones(300, device="cuda")
    grad[5] = float("inf")
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    gx, gw = zr.zr_linear_xent_bwd(grad, x, w, y, lse, "none")
    assert bool((gw[17] == -x[5].sign() * float("inf")).all())
    assert bool(torch.isfinite(gx[:5]).all()) and bool(torch.isfinite(gx[6:]).all())
