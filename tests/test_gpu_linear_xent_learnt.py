"""GPU tests of the linear head's cross entropy on rows that are learnt: the
label's probability p is within 2e-3 of 1, so its element of G = p - [label]
is a small difference, through the C ABI against the definition in 64 bits.

``learnt`` builds rows of positive terms (the worst case for sums that
truncate) whose label logit is 20 and whose other logits are 6 to 8 (or lower), and ends
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


def learnt(N, D, dtype, V=64, others=6.0):
    """x [N, D + 256], w [V, D + 256], labels, and G [N, V] in 64 bits."""
    g = torch.Generator("cuda").manual_seed(D + N)
    x = torch.zeros(N, D + 256, device="cuda")
    x[:, :D] = torch.rand(N, D, generator=g, device="cuda") / 2 + 0.5
    level = torch.rand(V, generator=g, device="cuda") * 2 + others
    level[1] = 20
    w = torch.zeros(V, D + 256, device="cuda")
    w[:, :D] = (level / x[:, :D].sum(1).mean())[:, None] * (torch.rand(V, D, generator=g, device="cuda") + 0.5)
    x[torch.arange(N), D + torch.arange(N)] = 1
    x, w = x.to(dtype), w.to(dtype)
    G = torch.softmax(x.double() @ w.double().t(), 1)
    G[:, 1] = -(G[:, :1].sum(1) + G[:, 2:].sum(1))
    assert float(G[:, 1].min()) > -2e-3
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 3, 16, 200])
@pytest.mark.parametrize("D", [512, 1024, 2048])
def test_label_is_as_exact_as_the_others(N, D, dtype):
    """The label's element has no error that is not in proportion to it, few
    rows or many, whatever path the forward took."""
    x, w, y, G = learnt(N, D, dtype)
    err = (gradient(x, w, y) - G).abs()[:, 1]
    assert (err <= proportion(D + 256, dtype) * G[:, 1].abs()).all(), float((err / G[:, 1].abs()).max())


def proportion(D, dtype):
    """Relative error of the label's element, -sum / (sum + p): twice that of
    the exponentials.  Logits of 20 and 8: binary32 adds chunks of 64 terms, 24
    steps of at most 2u each, and D / 64 chunks, parts leave out 4u; bfloat16
    adds 64 steps of 2u and D / 1024 chunks.  Arguments are rounded at 20 at most
    (2u), exponentials good to 2^-22, 128 additions and a few roundings; the
    result's type and G's, three parts or one."""
    if dtype == torch.float32:
        return 28 * (48 + 4 + D / 64) * U + 2 * (40 * U + 2.0 ** -22) + 140 * U
    return 28 * (128 + D / 1024 + 2) * U + 2 * (40 * U + 2.0 ** -22) + 140 * U + 2.0 ** -8 + 2.0 ** -16


def test_label_over_pieces():
    """A vocabulary that the workspace takes in two pieces, the label's first."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40e9:
        pytest.skip("needs 40 GB")
    x, w, y, G = learnt(256, 128, torch.float32, V=700001, others=-2.0)
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    _, gw = zr.zr_linear_xent_bwd(torch.ones(256, device="cuda"), x, w, y, lse, "none")
    err = (gw[1, 128:].double() - G[:, 1]).abs()
    # A row's sum has 700001 / 128 partial sums, added 171 to a lane.
    assert (err <= (proportion(384, torch.float32) + 180 * U) * G[:, 1].abs()).all(), float((err / G[:, 1].abs()).max())


def test_one_row_gradient_norm():
    """The whole binary32 gradient of one to eight rows, some learnt, some not."""
    for N in (1, 2, 8):
        for seed in range(4):
            g = torch.Generator("cuda").manual_seed(seed)
            w = torch.randn(5003, 384, generator=g, device="cuda") / 384 ** 0.5
            y = torch.randint(0, 5003, (N,), generator=g, device="cuda")
            x = torch.randn(N, 384, generator=g, device="cuda") + (9 + 3 * torch.rand(N, 1, generator=g, device="cuda")) * w[y]
            _, lse = zr.zr_linear_xent_fwd(x, w, y)
            got = zr.zr_linear_xent_bwd(torch.ones((), device="cuda"), x, w, y, lse)
            G = torch.softmax(x.double() @ w.double().t(), 1) / N
            G[torch.arange(N), y] -= 1 / N
            for a, b in zip(got, (G @ w.double(), G.t() @ x.double())):
                # Terms of logits of both signs: |x| |w| is about 13 times 20 / 12 of them.
                assert float((a.double() - b).norm() / b.norm()) <= proportion(384, torch.float32), (N, seed)


def test_lse_near_its_maximum():
    """A row's lse where one logit is nearly all of it: l's error, whatever it
    is, is one logit's, so lse - l shows the sum's own error: exponentials of
    2^-22, their sum and logarithm, 8u, and one rounding of lse, u |lse|."""
    for dtype in (torch.float32, torch.bfloat16):
        for level in (20.0, 75.0):
            g = torch.Generator("cuda").manual_seed(int(level))
            x = torch.zeros(4096, 64, device="cuda")
            x[:, 0] = level * (1 + torch.rand(4096, generator=g, device="cuda") / 8)
            w = torch.zeros(300, 64, device="cuda")
            w[7, 0] = 1
            x, w = x.to(dtype), w.to(dtype)
            _, lse = zr.zr_linear_xent_fwd(x, w, torch.full((4096,), 7, device="cuda"), "none")
            want = torch.logsumexp(x.double() @ w.double().t(), 1)
            assert ((lse.double() - want).abs() <= 2.0 ** -22 + 8 * U + U * want).all(), (dtype, level)


def test_bf16_label_over_pieces():
    """A bfloat16 vocabulary in two pieces: the label's element is p - 1 from
    lse, off by lse's rounding (u |lse|), two exponentials of 2^-22, their sums
    and the logits' errors in proportion, besides the roundings to bfloat16."""
    free, _ = torch.cuda.mem_get_info()
    if free < 60e9:
        pytest.skip("needs 60 GB")
    x, w, y, G = learnt(256, 64, torch.bfloat16, V=2100001, others=-4.0)
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "none")
    _, gw = zr.zr_linear_xent_bwd(torch.ones(256, device="cuda"), x, w, y, lse, "none")
    err = (gw[1, 64:].double() - G[:, 1]).abs()
    bound = proportion(320, torch.bfloat16) * G[:, 1].abs() + 20 * U + 2.0 ** -21 + 16 * U
    assert (err <= bound).all(), float((err / bound).max())


def test_long_positive_sums_are_not_short():
    """bfloat16 gradients that sum 100000 positive terms: the mean signed
    relative error over 2048 columns of different size.  8192 terms in one go
    lose 512 truncating steps of 2u at most, their sums in registers 64u; the
    results' own rounding, 0.0017, averages over the columns (5 sigma)."""
    g = torch.Generator("cuda").manual_seed(1)
    N, V, D = 4096, 100000, 2048
    size = torch.rand(D, generator=g, device="cuda") * 1.5 + 0.5
    w = ((torch.rand(V, D, generator=g, device="cuda") + 0.5) * size).bfloat16()
    w[0] = 0.01
    x = (torch.randn(N, D, generator=g, device="cuda") * 0.03).bfloat16()
    y = torch.zeros(N, dtype=torch.int64, device="cuda")
    _, lse = zr.zr_linear_xent_fwd(x, w, y)
    gx, _ = zr.zr_linear_xent_bwd(torch.tensor(float(N), device="cuda"), x, w, y, lse, want=(True, False))
    W = w.double()
    off = []
    for at in range(0, N, 1024):
        G = torch.softmax(x[at:at + 1024].double() @ W.t(), 1)
        G[:, 0] -= 1
        want = G @ W
        off.append(((gx[at:at + 1024].double() - want) / want).mean())
    mean = float(sum(off) / len(off))
    assert abs(mean) <= (512 * 2 + 64) * U + 5 * 0.0017 / D ** 0.5, mean
