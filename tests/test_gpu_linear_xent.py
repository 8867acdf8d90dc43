"""GPU tests of the linear head's cross entropy (zr_linear_xent_fwd /
zr_linear_xent_bwd) against its definition in 64 bits, through the C ABI.

Tolerances, u = 2^-24.  A = sum |x_d w_d| of a logit.
* A product of K terms accumulates in binary32, 16 terms to a step; each step
  may lose one unit in the last place of the running sum (2u): (K / 16 + 16)
  2u A.  Binary32 tensors take six products instead of one, and the parts
  leave out 4u A.  Call this eps(K) A.
* lse: the largest logit error of the row; the exponentials are good to 2^-21
  and their arguments, l and the maximum, are rounded once each: 2u (|l| +
  |lse|); at most 400 additions of positive terms, 32 at a time: 64u.
* loss: lse's and the label's logit errors, and one rounding of each.
* G = c (p - [label]): p times (the logit's, lse's and the exponential's
  errors); stored in bfloat16 (2^-8 |G|), or in three parts (4u |G|).
* gradients: G's error against |W| (|X|), eps(K) of the sum of |G W|, the
  piecewise sums (2u per piece), one rounding to the storage type.
"""
import numpy as np
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


def eps(K, dtype):
    return (6 * K / 16 + 16) * 2 * U + 4 * U if dtype == torch.float32 else (K / 16 + 16) * 2 * U


def close(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.numel(),
                           float(((got - want).abs() / bound).nan_to_num(1e9).max()))


class Ref:
    """The definition in 64 bits, with the error bounds above."""

    def __init__(self, x, w, labels, reduction="mean", grad_loss=None):
        self.dtype, D = x.dtype, w.shape[1]
        X, W, y = x.double().reshape(-1, D), w.double(), labels.reshape(-1).long()
        V = W.shape[0]
        l = X @ W.t()
        A = X.abs() @ W.abs().t()
        self.valid = y != IGN
        safe = torch.where(self.valid, y, torch.zeros_like(y))
        lerr = eps(D, self.dtype) * A
        self.lse = torch.logsumexp(l, 1)
        top = l.abs().max(1).values
        self.lse_err = lerr.max(1).values + 2.0 ** -21 + 2 * U * (top + self.lse.abs()) + 64 * U
        at = l.gather(1, safe[:, None])[:, 0]
        at_err = lerr.gather(1, safe[:, None])[:, 0]
        zero = torch.zeros_like(at)
        self.rows = torch.where(self.valid, self.lse - at, zero)
        self.rows_err = torch.where(self.valid, self.lse_err + at_err + 2 * U * (self.lse.abs() + at.abs()), zero)
        n = int(self.valid.sum())
        self.count = n
        div = max(n, 1) if reduction == "mean" else 1
        self.loss, self.loss_err = self.rows.sum() / div, (self.rows_err + 4 * U * self.rows.abs()).sum() / div
        if reduction == "none":
            self.loss, self.loss_err = self.rows, self.rows_err
        if grad_loss is None:
            return
        c = grad_loss.double().reshape(-1) / (n if reduction == "mean" and n else 1)
        c = torch.where(self.valid, c.expand(len(y)), zero)
        p = torch.exp(l - self.lse[:, None])
        G = p.clone()
        G[torch.arange(len(y)), safe] -= 1
        G *= c[:, None]
        gerr = c.abs()[:, None] * p * (lerr + self.lse_err[:, None] + 2.0 ** -21 + 2 * U * (l.abs() + self.lse.abs()[:, None]))
        gerr += G.abs() * (2.0 ** -8 if self.dtype == torch.bfloat16 else 4 * U) + 4 * U * c.abs()[:, None] * p
        self.G, self.gerr, self.X, self.W = G, gerr, X, W
        us = 2.0 ** -8 if self.dtype == torch.bfloat16 else U
        self.gx, self.gw = G @ W, G.t() @ X
        e = gerr @ W.abs() + (eps(V, self.dtype) + 64 * U) * (G.abs() @ W.abs())
        self.gx_err = e + us * (self.gx.abs() + e) + 1e-38
        e = gerr.t() @ X.abs() + eps(len(y), self.dtype) * (G.abs().t() @ X.abs())
        self.gw_err = e + us * (self.gw.abs() + e) + 1e-38


def make(seed, N, V, D, dtype, ignored=0.1):
    g = torch.Generator("cuda").manual_seed(seed)
    w = (torch.randn(V, D, generator=g, device="cuda") / D ** 0.5).to(dtype)
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    x = (torch.randn(N, D, generator=g, device="cuda") +
         torch.rand(N, 1, generator=g, device="cuda") * 8 * w[y].float()).to(dtype)
    y = torch.where(torch.rand(N, generator=g, device="cuda") < ignored, torch.full_like(y, IGN), y)
    return x, w, y


def check(x, w, y, reduction="mean", grad=None, want=(True, True)):
    lead = x.shape[:-1]
    if grad is None:
        grad = torch.rand(lead if reduction == "none" else (), device="cuda") + 0.5
    ref = Ref(x, w, y, reduction, grad)
    loss, lse = zr.zr_linear_xent_fwd(x, w, y, reduction, IGN)
    close(lse.reshape(-1), ref.lse, ref.lse_err, "lse")
    close(loss.reshape(-1) if reduction == "none" else loss, ref.loss, ref.loss_err + 1e-38, "loss")
    gx, gw = zr.zr_linear_xent_bwd(grad, x, w, y, lse, reduction, IGN, want=want)
    assert (gx is not None, gw is not None) == tuple(want)
    if gx is not None:
        close(gx.reshape(-1, x.shape[-1]), ref.gx, ref.gx_err, "grad_x")
        assert not gx.reshape(-1, x.shape[-1])[~ref.valid].any()
    if gw is not None:
        close(gw, ref.gw, ref.gw_err, "grad_w")
    return loss, lse, gx, gw


SIZES = [(128, 256, 64), (1, 1, 1), (1, 2, 3), (1, 300, 64), (2, 5, 8), (7, 64, 17), (33, 33, 33),
         (127, 255, 65), (129, 257, 72), (128, 512, 128), (130, 1000, 200), (256, 256, 256),
         (257, 640, 129), (300, 4099, 96), (1000, 777, 384), (64, 9001, 768), (515, 1030, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V,D", SIZES)
def test_sizes(N, V, D, dtype):
    check(*make(N + V + D, N, V, D, dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
def test_reductions_and_each_gradient_alone(reduction, dtype):
    for N in (37, 700):
        x, w, y = make(N, N, 450, 80, dtype)
        for want in ((True, True), (True, False), (False, True)):
            check(x, w, y, reduction, want=want)
        check(x, w, y.int(), reduction)


@pytest.mark.parametrize("dtype", DTYPES)
def test_layouts(dtype):
    """Leading dims, pitches, odd bases, transposed and expanded operands,
    strided labels."""
    x, w, y = make(3, 420, 333, 96, dtype)
    check(x.view(6, 70, 96), w, y.view(6, 70))
    check(x.view(6, 70, 96).transpose(0, 1), w, y.view(6, 70).t().contiguous())
    wide = torch.randn(420, 200, device="cuda").to(dtype)
    for sl in (slice(0, 96), slice(8, 104), slice(3, 99)):
        check(wide[:, sl], w, y)
    check(x, torch.randn(96, 333, device="cuda").to(dtype).t(), y)
    check(x[:, ::2], w[:, 48:], y)
    check(x[:1].expand(420, 96), w[::3], torch.where(y < 0, y, y % 111))
    check(x[0], w, y[0].clamp(min=0))
    pair = torch.stack((y, y + 1), 1)
    check(x, w, pair[:, 0])
    odd = torch.empty(333 * 96 + 1, dtype=dtype, device="cuda")
    odd[1:] = w.reshape(-1)
    check(x, odd[1:].view(333, 96), y)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_left_out(dtype):
    """Every row ignored; infinities and NaN in ignored rows; labels that are
    no class."""
    x, w, y = make(4, 300, 500, 64, dtype)
    none = torch.full_like(y, IGN)
    loss, lse, gx, gw = check(x, w, none)
    assert float(loss) == 0 and not gx.any() and not gw.any()
    assert float(zr.zr_linear_xent_fwd(x, w, none, "sum", IGN)[0]) == 0
    y[5] = y[200] = y[201] = IGN
    clean = check(x, w, y)
    bad = x.clone()
    bad[5], bad[200], bad[201, 3] = float("nan"), float("inf"), -float("inf")
    loss, lse = zr.zr_linear_xent_fwd(bad, w, y, "mean", IGN)
    g = torch.tensor(0.75, device="cuda")
    got = zr.zr_linear_xent_bwd(g, bad, w, y, lse, "mean", IGN)
    want = zr.zr_linear_xent_bwd(g, x, w, y, clean[1], "mean", IGN)
    assert torch.equal(loss, clean[0])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for label in (500, -1, 2 ** 40):
        z = y.clone()
        z[7] = label
        rows, lse = zr.zr_linear_xent_fwd(x, w, z, "none", IGN)
        assert torch.isnan(rows[7]) and not torch.isnan(rows[:7]).any()
        gx, _ = zr.zr_linear_xent_bwd(torch.ones_like(rows), x, w, z, lse, "none", IGN)
        assert torch.isnan(gx[7]).all() and not torch.isnan(gx[8:]).any()


def test_large_logits():
    """Logits of several hundred: the running maximum keeps exponentials in range."""
    for dtype in DTYPES:
        x, w, y = make(5, 200, 700, 64, dtype, ignored=0)
        check((x.float() * 60).to(dtype), w, y)
        check(-(x.float() * 60).to(dtype), w, y)
        check(torch.zeros_like(x), w, y)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss, step 1e-5 (truncation about
    1e-10 here), against the binary32 gradients."""
    x, w, y = make(6, 9, 23, 16, torch.float32)
    g = torch.tensor(1.0, device="cuda")
    _, lse = zr.zr_linear_xent_fwd(x, w, y, "mean", IGN)
    grads = zr.zr_linear_xent_bwd(g, x, w, y, lse, "mean", IGN)
    for k, got in enumerate(grads):
        base = [x.double(), w.double()]
        for i in range(0, got.numel(), 7):
            v = []
            for s in (1, -1):
                args = [t.clone() for t in base]
                args[k].view(-1)[i] += s * 1e-5
                v.append(float(Ref(args[0], args[1], y).loss))
            d = (v[0] - v[1]) / 2e-5
            assert abs(d - float(got.reshape(-1)[i])) <= 1e-6 * (1 + abs(d)), (k, i)


@pytest.mark.parametrize("dtype", DTYPES)
def test_guard_bands(dtype):
    x, w, y = make(7, 131, 261, 72, dtype)
    loss, lse = zr.zr_linear_xent_fwd(x, w, y, "mean", IGN)
    g = torch.tensor(1.0, device="cuda")
    want = zr.zr_linear_xent_bwd(g, x, w, y, lse, "mean", IGN)
    for off in (0, 1, 8):
        bufs, outs = [], []
        for t in (x, w):
            b = torch.full((8192 + off + t.numel(),), -7.25, dtype=dtype, device="cuda")
            bufs.append(b)
            outs.append(b[4096 + off:4096 + off + t.numel()].view(t.shape))
        ws = torch.full((1 << 22,), 0xAB, dtype=torch.uint8, device="cuda")
        zr.zr_linear_xent_bwd(g, x, w, y, lse, "mean", IGN, grads=outs, workspace=ws)
        for b, o, v in zip(bufs, outs, want):
            assert torch.equal(o, v)
            assert bool((b[:4096 + off] == -7.25).all()) and bool((b[4096 + off + o.numel():] == -7.25).all())


def test_deterministic_empty_other_stream_and_graph():
    x, w, y = make(8, 1030, 2000, 128, torch.bfloat16)
    g = torch.tensor(1.0, device="cuda")

    def step():
        loss, lse = zr.zr_linear_xent_fwd(x, w, y, "mean", IGN)
        return (loss, lse, *zr.zr_linear_xent_bwd(g, x, w, y, lse, "mean", IGN))

    a = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = step()
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(c, step()))
    e = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    ye = torch.empty((0,), dtype=torch.int64, device="cuda")
    for red in ("mean", "sum", "none"):
        loss, lse = zr.zr_linear_xent_fwd(e, w, ye, red, IGN)
        assert lse.shape == (0,) and (float(loss) == 0 if red != "none" else loss.shape == (0,))
        gx, gw = zr.zr_linear_xent_bwd(torch.ones_like(loss), e, w, ye, lse, red, IGN)
        assert gx.shape == (0, 128) and not gw.any()


@pytest.mark.parametrize("dtype,N,V,D", [(torch.bfloat16, 150001, 6007, 40), (torch.float32, 70000, 6007, 40)])
def test_pieces_of_the_vocabulary(dtype, N, V, D):
    """More logits than one piece of the workspace holds: the gradient of x is
    summed over pieces.  Rows are checked in samples, grad_w by its columns."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40e9:
        pytest.skip("needs 40 GB")
    x, w, y = make(9, N, V, D, dtype)
    loss, lse = zr.zr_linear_xent_fwd(x, w, y, "mean", IGN)
    grad = torch.tensor(float(N), device="cuda")
    gx, gw = zr.zr_linear_xent_bwd(grad, x, w, y, lse, "mean", IGN)
    count = int((y != IGN).sum())
    gw_ref = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    gw_err = torch.zeros_like(gw_ref)
    total = 0.0
    for at in range(0, N, 8192):
        r = Ref(x[at:at + 8192], w, y[at:at + 8192], "sum", grad / count)
        close(lse[at:at + 8192], r.lse, r.lse_err, "lse")
        close(gx[at:at + 8192], r.gx, r.gx_err, "grad_x")
        total += float(r.rows.sum())
        gw_ref += r.gw
        gw_err += r.gerr.t() @ r.X.abs() + eps(N, dtype) * (r.G.abs().t() @ r.X.abs())
    us = 2.0 ** -8 if dtype == torch.bfloat16 else U
    close(gw, gw_ref, gw_err + us * (gw_ref.abs() + gw_err), "grad_w")
    assert abs(float(loss) - total / count) <= 1e-4 * total / count


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V,D", [(1, 40000, 72), (40, 20000, 65), (300, 9001, 200), (129, 33000, 64), (2500, 130, 384),
                                   (9000, 65, 130)])
def test_long_sums_in_slices(N, V, D, dtype):
    """Few rows, or few classes: one gradient's sum is cut into slices."""
    x, w, y = make(N + V, N, V, D, dtype)
    for want in ((True, True), (True, False), (False, True)):
        check(x, w, y, "mean", want=want)
    check(x, w, y, "none")
    loss, lse = zr.zr_linear_xent_fwd(x, w, y, "sum", IGN)
    g = torch.tensor(0.5, device="cuda")
    want = zr.zr_linear_xent_bwd(g, x, w, y, lse, "sum", IGN)
    bufs = [torch.full((t.numel() + 17,), -7.25, dtype=dtype, device="cuda") for t in (x, w)]
    outs = [b[1:1 + t.numel()].view(t.shape) for b, t in zip(bufs, (x, w))]
    zr.zr_linear_xent_bwd(g, x, w, y, lse, "sum", IGN, grads=outs)
    for b, o, v in zip(bufs, outs, want):
        assert torch.equal(o, v) and bool((b[:1] == -7.25).all()) and bool((b[1 + o.numel():] == -7.25).all())


def test_slices_over_pieces():
    """Few rows against more classes than one piece of the workspace holds."""
    free, _ = torch.cuda.mem_get_info()
    if free < 40e9:
        pytest.skip("needs 40 GB")
    check(*make(11, 280, 650000, 24, torch.float32))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5])
def test_few_rows(N, dtype):
    """The forward's own path for a handful of rows, and around it."""
    for V, D in ((1, 1), (3, 7), (31, 8), (33, 264), (2500, 768), (1501, 1000), (700, 5000), (40, 12288),
                 (40, 12289)):
        x, w, y = make(V + D, N, V, D, dtype, ignored=0)
        check(x, w, y)
        wide = torch.randn(V, D + 8, device="cuda").to(dtype)
        check(x, wide[:, :D], y, "none")
        check(x, wide[:, 1:D + 1], y, "sum")
        tall = torch.randn(N, 3, D, device="cuda").to(dtype)
        check(tall[:, 1], w, y)
        check(torch.randn(D, N, device="cuda").to(dtype).t(), w, y)
    y[:] = IGN
    assert float(zr.zr_linear_xent_fwd(x, w, y)[0]) == 0


@pytest.mark.parametrize("N", [5, 8, 9, 16, 17])
def test_several_rows(N):
    """binary32 rows in groups of eight, and the first count past them."""
    for V, D in ((1, 1), (33, 264), (2501, 769), (1500, 1000), (40, 6144), (40, 6145)):
        x, w, y = make(V + D + N, N, V, D, torch.float32)
        for reduction in ("mean", "none"):
            check(x, w, y, reduction)
    bad = x.clone()
    bad[4] = float("nan")
    y = y.clamp(min=0)
    rows, _ = zr.zr_linear_xent_fwd(bad, w, y, "none", IGN)
    want, _ = zr.zr_linear_xent_fwd(x, w, y, "none", IGN)
    assert torch.isnan(rows[4]) and torch.equal(rows[:4], want[:4]) and torch.equal(rows[5:], want[5:])


def test_one_row_sums_to_binary32():
    """Long rows of positive terms: the worst case for sums that truncate."""
    for N in (1, 200):
        for D in (64, 2048, 4096, 16384):
            g = torch.Generator("cuda").manual_seed(D)
            x = torch.rand(N, D, generator=g, device="cuda").bfloat16()
            w = torch.rand(3, D, generator=g, device="cuda").bfloat16()
            lse = zr.zr_linear_xent_fwd(x, w, torch.zeros(N, dtype=torch.int64, device="cuda"))[1]
            want = torch.logsumexp(x.double() @ w.double().t(), 1)
            # 128 truncating steps of at most 2u, then a few roundings.
            assert ((lse.double() - want).abs() <= (128 * 2 + D / 2048 + 8) * U * want).all(), (N, D)
