"""GPU tests of layer norm (zr_layer_norm_fwd / zr_layer_norm_bwd) against its
definition in 64 bits, through the C ABI.

Tolerances, u = 2^-24 (binary32) and u_s the storage type's unit roundoff
(2^-24, bf16 2^-8).  A row's sums take at most 32 additions per lane (a long
row: D / 1024 + 8), then at most 13 levels, so a sum is within K u sum|terms|,
K = 48 + D / 1024.

* mean: K u mean|x|, and one rounding.
* rstd: the differences carry the mean's error dm, which changes the variance
  by dm^2; its sum K u; half of both relative errors reaches rstd, plus the
  addition of eps, the root and the reciprocal: ((K + 4) u + (dm rstd)^2) rstd.
* y: |gamma| rstd (dm + 2u|x - mu|) + |gamma xh| (rstd's relative error + 3u)
  + 2u|y|, then u_s |y|.
* grad_x, mean and rstd being inputs: xh is within 2u|xh|, each mean within
  (K + 4) u of its absolute terms, a few roundings after:
  rstd (K + 12) u (|q| + mean|q| + |xh| mean|q xh|), then u_s |grad_x|.
* grad_gamma, grad_beta over R rows: a lane adds at most R / 128 + 1 rows, the
  row groups 16 more, the second pass is compensated with a tree of 8:
  (R / 128 + 40) u sum|terms|, then u_s of the value.
"""
import numpy as np
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


def us(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def definition(x, gamma, beta, eps):
    x = x.double().cpu()
    mu = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mu) * rstd
    if gamma is not None:
        y = y * gamma.double().cpu()
    if beta is not None:
        y = y + beta.double().cpu()
    return y, mu, rstd


def check(got, want, bound, what):
    got = got.double().cpu()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((got - want).abs() / bound).nan_to_num(1e9).max()))


def check_fwd(y, mean, rstd, x, gamma, beta, eps):
    wy, mu, rs = definition(x, gamma, beta, eps)
    D = x.shape[-1]
    K = 48 + D / 1024
    xd = x.double().cpu()
    ga = gamma.double().cpu().abs() if gamma is not None else 1.0
    dm = (K + 1) * U * xd.abs().mean(-1, keepdim=True)
    rel = (K + 4) * U + (dm * rs) ** 2
    if mean is not None:
        check(mean, mu[..., 0], dm[..., 0] + 1e-45, "mean")
        check(rstd, rs[..., 0], (rel * rs)[..., 0], "rstd")
    xh = (xd - mu).abs() * rs
    b = ga * (rs * dm + 2 * U * xh) + ga * xh * (rel + 3 * U) + 2 * U * wy.abs()
    check(y, wy, b + us(y.dtype) * (wy.abs() + b) + 1e-40, "y")


def make(gen, rows, D, dtype, shift=0.0):
    x = torch.randn(rows + (D,), generator=gen) * torch.exp(0.5 * torch.randn(D, generator=gen)) + shift
    gamma = torch.rand(D, generator=gen) + 0.5
    beta = 0.1 * torch.randn(D, generator=gen)
    return x.to(dtype).cuda(), gamma.to(dtype).cuda(), beta.to(dtype).cuda()


DIMS = [1, 2, 7, 8, 16, 31, 32, 33, 64, 65, 72, 128, 129, 256, 260, 384, 513, 768, 1000, 1001, 1024,
        1025, 1032, 2048, 2056, 4100, 8192, 8193, 8200, 20000]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", DIMS)
def test_forward(D, dtype):
    gen = torch.Generator().manual_seed(D)
    for rows in ((1,), (2, 3), (37,)):
        x, gamma, beta = make(gen, rows, D, dtype)
        y, mean, rstd = zr.zr_layer_norm_fwd(x, gamma, beta, 1e-5)
        check_fwd(y, mean, rstd, x, gamma, beta, 1e-5)


def check_bwd(gx, gg, gb, g, x, gamma, mean, rstd):
    D = x.shape[-1]
    K = 48 + D / 1024
    gd, xd = g.double().cpu(), x.double().cpu()
    m, r = mean.double().cpu()[..., None], rstd.double().cpu()[..., None]
    ga = gamma.double().cpu() if gamma is not None else torch.ones(D, dtype=torch.float64)
    xh = (xd - m) * r
    q = gd * ga
    if gx is not None:
        want = r * (q - q.mean(-1, keepdim=True) - xh * (q * xh).mean(-1, keepdim=True))
        b = r * (K + 12) * U * (q.abs() + q.abs().mean(-1, keepdim=True) +
                                xh.abs() * (q * xh).abs().mean(-1, keepdim=True))
        check(gx, want, b + us(gx.dtype) * (want.abs() + b) + 1e-40, "grad_x")
    lead = tuple(range(x.dim() - 1))
    rows = x.numel() // D
    for got, terms, what in ((gg, gd * xh, "grad_gamma"), (gb, gd, "grad_beta")):
        if got is None:
            continue
        want = terms.sum(lead) if lead else terms
        mag = terms.abs().sum(lead) if lead else terms.abs()
        b = (rows / 128 + 40) * U * mag
        check(got, want, b + us(got.dtype) * (want.abs() + b) + 1e-40, what)


def stats(x, eps=1e-5):
    xd = x.double()
    mu = xd.mean(-1)
    rstd = 1 / torch.sqrt(((xd - mu[..., None]) ** 2).mean(-1) + eps)
    return mu.float(), rstd.float()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", DIMS)
def test_backward(D, dtype):
    gen = torch.Generator().manual_seed(1000 + D)
    for rows in ((1,), (2, 3), (197,)):
        x, gamma, _ = make(gen, rows, D, dtype)
        g = torch.randn(x.shape, generator=gen).to(dtype).cuda()
        mean, rstd = stats(x)
        gx, gg, gb = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd)
        check_bwd(gx, gg, gb, g, x, gamma, mean, rstd)


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_many_rows_and_each_gradient_alone(dtype):
    gen = torch.Generator().manual_seed(5)
    for rows, D in ((20000, 48), (5000, 768), (3000, 1100), (300, 9000)):
        x, gamma, _ = make(gen, (rows,), D, dtype)
        g = torch.randn(x.shape, generator=gen).to(dtype).cuda()
        mean, rstd = stats(x)
        for want in ((True, True, True), (True, False, False), (False, True, False),
                     (False, False, True), (False, True, True), (True, False, True)):
            got = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd, want=want)
            assert tuple(v is not None for v in got) == want
            check_bwd(*got, g, x, gamma, mean, rstd)


@pytest.mark.parametrize("dtype", DTYPES)
def test_layouts(dtype):
    """Pitches, odd bases, transposed and permuted views, expanded gradients,
    strided outputs, gamma and beta absent or strided."""
    gen = torch.Generator().manual_seed(6)

    def rnd(*s):
        return torch.randn(s, generator=gen).to(dtype).cuda()

    views = [rnd(37, 1024)[:, :1001], rnd(37, 1024)[:, :1000], rnd(37, 1000)[:, 3:903],
             rnd(300, 37).t(), rnd(5, 7, 6, 64).permute(2, 0, 1, 3), rnd(4, 48, 6).permute(2, 0, 1),
             rnd(1, 96).expand(9, 96), rnd(9, 1).expand(9, 40), rnd(2, 3, 4, 2, 3, 2, 3, 24)[:, :, ::2]]
    for x in views:
        D = x.shape[-1]
        for gamma, beta in ((rnd(D), rnd(D)), (None, None), (rnd(2 * D)[::2], None), (None, rnd(D + 1)[1:])):
            y, mean, rstd = zr.zr_layer_norm_fwd(x, gamma, beta, 1e-3)
            check_fwd(y, mean, rstd, x, gamma, beta, 1e-3)
            g = rnd(*x.shape)
            for gg in (g, g[:1].expand(x.shape), g.transpose(0, 1).contiguous().transpose(0, 1)):
                out = zr.zr_layer_norm_bwd(gg, x, gamma, mean, rstd)
                check_bwd(*out, gg, x, gamma, mean, rstd)
    x = views[1]
    store = torch.full((37, 2 * 1000 + 1), -7.25, dtype=dtype, device="cuda")
    y, mean, rstd = zr.zr_layer_norm_fwd(x, out=store[:, 1::2], keep_stats=False)
    assert mean is None and rstd is None
    check_fwd(y, None, None, x, None, None, 1e-5)
    assert torch.all(store[:, ::2] == -7.25)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [7, 40, 768, 1001, 2048, 9000])
def test_in_place_and_guard_bands(D, dtype):
    gen = torch.Generator().manual_seed(7)
    rows, pad = 45, 4096
    x, gamma, beta = make(gen, (rows,), D, dtype)
    ref = zr.zr_layer_norm_fwd(x, gamma, beta)[0]
    for off in (0, 1, 8):
        def banded(n):
            buf = torch.full((2 * pad + off + n,), -7.25, dtype=dtype, device="cuda")
            return buf, buf[pad + off:pad + off + n]

        def intact(buf, n):
            return bool((buf[:pad + off] == -7.25).all()) and bool((buf[pad + off + n:] == -7.25).all())

        buf, flat = banded(rows * D)
        y = flat.view(rows, D)
        y.copy_(x)
        _, mean, rstd = zr.zr_layer_norm_fwd(y, gamma, beta, out=y)
        check_fwd(y, mean, rstd, x, gamma, beta, 1e-5)
        assert intact(buf, rows * D)
        g = torch.randn(x.shape, generator=gen).to(dtype).cuda()
        for alias in ("g", "x"):
            buf, flat = banded(rows * D)
            gx = flat.view(rows, D)
            gx.copy_(g if alias == "g" else x)
            gbuf, gg = banded(D)
            bbuf, gb = banded(D)
            zr.zr_layer_norm_bwd(gx if alias == "g" else g, gx if alias == "x" else x, gamma, mean, rstd,
                                 grads=(gx, gg, gb))
            check_bwd(gx, gg, gb, g, x, gamma, mean, rstd)
            assert intact(buf, rows * D) and intact(gbuf, D) and intact(bbuf, D)
    assert ref.shape == x.shape


def test_bad_rows_stay_alone():
    """A row of infinities or NaN, and a constant row, leave the others as
    they are."""
    gen = torch.Generator().manual_seed(8)
    for D in (24, 768, 1500, 9000):
        x, gamma, beta = make(gen, (19,), D, torch.float32)
        clean = x.clone()
        x[3, 5] = float("nan")
        x[7, 0] = float("inf")
        x[11] = 3.25
        y, mean, rstd = zr.zr_layer_norm_fwd(x, gamma, beta)
        y0 = zr.zr_layer_norm_fwd(clean, gamma, beta)[0]
        keep = torch.ones(19, dtype=torch.bool)
        keep[[3, 7, 11]] = False
        assert torch.equal(y[keep], y0[keep])
        assert torch.isnan(y[3]).all() and torch.isnan(y[7]).all()
        check_fwd(y[11:12], mean[11:12], rstd[11:12], x[11:12], gamma, beta, 1e-5)
        g = torch.randn(x.shape, generator=gen).cuda()
        gx = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd)[0]
        m0, r0 = stats(clean)
        gx0 = zr.zr_layer_norm_bwd(g, clean, gamma, torch.where(keep.cuda(), mean, m0),
                                   torch.where(keep.cuda(), rstd, r0))[0]
        assert torch.equal(gx[keep], gx0[keep])


def test_large_offset():
    """A mean a thousand times the spread: the two-pass variance holds."""
    gen = torch.Generator().manual_seed(9)
    for D in (96, 768, 9000):
        x, gamma, beta = make(gen, (9,), D, torch.float32, shift=1000.0)
        check_fwd(*zr.zr_layer_norm_fwd(x, gamma, beta), x, gamma, beta, 1e-5)


def test_gradient_against_differences():
    """d/dx, d/dgamma, d/dbeta of sum(w * y) by central differences of the
    64-bit definition: step h leaves a truncation error of about h^2 times the
    third derivative (rstd^3-sized here), h = 1e-5."""
    gen = torch.Generator().manual_seed(10)
    x, gamma, beta = make(gen, (3,), 37, torch.float32)
    w = torch.randn(x.shape, generator=gen)
    y, mean, rstd = zr.zr_layer_norm_fwd(x, gamma, beta, 1e-2)
    gx, gg, gb = zr.zr_layer_norm_bwd(w.cuda(), x, gamma, mean, rstd)
    base = [t.double().cpu() for t in (x, gamma, beta)]
    for k, got in enumerate((gx, gg, gb)):
        flat = got.double().cpu().reshape(-1)
        for i in range(0, flat.numel(), 5):
            vals = []
            for s in (1, -1):
                args = [t.clone() for t in base]
                args[k].view(-1)[i] += s * 1e-5
                vals.append(float((w.double() * definition(*args, 1e-2)[0]).sum()))
            diff = (vals[0] - vals[1]) / 2e-5
            assert abs(diff - float(flat[i])) <= 2e-5 * (1 + abs(diff)) * 10, (k, i)


def test_deterministic_empty_and_other_stream():
    gen = torch.Generator().manual_seed(11)
    x, gamma, beta = make(gen, (4001,), 768, torch.bfloat16)
    g = torch.randn(x.shape, generator=gen).to(torch.bfloat16).cuda()
    mean, rstd = stats(x)
    a = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd)
        y2 = zr.zr_layer_norm_fwd(x, gamma, beta)[0]
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert torch.equal(y2, zr.zr_layer_norm_fwd(x, gamma, beta)[0])
    e = torch.empty((0, 768), device="cuda")
    ga = torch.ones(768, device="cuda")
    y, mean, rstd = zr.zr_layer_norm_fwd(e, ga)
    assert y.shape == (0, 768) and mean.shape == (0,)
    gx, gg, gb = zr.zr_layer_norm_bwd(e, e, ga, mean, rstd)
    assert gx.shape == (0, 768) and not gg.any() and not gb.any()


def test_rows_past_32_bit_offsets():
    """65,600 rows with a pitch of 40,000 elements: offsets past 2^31."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12e9:
        pytest.skip("needs 12 GB")
    wide = torch.zeros((65600, 40000), dtype=torch.bfloat16, device="cuda")
    x = wide[:, 39000:39256]
    x.normal_(generator=torch.Generator("cuda").manual_seed(12))
    y, mean, rstd = zr.zr_layer_norm_fwd(x)
    pick = torch.tensor([0, 1, 53686, 53687, 65599], device="cuda")
    check_fwd(y[pick], mean[pick], rstd[pick], x[pick], None, None, 1e-5)
    g = torch.randn((256,), device="cuda").to(torch.bfloat16).expand(65600, 256)
    gx, _, gb = zr.zr_layer_norm_bwd(g, x, None, mean, rstd)
    check_bwd(gx[pick], None, None, g[pick], x[pick], None, mean[pick], rstd[pick])
    want = g[0].double().cpu() * 65600
    check(gb, want, (65600 / 128 + 40) * U * want.abs() + 2.0 ** -8 * want.abs() * 1.01, "grad_beta")


def test_graph_capture():
    gen = torch.Generator().manual_seed(13)
    x, gamma, beta = make(gen, (513,), 384, torch.float32)
    g = torch.randn(x.shape, generator=gen).cuda()
    zr.zr_layer_norm_fwd(x, gamma, beta)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = zr.zr_layer_norm_fwd(x, gamma, beta)
        out = zr.zr_layer_norm_bwd(g, x, gamma, mean, rstd)
    x.copy_(torch.randn(x.shape, generator=gen))
    graph.replay()
    torch.cuda.synchronize()
    check_fwd(y, mean, rstd, x, gamma, beta, 1e-5)
    check_bwd(*out, g, x, gamma, mean, rstd)
