"""GPU tests of the AdamW step (zr_adamw_step, zr_adamw_state).

binary32 states and parameters against the formulas in 64 bits.  Each operation
is one rounding of 2^-24: m = b1 m + c1 g is within 3 * 2^-24 of |b1 m| + |c1 g|
(two products, the sum, and the two factors' rounding: 4); v likewise with g * g once more (5); the update
u = rate * (m / d) takes m's relative error, d's (half of v's, the root's, two roundings and the sum's) and four
of its own, of |b1 m| + |c1 g| in place of |m|: under 16 * 2^-24 of it; the parameter is
rounded once more.  8-bit states are compared bit by bit with a restatement in
numpy of the format in include/zr.h.
"""
import numpy as np
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HOW = dict(lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.05)


def step64(p, g, m, v, t, lr, betas, eps, weight_decay, scale=1.0):
    """The formulas in 64 bits, and the size of m's two terms."""
    b1, b2 = betas
    p, g, m, v = p.double(), g.double() * scale, m.double(), v.double()
    size = b1 * m.abs() + (1 - b1) * g.abs()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    d = (v / (1 - b2 ** t)).sqrt() + eps
    u = lr * m / (1 - b1 ** t) / d
    return p - lr * weight_decay * p - u, m, v, size, lr * size / (1 - b1 ** t) / d + lr * weight_decay * p.abs()


def make(sizes, seed=5, grad=torch.float32, odd=False):
    """Lists of p, g, m, v, copies; odd: views at odd addresses of larger buffers."""
    gen = torch.Generator("cuda").manual_seed(seed)
    n = sum(sizes) + len(sizes)

    def cut(t):
        out, at = [], 1 if odd else 0
        for s in sizes:
            out.append(t[at:at + s] if odd else t[at:at + s].clone())
            at += s + (1 if odd else 0)
        return out

    p = torch.randn(n + 1, generator=gen, device="cuda") * 0.1
    g = torch.randn(n + 1, generator=gen, device="cuda") * torch.exp(torch.randn(n + 1, generator=gen, device="cuda") * 2 - 4)
    v = g * g * (torch.rand(n + 1, generator=gen, device="cuda") + 0.2)
    m = v.sqrt() * torch.randn(n + 1, generator=gen, device="cuda") * 0.3
    return [cut(x) for x in (p, g.to(grad), m, v, torch.empty(n + 1, dtype=torch.bfloat16, device="cuda"))]


SIZES = [[1], [255, 256, 257], [4096, 1, 2049, 0, 30000], [7] * 41, [1000 + i for i in range(403)]]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_states_of_32_bits(sizes, grad, odd):
    ps, gs, ms, vs, cs = make(sizes, grad=grad, odd=odd)
    want = [step64(*x, 3, **HOW) for x in zip(ps, gs, ms, vs)]
    old = [p.clone() for p in ps]
    kept = [g.clone() for g in gs]
    zr.zr_adamw_step(ps, gs, ms, vs, 3, HOW["lr"], HOW["betas"], HOW["eps"], HOW["weight_decay"], copies=cs)
    for p, g, m, v, c, o, k, (p64, m64, v64, size, us) in zip(ps, gs, ms, vs, cs, old, kept, want):
        assert bool(((m.double() - m64).abs() <= 4 * U * size + 1e-44).all())
        assert bool(((v.double() - v64).abs() <= 5 * U * v64 + 1e-44).all())
        assert bool(((p.double() - p64).abs() <= U * p64.abs() + 17 * U * us).all())
        assert torch.equal(c, p.bfloat16()) and torch.equal(g, k)
        assert p.numel() == 0 or not torch.equal(p, o)


def test_neighbours_untouched():
    """Views with one element between them: those elements keep their values."""
    sizes = [300, 5, 257, 2048]
    buf = [torch.full((sum(sizes) + len(sizes) + 1,), 7.0, device="cuda") for _ in range(4)]
    at, views = 1, [[] for _ in buf]
    for s in sizes:
        for l, b in zip(views, buf):
            l.append(b[at:at + s])
        at += s + 1
    zr.zr_adamw_step(*views, 1, 1e-2)
    gaps = [0]
    for s in sizes:
        gaps.append(gaps[-1] + s + 1)
    for b in buf:
        assert bool((b[gaps] == 7).all())
    assert all(bool((p != 7).all()) for p in views[0])


def philox(counters, tensor, step, seed):
    c = [counters.astype(np.uint64), np.full(len(counters), tensor, np.uint64), np.full(len(counters), step & 0xFFFFFFFF, np.uint64),
         np.full(len(counters), step >> 32, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).reshape(-1)


def value(code, scale, signed):
    """What codes stand for, in 64 bits, from the format's fields."""
    code = code.astype(np.int64)
    mag = code & 127 if signed else code
    e, f = mag >> 3, mag & 7
    top = 14 if signed else 30
    x = np.where(e == 0, f / 8 * 2.0 ** (1 - top), (1 + f / 8) * 2.0 ** (e - top))
    s = np.repeat(scale.astype(np.float64), 256)[:len(code)]
    return np.where(signed & (code > 127), -x, x) * s


def encode(x, words, signed):
    """Codes and scales of binary32 values."""
    code, scale = np.zeros(len(x), np.uint8), np.zeros(-(-len(x) // 256), np.float32)
    top = 14 if signed else 30
    for b in range(len(scale)):
        y = np.abs(x[256 * b:256 * b + 256].astype(np.float64))
        e = max(np.frexp(y.max())[1] - 1, -90) if y.max() > 0 else -90
        scale[b] = 2.0 ** e
        y = y / 2.0 ** e
        w = words[256 * b:256 * b + 256].astype(np.int64)
        r = ((w & 0xFFFF) if signed else (w >> 16)) * 16 + 8
        binade = np.maximum(np.frexp(y)[1] - 1, 1 - top)
        step = 2.0 ** (binade - 3)
        # Below the smallest code's 2^-20 the pattern has no bits: what is left is rounded to it first.
        fine = np.rint(y / step * 2 ** 20)
        n = (fine + r) // 2 ** 20
        c = np.where(n < 8, n, 8 * (binade + top) + n - 8)
        code[256 * b:256 * b + 256] = c.astype(np.uint8) | ((np.signbit(x[256 * b:256 * b + 256]).astype(np.uint8) << 7) if signed else 0)
    return code, scale


def codes(sizes, odd):
    off = 1 if odd else 0
    c = [torch.zeros(s + off, dtype=torch.uint8, device="cuda")[off:] for s in sizes]
    s = [torch.zeros(-(-n // 256), device="cuda") for n in sizes]
    return c, s


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [255, 256, 257], [4096, 1, 2049, 0, 30000], [70] * 41], ids=lambda s: f"{len(s)}x{s[0]}")
def test_states_of_8_bits(sizes, grad, odd):
    ps, _, _, _, cs = make(sizes, odd=odd)
    ms, msc = codes(sizes, odd)
    vs, vsc = codes(sizes, odd)
    seed = 0xFEDCBA9876543210
    for t in (1, 2, 3):
        gs = make(sizes, seed=20 + t, grad=grad, odd=odd)[1]
        host = [[x.cpu().numpy() for x in l] for l in (ms, vs, msc, vsc)]
        g32, p32 = [g.float().cpu().numpy() for g in gs], [p.cpu().numpy() for p in ps]
        old = [p.clone() for p in ps]
        zr.zr_adamw_step(ps, gs, ms, vs, t, HOW["lr"], HOW["betas"], HOW["eps"], HOW["weight_decay"], copies=cs, m_scales=msc, v_scales=vsc, seed=seed)
        mo, vo = zr.zr_adamw_state(ms, vs, msc, vsc)
        f = np.float32
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            m = value(host[0][i], host[2][i], True).astype(f)  # exact: four bits and a power of two
            v = value(host[1][i], host[3][i], False).astype(f)
            _, _, _, _, us = step64(old[i], gs[i], torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda(), t, **HOW)
            p64 = step64(old[i], gs[i], torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda(), t, **HOW)[0]
            assert bool(((ps[i].double() - p64).abs() <= U * p64.abs() + 17 * U * us).all())
            m = f(0.9) * m + f(1 - 0.9) * g32[i]
            v = f(0.99) * v + f(1 - 0.99) * (g32[i] * g32[i])
            words = philox(np.arange(-(-n // 4)), i, t, seed)[:n]
            for x, signed, code, scale, val in ((m, True, ms[i], msc[i], mo[i]), (v, False, vs[i], vsc[i], vo[i])):
                c, s = encode(x, words, signed)
                assert np.array_equal(scale.cpu().numpy(), s)
                assert np.array_equal(code.cpu().numpy(), c)
                assert np.array_equal(val.double().cpu().numpy(), value(c, s, signed))
        assert all(torch.equal(c, p.bfloat16()) for c, p in zip(cs, ps))


def test_rounding_moves_the_mean():
    """v decays by 1 part in 1000 a step, far below its 3-bit mantissa: rounded to nearest it would stand still.  The mean over
    n elements of v after 64 steps of g = 0 is 0.999^64 of the start; an element's relative variance grows by at most
    (step / v) * 0.001 <= 0.125 * 0.001 a step, so the mean's standard deviation is below sqrt(64 * 1.25e-4 / n) = 1.8e-4; five of them."""
    n = 256 * 1024
    p, g, m = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    v = torch.randint(0xB0, 0xF7, (n,), device="cuda").to(torch.uint8)
    v[::256] = 0xF7  # each block's largest keeps its binade
    sc = [torch.ones(n // 256, device="cuda") for _ in range(2)]
    start = zr.zr_adamw_state([m], [v], [sc[0]], [sc[1]])[1][0].double()
    for t in range(1, 65):
        zr.zr_adamw_step([p], [g], [m], [v], t, 1e-3, (0.9, 0.999), m_scales=[sc[0]], v_scales=[sc[1]], seed=9)
    end = zr.zr_adamw_state([m], [v], [sc[0]], [sc[1]])[1][0].double()
    ratio = float((end / start).mean())
    assert abs(ratio - 0.999 ** 64) < 5 * 1.8e-4 + 64 * 2 ** -17, ratio


def test_blocks_that_are_not_finite():
    n = 256 * 4
    p, g = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    g[5], g[256 + 5], g[512 + 5] = float("inf"), float("nan"), 1e30  # 1e30 squared overflows v alone
    ms, vs = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
    a, b = [torch.zeros(4, device="cuda") for _ in range(2)]
    zr.zr_adamw_step([p], [g], [ms], [vs], 1, 1e-3, m_scales=[a], v_scales=[b])
    assert torch.isnan(a).tolist() == [True, True, False, False] and torch.isnan(b).tolist() == [True, True, True, False]
    m, v = zr.zr_adamw_state([ms], [vs], [a], [b])
    assert bool(torch.isnan(m[0][:512]).all()) and bool(torch.isfinite(m[0][512:]).all())
    assert bool(torch.isnan(v[0][:768]).all()) and bool(torch.isfinite(v[0][768:]).all())
    assert bool(torch.isfinite(p[768:]).all()) and bool(torch.isfinite(p[:5]).all())


def test_decay_per_tensor_and_values_from_the_device():
    sizes = [1000, 2000]
    ps, gs, ms, vs, _ = make(sizes)
    rs = [[x.clone() for x in l] for l in (ps, gs, ms, vs)]
    lr, scale = torch.tensor(2e-3, device="cuda"), torch.tensor([0.25], device="cuda")
    count = torch.tensor([6], device="cuda")
    want = [step64(*x, 10, 2e-3, (0.9, 0.99), 1e-8, w, scale=0.25) for x, w in zip(zip(*rs), (0.0, 0.3))]
    zr.zr_adamw_step(ps, gs, ms, vs, 4, 55.0, (0.9, 0.99), 1e-8, [0.0, 0.3], device_step=count, device_lr=lr, grad_scale=scale)
    # The factors come from binary32 here: the logarithms' rounding and expm1's, 4 * 2^-24 of each more.
    for p, m, v, (p64, m64, v64, size, us) in zip(ps, ms, vs, want):
        assert bool(((m.double() - m64).abs() <= 5 * U * size).all()) and bool(((v.double() - v64).abs() <= 7 * U * v64).all())
        assert bool(((p.double() - p64).abs() <= U * p64.abs() + 26 * U * us).all())


def test_captured_step_goes_on():
    sizes = [700, 4096]
    ps, gs, ms, vs, cs = make(sizes)
    rs = [[x.clone() for x in l] for l in (ps, gs, ms, vs)]
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zr.zr_adamw_step(ps, gs, ms, vs, 1, 1e-3, device_step=count, copies=cs)
        count += 1
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for t in (1, 2, 3):
        zr.zr_adamw_step(*rs, t, 1e-3, device_step=torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert all(torch.equal(a, b) for x, y in zip((ps, ms, vs), (rs[0], rs[2], rs[3])) for a, b in zip(x, y))
    assert int(count) == 3 and all(torch.equal(c, p.bfloat16()) for c, p in zip(cs, ps))


def test_other_stream_and_nothing_to_do():
    ps, gs, ms, vs, _ = make([5000])
    want = step64(ps[0], gs[0], ms[0], vs[0], 1, 1e-3, (0.9, 0.999), 1e-8, 0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        zr.zr_adamw_step(ps, gs, ms, vs, 1, 1e-3)
    side.synchronize()
    assert bool(((ps[0].double() - want[0]).abs() <= U * want[0].abs() + 17 * U * want[4]).all())
    zr.zr_adamw_step([], [], [], [], 1, 1e-3)
    e = torch.empty(0, device="cuda")
    zr.zr_adamw_step([e], [e], [e], [e], 1, 1e-3)


def test_refusals_of_the_binding():
    f, b = torch.zeros(300, device="cuda"), torch.zeros(300, dtype=torch.uint8, device="cuda")
    g, m, v = (torch.zeros(300, device="cuda") for _ in range(3))
    with pytest.raises(ValueError):
        zr.zr_adamw_step([f], [g, g], [m], [v], 1, 1e-3)
    with pytest.raises(ValueError):
        zr.zr_adamw_step([f], [g[:-1]], [m], [v], 1, 1e-3)
    with pytest.raises(ValueError):
        zr.zr_adamw_step([f[::2]], [g[:150]], [m[:150]], [v[:150]], 1, 1e-3)
    with pytest.raises(TypeError):
        zr.zr_adamw_step([f.half()], [g], [m], [v], 1, 1e-3)
    with pytest.raises(TypeError):
        zr.zr_adamw_step([f], [g], [b], [b], 1, 1e-3)
    with pytest.raises(ValueError):
        zr.zr_adamw_step([f], [g], [b], [b.clone()], 1, 1e-3, m_scales=[m[:2]])
    with pytest.raises(ValueError):
        zr.zr_adamw_step([f.cpu()], [g], [m], [v], 1, 1e-3)
    for bad in (dict(lr=float("nan")), dict(betas=(1.0, 0.9)), dict(step=0), dict(eps=-1.0), dict(params=[m])):
        with pytest.raises(zr.ZrError):
            zr.zr_adamw_step(**{**dict(params=[f], grads=[g], ms=[m], vs=[v], step=1, lr=1e-3), **bad})
