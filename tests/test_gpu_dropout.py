"""GPU tests of dropout with a residual (zr_dropout_fwd / zr_dropout_bwd).

The mask is exact: word i mod 4 of Philox4x32-10 at counter offset + i div 4,
restated here in NumPy's unsigned integers and pinned to the paper's published
known answers.  The values are exact too: one binary32 multiplication by the
binary32 scale, one addition, one rounding to the storage type, so every
output is compared bit for bit (any NaN matching any NaN).
"""
import numpy as np
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr
from parity import bitexact

gpu = pytest.mark.gpu
M = 0xFFFFFFFF
DTYPES = [torch.float32, torch.bfloat16]


def philox(c, key, rounds=10):
    """[n, 4] words of [n, 4] counters under a 2-word key."""
    c = [np.asarray(c)[:, i].astype(np.uint64) for i in range(4)]
    k = [key[0], key[1]]
    for r in range(rounds):
        p = c[0] * np.uint64(0xD2511F53)
        q = c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        m = np.uint64(M)
        c = [(q >> s) ^ c[1] ^ np.uint64(k[0]), q & m, (p >> s) ^ c[3] ^ np.uint64(k[1]), p & m]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    return np.stack(c, 1).astype(np.uint64)


def keep_mask(n, p, seed, offset):
    at = [(offset + i) & ((1 << 64) - 1) for i in range((n + 3) // 4)]
    c = np.zeros((len(at), 4), np.uint64)
    c[:, 0] = [a & M for a in at]
    c[:, 1] = [a >> 32 for a in at]
    w = philox(c, (seed & M, (seed >> 32) & M)).reshape(-1)[:n]
    return w >= round(p * 2 ** 32)


def test_generator_known_answers():
    """The known-answer vectors published with Philox4x32-10."""
    c = np.array([[0, 0, 0, 0], [M, M, M, M], [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]])
    keys = [(0, 0), (M, M), (0xA4093822, 0x299F31D0)]
    want = [[0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8],
            [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD],
            [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]]
    for i in range(3):
        assert philox(c[i:i + 1], keys[i])[0].tolist() == want[i]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    zr.build()
    zr.lib()


def expect(x, r, p, seed, offset):
    """The definition, binary32 per operation."""
    keep = torch.from_numpy(keep_mask(x.numel(), p, seed, offset)).view(x.shape)
    scale = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    y = torch.where(keep, x.float().cpu() * torch.tensor(scale), torch.zeros(()))
    if r is not None:
        y = r.float().cpu() + y
    return y.to(x.dtype).float()


def same(got, want, what):
    bitexact(got.float().cpu().numpy(), want.numpy(), what)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 15, 31, 1023, 1024, 4096, 4097, 33333])
def test_lengths(lib, n, dtype):
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=gen).to(dtype).cuda()
    r = torch.randn(n, generator=gen).to(dtype).cuda()
    for p, seed, offset in ((0.2, 1234567890123456789, 7), (0.5, -1 & (2 ** 64 - 1), 2 ** 32 - 2),
                            (0.9, 3, 2 ** 64 - 3), (0.0, 5, 0), (1.0, 5, 0), (1e-12, 8, 9)):
        same(zr.zr_dropout_fwd(x, p, seed, offset, residual=r), expect(x, r, p, seed, offset), (n, p))
        same(zr.zr_dropout_fwd(x, p, seed, offset), expect(x, None, p, seed, offset), (n, p))
        same(zr.zr_dropout_bwd(x, p, seed, offset), expect(x, None, p, seed, offset), (n, p))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_layouts(lib, dtype):
    """The mask follows the row-major index whatever the strides."""
    gen = torch.Generator().manual_seed(3)

    def rnd(*s):
        return torch.randn(s, generator=gen).to(dtype).cuda()

    args = (0.3, 99, 1 << 40)
    for x in (rnd(37, 1024)[:, :1000], rnd(37, 1024)[:, :1001], rnd(37, 64)[:, 1:57], rnd(300, 37).t(),
              rnd(5, 7, 6, 64).permute(2, 0, 1, 3), rnd(9, 1).expand(9, 40), rnd(1, 96).expand(9, 96),
              rnd(2, 3, 4, 2, 3, 2, 3, 24)[:, :, ::2], rnd(1001)[1:], rnd()):
        r = rnd(*x.shape)
        for res in (None, r, r.flip(0).flip(0) if x.dim() else r,
                    r[:1].expand(x.shape) if x.dim() else r):
            same(zr.zr_dropout_fwd(x, *args, residual=res), expect(x, res, *args), (x.shape, x.stride()))
        if x.dim() == 2:
            store = torch.full((x.shape[1], x.shape[0]), -7.25, dtype=dtype, device="cuda")
            zr.zr_dropout_bwd(x, *args, grad_x=store.t())
            same(store.t(), expect(x, None, *args), "transposed out")


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_guard_bands_and_special_values(lib, dtype):
    gen = torch.Generator().manual_seed(4)
    for n in (1, 7, 4096, 5003):
        for off in (0, 1, 8):
            x = torch.randn(n, generator=gen).to(dtype)
            r = torch.randn(n, generator=gen).to(dtype)
            x[:: 3] = float("nan")
            x[1:: 5] = float("inf")
            r[2:: 7] = -float("inf")
            want = expect(x, r, 0.6, 11, 12)
            for alias in ("x", "r"):
                buf = torch.full((8192 + off + n,), -7.25, dtype=dtype, device="cuda")
                t = buf[4096 + off:4096 + off + n]
                t.copy_(x if alias == "x" else r)
                zr.zr_dropout_fwd(t if alias == "x" else x.cuda(), 0.6, 11, 12,
                                  residual=t if alias == "r" else r.cuda(), out=t)
                same(t, want, (n, off, alias))
                assert bool((buf[:4096 + off] == -7.25).all()) and bool((buf[4096 + off + n:] == -7.25).all())
    x = torch.full((64,), float("nan"), dtype=dtype, device="cuda")
    assert not zr.zr_dropout_bwd(x, 1.0, 1).any()  # a dropped NaN leaves nothing


@gpu
def test_backward_is_the_forwards_derivative(lib):
    """The map is linear in x: differences of the forward give the backward."""
    x = torch.zeros(257, device="cuda")
    e = torch.ones(257, device="cuda")
    r = torch.zeros(257, device="cuda")
    d = zr.zr_dropout_fwd(x + e, 0.25, 5, 6, residual=r) - zr.zr_dropout_fwd(x, 0.25, 5, 6, residual=r)
    g = torch.randn(257, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(zr.zr_dropout_bwd(g, 0.25, 5, 6), g * d)


@gpu
def test_large_and_rate(lib):
    """2.2 billion elements: indices past 2^31, and the share that is kept
    (binomial, six standard deviations)."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12e9:
        pytest.skip("needs 12 GB")
    n = (1 << 31) + 100003
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = zr.zr_dropout_fwd(x, 0.2, 77, 13, out=x)
    kept = int((y != 0).sum())
    assert abs(kept - 0.8 * n) <= 6 * (n * 0.16) ** 0.5
    for at in (0, (1 << 31) - 64, n - 64 - (n - 64) % 4):
        want = keep_mask(64, 0.2, 77, 13 + at // 4)
        assert np.array_equal((y[at:at + 64] != 0).cpu().numpy()[:n - at], want[:n - at])


@gpu
def test_graph_replays_draw_new_masks(lib):
    x = torch.ones(4099, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    zr.zr_dropout_fwd(x, 0.5, 21, 4, device_offset=step)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = zr.zr_dropout_fwd(x, 0.5, 21, 4, device_offset=step)
        gx = zr.zr_dropout_bwd(x, 0.5, 21, 4, device_offset=step)
    for at in (0, 1025, 2 ** 40):
        step.fill_(at)
        graph.replay()
        torch.cuda.synchronize()
        same(y, expect(x, None, 0.5, 21, 4 + at), at)
        assert torch.equal(y, gx)


@gpu
def test_other_stream_and_empty(lib):
    x = torch.randn(100003, generator=torch.Generator().manual_seed(2)).cuda()
    a = zr.zr_dropout_fwd(x, 0.1, 1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = zr.zr_dropout_fwd(x, 0.1, 1, 2)
    s.synchronize()
    assert torch.equal(a, b)
    assert zr.zr_dropout_fwd(torch.empty((0, 5), device="cuda"), 0.1, 1).shape == (0, 5)
