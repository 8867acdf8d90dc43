"""GPU tests of causal attention (zr_attention_fwd / zr_attention_bwd) against
64 bits (attn64.py has the definition and the bounds)."""
import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr
from attn64 import check, reference, run

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(lead, h, kv, d, dtype, seed=1, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randn(*lead, h, d, generator=g, device="cuda") * size
    k = torch.randn(*lead, kv, d, generator=g, device="cuda") + 0.5 * torch.randn(kv, d, generator=g, device="cuda")
    v, go = torch.randn(*lead, kv, d, generator=g, device="cuda"), torch.randn(*lead, h, d, generator=g, device="cuda")
    return [x.to(dtype) for x in (q, k, v, go)]


def packed(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).int()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513, 1100])
def test_lengths(t, d, dtype):
    q, k, v, go = make((2, t), 2, 2, d, dtype)
    run(zr, q, k, v, go=go)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [1, 3, 8, 16, 40, 72, 80, 96, 104, 120, 33, 130, 192, 256])
def test_head_sizes(d, dtype):
    q, k, v, go = make((1, 150), 2, 1, d, dtype)
    run(zr, q, k, v, go=go)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("h,kv", [(1, 1), (4, 1), (6, 2), (6, 3), (5, 5), (12, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_grouped_heads(h, kv, d, dtype):
    q, k, v, go = make((1, 200), h, kv, d, dtype)
    run(zr, q, k, v, go=go)


@pytest.mark.parametrize("d", [64, 81, 128])
@pytest.mark.parametrize("lengths", [None, [1, 4100, 0, 129, 255, 700, 30]])
def test_shares_of_a_rows_keys(lengths, d):
    """Few heads and long sequences: a pair of query tiles' keys are worked on in shares, some of them empty."""
    t = sum(lengths) if lengths else 4133
    lead = (t,) if lengths else (1, t)
    q, k, v, go = make(lead, 1, 1, d, BF16, size=2.0)
    off = packed(lengths) if lengths else None
    out, lse, *_ = run(zr, q, k, v, offsets=off, go=go)
    again, _, low = zr.zr_attention_fwd(q, k, v, None, off, keep_lse=False)
    assert torch.equal(out, again) and low is None
    wide = torch.full((*q.shape[:-1], d + 3), 7.0, device="cuda", dtype=BF16)
    zr.zr_attention_fwd(q, k, v, None, off, out=wide[..., 2:d + 2])
    assert torch.equal(wide[..., 2:d + 2], out) and bool((wide[..., :2] == 7).all()) and bool((wide[..., d + 2:] == 7).all())


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lengths", [None, [1, 700, 0, 129, 255], [30] * 40])
def test_shares_of_a_key_tile(lengths, d):
    """Few key tiles for the GPU: each is worked on in shares, some of them empty."""
    t = sum(lengths) if lengths else 1100
    lead = (t,) if lengths else (1, t)
    q, k, v, go = make(lead, 8, 1, d, BF16)
    off = packed(lengths) if lengths else None
    full = run(zr, q, k, v, offsets=off, go=go)
    out, lse, low = zr.zr_attention_fwd(q, k, v, None, off, keep_low=True)
    gk = zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off, want=(False, True, False))[1]
    assert torch.equal(gk, full[3])
    if lengths:  # rows in no sequence stay as they are
        off = off[:-1].contiguous()
        grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
        zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off, grads=grads)
        assert all(bool((x[int(off[-1]):] == 7).all()) for x in grads) and torch.equal(grads[1][:int(off[-1])], full[3][:int(off[-1])])


LENGTHS = [[5, 1, 17, 64], [128, 128], [1] * 40, [129, 0, 0, 255, 1, 300], [1000], [0, 0, 7], [64, 63, 65, 127, 128, 129, 2, 256, 257]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda s: "-".join(map(str, s))[:24])
def test_packed(lengths, d, dtype):
    q, k, v, go = make((sum(lengths),), 4, 2, d, dtype)
    run(zr, q, k, v, offsets=packed(lengths), go=go)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(d, dtype):
    """More than a warp's worth of borders."""
    lengths = [(i * 37) % 90 for i in range(150)]
    q, k, v, go = make((sum(lengths),), 2, 1, d, dtype)
    run(zr, q, k, v, offsets=packed(lengths), go=go)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_in_no_sequence(d, dtype):
    """Rows before the first and behind the last sequence hold NaN and infinity, and stay as they were."""
    lengths, first, tail = [70, 130, 1], 9, 150
    n = first + sum(lengths) + tail
    q, k, v, go = make((n,), 2, 2, d, dtype)
    off = packed(lengths) + first
    want = reference(q, k, v, d ** -0.5, off, go)
    for i, x in enumerate((q, k, v, go)):
        x[:first] = (float("nan"), float("inf"), float("nan"), float("-inf"))[i]
        x[n - tail:] = (float("inf"), float("nan"), float("inf"), float("nan"))[i]
    out, lse = torch.full_like(q, 7.0), None
    out, lse, low = zr.zr_attention_fwd(q, k, v, None, off, out=out, keep_low=True)
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off, grads=grads)
    check(lse, want["lse"])
    for x, name in zip((out, *grads), ("out", "gq", "gk", "gv")):
        check(x, want[name])
        assert bool((x[:first] == 7).all()) and bool((x[n - tail:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_another_sequences_nan_stays_there(d, dtype):
    lengths = [100, 90, 200]
    q, k, v, go = make((sum(lengths),), 2, 2, d, dtype)
    off = packed(lengths)
    want = reference(q, k, v, d ** -0.5, off, go)
    mid = slice(100, 190)
    for x in (q, k, v, go):
        x[mid] = float("nan")
    out, lse, low = zr.zr_attention_fwd(q, k, v, None, off, keep_low=True)
    grads = zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off)
    for x, name in zip((out, lse, *grads), ("out", "lse", "gq", "gk", "gv")):
        for part in (slice(0, 100), slice(190, 390)):
            check(x[part], tuple(y[part] for y in want[name]))
        assert bool(torch.isnan(x[mid]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0.0, 8.0, 40.0])
def test_flat_and_peaked_rows(size, d, dtype):
    """All scores equal; rows whose weight is almost all on one token, whose own gradient is a small difference."""
    q, k, v, go = make((1, 300), 2, 2, d, dtype, size=size)
    run(zr, q, k, v, go=go)
    run(zr, q, k, v, go=go, low=False)


def test_peaked_rows_keep_their_gradient():
    """One token has all but 2^-9 of each row's weight: ds is a difference of two numbers that agree to 2^-9.  With low,
    delta is held to 2^-16 of the sum, so grad_q's error stays below 2^-16 * 2 / 2^-9 = 2^-6 of its size plus the operands' 2^-8."""
    t, d = 256, 64
    g = torch.Generator("cuda").manual_seed(4)
    k = torch.randn(t, 1, d, generator=g, device="cuda").bfloat16()
    q = torch.zeros(t, 1, d, device="cuda")
    q[:] = 14.0 * k[:1].float() / k[:1].float().norm() ** 2 * 8  # a score of 14 at token 0
    q = q.bfloat16()
    v, go = (torch.randn(t, 1, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    want = reference(q, k, v, d ** -0.5, None, go)["gq"][0]
    out, lse, low = zr.zr_attention_fwd(q, k, v, keep_low=True)
    gq = zr.zr_attention_bwd(go, q, k, v, out, lse, low, want=(True, False, False))[0]
    assert float((gq[1:].double() - want[1:]).norm() / want[1:].norm()) < 2.0 ** -6 + 2.0 ** -8


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(d, dtype):
    b, t, h, kv = 2, 140, 4, 2
    q, k, v, go = make((b, t), h, kv, d, dtype)
    want = reference(q, k, v, 0.11, None, go)

    def same(q, k, v, go, grads):
        out, lse, low = zr.zr_attention_fwd(q, k, v, 0.11, keep_low=True)
        check(out, want["out"])
        check(lse, want["lse"])
        got = zr.zr_attention_bwd(go, q, k, v, out, lse, low, 0.11, grads=grads)
        for x, n in zip(got, ("gq", "gk", "gv")):
            check(x, want[n])

    qkv = torch.cat([q, k, v], 2)  # one projection's rows, and gradients into the same layout
    grad = torch.full_like(qkv, 5.0)
    same(*qkv.split([h, kv, kv], 2), go, grad.split([h, kv, kv], 2))
    assert not bool((grad == 5).all(-1).any())
    first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v, go)]  # heads first
    same(*first, [torch.empty_like(x) for x in first[:3]])
    odd = []
    for x in (q, k, v, go):  # odd addresses, rows an odd number of elements apart
        wide = torch.zeros(b, t, x.shape[2], d + 1, device="cuda", dtype=dtype)
        wide[..., 1:] = x
        odd.append(wide[..., 1:])
    same(*odd, [torch.empty(b, t, x.shape[2], d + 1, device="cuda", dtype=dtype)[..., 1:] for x in odd[:3]])
    same(q, k, v, torch.stack([go, go], -1)[..., 0], (None,) * 3)  # every other element
    ones = go[:1, :1].expand(b, t, h, d)  # a broadcast gradient
    w2 = reference(q, k, v, 0.11, None, ones)
    out, lse, low = zr.zr_attention_fwd(q, k, v, 0.11, keep_low=True)
    for x, n in zip(zr.zr_attention_bwd(ones, q, k, v, out, lse, low, 0.11), ("gq", "gk", "gv")):
        check(x, w2[n])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_partial_wants_and_scales(d, dtype):
    q, k, v, go = make((1, 130), 2, 1, d, dtype)
    full = run(zr, q, k, v, 0.3, go=go)
    run(zr, q, k, v, 0.0, go=go)
    run(zr, q, k, v, -0.2, go=go)
    out, lse, low = zr.zr_attention_fwd(q, k, v, 0.3, keep_low=True)
    for want in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 0, 1)):
        got = zr.zr_attention_bwd(go, q, k, v, out, lse, low, 0.3, want=want)
        for w, x, y in zip(want, got, full[2:]):
            assert (x is not None and torch.equal(x, y)) if w else x is None
    assert zr.zr_attention_fwd(q, k, v, 0.3, keep_lse=False)[1:] == (None, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_reproducible_on_streams_and_in_graphs(d, dtype):
    lengths = [300, 5, 511, 1]
    q, k, v, go = make((sum(lengths),), 4, 2, d, dtype)
    off = packed(lengths)

    def step():
        out, lse, low = zr.zr_attention_fwd(q, k, v, None, off, keep_low=True)
        return out, lse, *zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off)

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
        mine = step()
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, other, mine))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = step()
        graphs.append((g, got))
    off.copy_(packed([1, 511, 5, 300]))  # the borders are read when the kernels run
    for g, _ in graphs:
        g.replay()
    want = reference(q, k, v, d ** -0.5, off, go)
    for _, got in graphs:
        for x, n in zip(got, ("out", "lse", "gq", "gk", "gv")):
            check(x, want[n])


@pytest.mark.parametrize("d", [64, 128])
def test_differences(d):
    """The gradients against central differences of the forward in binary32: f = sum of c * out.  A score moves by h times a unit direction;
    f's own error (attn64's bound of out) over h, and the third derivative's h^2, bound the difference."""
    t, h = 70, 2.0 ** -6
    q, k, v, c = make((t,), 2, 1, d, F32, seed=9)
    out, lse, low = zr.zr_attention_fwd(q, k, v)
    grads = zr.zr_attention_bwd(c, q, k, v, out, lse)
    for i, g in enumerate(grads):
        args = [q, k, v]
        u = torch.randn_like(args[i])
        u /= u.norm()
        f = []
        for s in (h, -h):
            moved = [x + s * u if j == i else x for j, x in enumerate(args)]
            f.append(float((zr.zr_attention_fwd(*moved)[0].double() * c.double()).sum()))
        rough = float((reference(q, k, v, d ** -0.5)["out"][1] * c.double().abs()).sum())
        want = float((g.double() * u.double()).sum())
        curve = h ** 2 * float(c.double().abs().sum() * v.abs().max()) * d ** -1.0
        assert abs((f[0] - f[1]) / (2 * h) - want) <= rough / h + curve, i


def test_empty():
    q, k, v, go = make((2, 0), 2, 1, 64, BF16)
    out, lse, low = zr.zr_attention_fwd(q, k, v, keep_low=True)
    assert out.shape == q.shape and lse.shape == (2, 0, 2)
    assert [tuple(x.shape) for x in zr.zr_attention_bwd(go, q, k, v, out, lse, low)] == [tuple(x.shape) for x in (q, k, v)]
    q, k, v, go = make((10,), 2, 1, 64, BF16)
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    zr.zr_attention_fwd(q, k, v, None, none, out=out)
    assert bool((out == 3).all())


@pytest.mark.parametrize("borders", [[0, -5, 30, 30, 99999], [50, 20, 60], [-2147483648, 2147483647]])
@pytest.mark.parametrize("d", [64, 128])
def test_borders_outside_are_cut(borders, d):
    """Borders out of range or out of order: results of sequences that are in order are right, nothing faults."""
    q, k, v, go = make((60,), 2, 1, d, BF16)
    off = torch.tensor(borders, dtype=torch.int32, device="cuda")
    out, lse, low = zr.zr_attention_fwd(q, k, v, None, off, keep_low=True)
    zr.zr_attention_bwd(go, q, k, v, out, lse, low, None, off)
    torch.cuda.synchronize()
    if borders[0] < 0:
        check(out, reference(q, k, v, d ** -0.5)["out"])
