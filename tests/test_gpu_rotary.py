"""GPU tests of rotary positions (zr_rotary_fwd / zr_rotary_bwd) against the
definition in 64 bits.

Bound of one element of the pair (a, b): with c, s within e of the cosine and
sine, |error| <= e (|a| + |b|) m + rounding.  The kernel's angle is within
2^-33 of a turn (the bits below 2^-32 fall away; 2^-31 rad), its rest is rounded to 24 bits
(at most pi/4 * 2^-24), sincospif and the factor m add two roundings of 2^-23 together:
e < 4 * 2^-24 + 2^-30 < 5 * 2^-24.  The two products and the sum add 2 * 2^-24 (|a| + |b|), so 7 * 2^-24 m (|a| + |b|) in
binary32, and half a bf16 step, 2^-8 of the value, where it is stored so.
"""
import math

import pytest
import torch

import broadcast_elementwise_shape_gb300 as zr

pytestmark = pytest.mark.gpu


def rates(part, base=10000.0, factor=1.0, original=None, low=1.0, high=32.0):
    j = torch.arange(part // 2, dtype=torch.float64)
    f = base ** (-2 * j / part)
    if not original:
        return f / factor
    w = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
    return f * (w + (1 - w) / factor)


def reference(x, positions, f, interleaved, magnitude=1.0, back=False):
    """(result, size of what goes into it) in 64 bits."""
    part = 2 * len(f)
    a = (positions.double()[..., None] * f.to(x.device))[..., None, :]
    c, s = magnitude * torch.cos(a), magnitude * torch.sin(a) * (-1 if back else 1)
    x = x.double()
    i, k = (slice(0, part, 2), slice(1, part, 2)) if interleaved else (slice(0, part // 2), slice(part // 2, part))
    y, size = x.clone(), torch.zeros_like(x)
    y[..., i] = x[..., i] * c - x[..., k] * s
    y[..., k] = x[..., k] * c + x[..., i] * s
    size[..., i] = size[..., k] = abs(magnitude) * (x[..., i].abs() + x[..., k].abs())
    return y, size


def check(got, want, size):
    err = (got.double() - want).abs()
    bound = 7 * 2.0 ** -24 * size
    if got.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert bool((err <= bound).all()), float((err - bound).max())


CASES = [  # leading shape, heads, dim, part
    ((1,), 12, 64, 64), ((7,), 3, 64, 64), ((513,), 5, 128, 128), ((2, 33), 4, 64, 32), ((3, 1, 5), 1, 81, 32),
    ((257,), 1, 2, 2), ((65,), 20, 81, 80), ((19,), 2, 520, 512), ((4,), 7, 24, 24), ((100,), 6, 40, 16), ((), 4, 64, 64),
    ((5000,), 1, 16, 16), ((1,), 300, 128, 64),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lead,heads,dim,part", CASES)
def test_against_definition(lead, heads, dim, part, interleaved, dtype):
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randn(*lead, heads, dim, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, lead, generator=g, device="cuda")
    plan = zr.zr_rotary_plan(part, interleaved=interleaved, magnitude=1.25)
    f = rates(part)
    want, size = reference(x, pos, f, interleaved, 1.25)
    check(zr.zr_rotary_fwd(x, plan, pos), want, size)
    want, size = reference(x, pos, f, interleaved, 1.25, back=True)
    check(zr.zr_rotary_bwd(x, plan, pos), want, size)
    # Positions counted by the call, from a start.
    counted = 977 + (torch.arange(lead[-1], device="cuda").expand(lead) if lead else torch.tensor(0, device="cuda"))
    want, size = reference(x, counted, f, interleaved, 1.25)
    check(zr.zr_rotary_fwd(x, plan, start=977), want, size)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_and_negative_positions(dtype):
    x = torch.randn(6, 2, 64, device="cuda").to(dtype)
    pos = torch.tensor([0, -1, -70000, 1 << 24, (1 << 28) + 12345, -(1 << 28)], device="cuda")
    plan, f = zr.zr_rotary_plan(64), rates(64)
    # The rate is kept to 2^-53 of it: at 2^28 turns of the fastest pair that is 2^-25 of a turn, and as much in the
    # reference, which adds 2 * 2^-25 * 2 pi * (1 / (2 pi)) rad = 2^-24 * (|a| + |b|): within the bound's slack of the others.
    want, size = reference(x, pos, f, False)
    check(zr.zr_rotary_fwd(x, plan, pos), want, size * 8 / 7)
    check(zr.zr_rotary_fwd(x, plan, pos.int()), want, size * 8 / 7)
    check(zr.zr_rotary_fwd(x, plan, (pos - 5).int(), start=5), want, size * 8 / 7)


@pytest.mark.parametrize("kw", [dict(factor=4.0), dict(factor=8.0, original=4096), dict(factor=8.0, original=512, low=0.5, high=4.0),
                                dict(base=500000.0), dict(factor=0.5)])
def test_scaled_rates(kw):
    x = torch.randn(300, 2, 96, device="cuda")
    pos = torch.arange(300, device="cuda") * 331
    want, size = reference(x, pos, rates(96, **kw), False)
    check(zr.zr_rotary_fwd(x, zr.zr_rotary_plan(96, **kw), pos), want, size)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts_and_in_place(interleaved, dtype):
    g = torch.Generator("cuda").manual_seed(3)
    plan, f = zr.zr_rotary_plan(64, interleaved=interleaved), rates(64)
    pos = torch.arange(40, device="cuda").expand(3, 40)
    qkv = torch.randn(3, 40, 18, 64, generator=g, device="cuda").to(dtype)
    views = {
        "heads of a projection": qkv[:, :, 6:12],
        "heads first": qkv.transpose(1, 2).contiguous().transpose(1, 2)[:, :, :5],
        "odd base": torch.randn(3 * 40 * 4 * 64 + 1, generator=g, device="cuda").to(dtype)[1:].view(3, 40, 4, 64),
        "strided elements": torch.randn(3, 40, 4, 128, generator=g, device="cuda").to(dtype)[..., ::2],
        "expanded": torch.randn(3, 1, 4, 64, generator=g, device="cuda").to(dtype).expand(3, 40, 4, 64),
    }
    for name, x in views.items():
        want, size = reference(x, pos, f, interleaved)
        check(zr.zr_rotary_fwd(x, plan, pos), want, size)
        if name == "expanded":
            continue
        rest = qkv.clone()
        y = zr.zr_rotary_fwd(x, plan, pos, out=x)
        assert y.data_ptr() == x.data_ptr()
        check(x, want, size)
        if name == "heads of a projection":
            assert torch.equal(qkv[:, :, :6], rest[:, :, :6]) and torch.equal(qkv[:, :, 12:], rest[:, :, 12:])


def test_backward_is_the_transpose():
    """The turn is linear: <y, R x> = <R^T y, x>, in 64 bits of 32-bit results (a sum of n products each within the bound)."""
    x, g = torch.randn(50, 3, 64, device="cuda"), torch.randn(50, 3, 64, device="cuda")
    plan = zr.zr_rotary_plan(48, magnitude=0.7)
    a = (zr.zr_rotary_fwd(x, plan).double() * g.double()).sum()
    b = (zr.zr_rotary_bwd(g, plan).double() * x.double()).sum()
    assert abs(float(a - b)) <= 2 * 7 * 2.0 ** -24 * 2 * float((x.abs().sum(-1) * g.abs().amax(-1)).sum())


def test_infinities_stay_in_their_pair():
    x = torch.randn(4, 2, 64, device="cuda")
    x[1, 0, 3], x[2, 1, 60] = float("inf"), float("nan")
    y = zr.zr_rotary_fwd(x, zr.zr_rotary_plan(48), start=1)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 27] = want[2, 1, 60] = True
    assert torch.equal(bad, want)


def test_streams_graphs_and_empty():
    plan, f = zr.zr_rotary_plan(64), rates(64)
    x = torch.randn(64, 8, 64, device="cuda").bfloat16()
    pos = torch.arange(64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = zr.zr_rotary_fwd(x, plan, pos)
    side.synchronize()
    check(y, *reference(x, pos, f, False))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = zr.zr_rotary_fwd(x, plan, pos)
    pos += 1000
    graph.replay()
    check(y, *reference(x, pos, f, False))
    assert zr.zr_rotary_fwd(x[:0], plan, pos[:0]).shape == (0, 8, 64)
