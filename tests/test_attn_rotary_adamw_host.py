"""Host-side refusals and plans of the attention, the rotary positions and the
AdamW step (no GPU): every argument error is returned before any device call,
so made-up addresses do."""
import ctypes
import math

import pytest

import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrAdamw, ZrAdamwTensor, ZrRotary, ZrTensor, _i64

T = 1 << 36  # distance between made-up operands
NULL, RANK, SHAPE, SIZE, LAYOUT, DEVICE, WORKSPACE, DTYPE, VALUE = -1, -2, -3, -4, -5, -6, -7, -9, -10
F32, BF16 = 0, 1
I32, I64 = 0, 1


@pytest.fixture(scope="module")
def L():
    zr.build()
    return zr.lib()


class TT:
    """A zr_tensor at a made-up address."""

    def __init__(self, data, sizes, strides=None):
        self.sizes = _i64(sizes)
        self.strides = _i64(strides) if strides is not None else None
        self.desc = ZrTensor(data, len(sizes), self.sizes, self.strides)


NONE = ZrTensor(None, 0, None, None)


def test_attention_forward_refusals(L):
    q, kv = (2, 10, 4, 64), (2, 10, 2, 64)

    nb = ctypes.c_size_t(0)

    def fwd(q=TT(T, q), k=TT(2 * T, kv), v=TT(3 * T, kv), scale=0.1, off=None, n=0, out=4 * T, os=None, low=None, lse=5 * T, dt=BF16, ws=8 * T,
            size=1 << 24):
        nb.value = size
        return L.zr_attention_fwd(dt, q.desc, k.desc, v.desc, scale, off, n, out, os, low, lse, ws, ctypes.byref(nb), None)

    assert fwd(ws=None) == 0 and nb.value == 0 and fwd(ws=None, dt=F32) == 0 and nb.value == 0 and fwd(ws=16, size=0) == DEVICE
    need = 384 * 2 * 100 * (4 + 2 + 2)  # three parts of 64 elements per row of q, k and v
    f32 = dict(q=TT(T, (2, 100, 4, 64)), k=TT(2 * T, (2, 100, 2, 64)), v=TT(3 * T, (2, 100, 2, 64)), dt=F32)
    assert fwd(**f32, ws=None) == 0 and nb.value == need
    assert fwd(**f32) == DEVICE and fwd(**f32, size=need - 1) == WORKSPACE and fwd(**f32, ws=8 * T + 8) == WORKSPACE
    assert fwd(**f32, ws=4 * T) == LAYOUT
    odd = [TT(i * T, (2, 100, 1, d)) for i, d in ((1, 33), (2, 33), (3, 33))]  # rows of 64 elements: copies
    assert fwd(*odd, ws=None) == 0 and nb.value >= 128 * 2 * 100 * 3
    assert L.zr_attention_fwd(BF16, TT(T, q).desc, TT(2 * T, kv).desc, TT(3 * T, kv).desc, 0.1, None, 0, 4 * T, None, None, None, None, None, None) == NULL

    assert fwd() == DEVICE  # nothing but the addresses is wrong
    assert fwd(dt=5) == DTYPE and fwd(dt=F32, low=6 * T) == DTYPE
    assert fwd(q=TT(T, (4, 64))) == RANK and fwd(k=TT(2 * T, (10, 2, 64))) == RANK
    assert fwd(off=7 * T, n=2) == RANK                                  # borders go with rank 3
    assert fwd(q=TT(T, (2, 10, 3, 64))) == SHAPE                        # 3 heads read 2
    assert fwd(v=TT(3 * T, (2, 10, 1, 64))) == SHAPE and fwd(k=TT(2 * T, (2, 9, 2, 64)), v=TT(3 * T, (2, 9, 2, 64))) == SHAPE
    assert fwd(q=TT(T, (2, 10, 4, 32))) == SHAPE
    assert fwd(q=TT(T, (2, 10, 0, 64))) == SHAPE and fwd(k=TT(2 * T, (2, 10, 0, 64)), v=TT(3 * T, (2, 10, 0, 64))) == SHAPE
    wide = [TT(i * T, (2, 10, 1, 257)) for i in (1, 2, 3)]
    assert fwd(*wide) == SIZE
    long = [TT(i * T, (1, 1 << 30, 1, 1)) for i in (1, 2, 3)]
    assert fwd(*long) == SIZE
    many = [TT(i * T, (1 << 14, 1 << 14, 64, 1)) for i in (1, 2, 3)]
    assert fwd(*many) == SIZE
    p3 = [TT(i * T, (10, 2, 64)) for i in (1, 2, 3)]
    assert fwd(*p3, off=7 * T, n=-1) == SIZE
    assert fwd(*p3, off=7 * T + 2, n=1) == LAYOUT
    assert fwd(*p3, off=7 * T, n=1) == DEVICE and fwd(*p3) == DEVICE
    assert fwd(*p3, off=7 * T, n=0) == 0                                # no sequences
    for s in (float("nan"), float("inf")):
        assert fwd(scale=s) == VALUE
    assert fwd(q=TT(None, q)) == NULL and fwd(out=None) == NULL
    assert fwd(out=T) == LAYOUT and fwd(out=2 * T + 64) == LAYOUT and fwd(lse=T) == LAYOUT and fwd(low=4 * T) == LAYOUT
    assert fwd(lse=5 * T + 2) == LAYOUT and fwd(low=6 * T + 1) == LAYOUT
    assert fwd(os=_i64((0, 256, 64, 1))) == LAYOUT                      # out overlaps itself
    assert fwd(q=TT(T, q, (-1, 1, 1, 1))) == SIZE
    assert fwd(*[TT(None, (2, 0, 2, 64))] * 3, out=None, lse=None) == 0


def test_attention_backward_refusals(L):
    qs, kvs = (2, 10, 4, 64), (2, 10, 2, 64)
    nb = ctypes.c_size_t(0)

    def bwd(g=TT(T, qs), q=TT(2 * T, qs), k=TT(3 * T, kvs), v=TT(4 * T, kvs), o=TT(5 * T, qs), low=None, lse=6 * T, scale=0.1, off=None, n=0,
            gq=7 * T, gqs=None, gk=8 * T, gks=None, gv=9 * T, gvs=None, ws=10 * T, size=1 << 20, dt=BF16):
        nb.value = size
        return L.zr_attention_bwd(dt, g.desc, q.desc, k.desc, v.desc, o.desc, low, lse, scale, off, n, gq, gqs, gk, gks, gv, gvs, ws,
                                  ctypes.byref(nb), None)

    assert bwd() == DEVICE
    assert bwd(ws=None) == 0 and nb.value == 2 * 2 * 4 * 128 * 4  # lse and delta of 128 rows per batch entry and head
    assert bwd(size=2 * 2 * 4 * 128 * 4 - 1) == WORKSPACE and bwd(ws=10 * T + 8) == WORKSPACE
    assert L.zr_attention_bwd(BF16, *[TT(i * T, s).desc for i, s in ((1, qs), (2, qs), (3, kvs), (4, kvs), (5, qs))], None, 6 * T, 0.1, None, 0,
                              7 * T, None, 8 * T, None, 9 * T, None, None, None, None) == NULL
    assert bwd(dt=9) == DTYPE and bwd(dt=F32, low=11 * T) == DTYPE
    assert bwd(g=TT(T, (2, 10, 4, 32))) == SHAPE and bwd(o=TT(5 * T, (10, 4, 64))) == RANK
    assert bwd(lse=None) == NULL and bwd(g=TT(None, qs)) == NULL and bwd(o=TT(None, qs)) == NULL
    assert bwd(gq=T) == LAYOUT and bwd(gq=2 * T) == LAYOUT and bwd(gk=6 * T) == LAYOUT and bwd(gv=8 * T) == LAYOUT
    assert bwd(ws=7 * T) == LAYOUT and bwd(gq=None, gk=None, gv=None) == 0
    assert bwd(gqs=_i64((0, 256, 64, 1))) == LAYOUT
    # The parts of one projection's rows lie between one another.
    st = _i64((10 * 512, 512, 64, 1))
    part = dict(gq=7 * T, gqs=st, gk=7 * T + 2 * 256, gks=st, gv=7 * T + 2 * 384, gvs=st)
    assert bwd(**part) == DEVICE
    assert bwd(**{**part, "gk": 7 * T + 2 * 255}) == LAYOUT     # one element into grad_q's heads
    assert bwd(**{**part, "gv": 7 * T + 2 * 385}) == LAYOUT     # one element over the row's end, into the next token
    assert bwd(**{**part, "gks": _i64((10 * 511, 511, 64, 1))}) == LAYOUT
    assert bwd(**{**part, "gk": 7 * T + 2 * 256 + 1}) in (LAYOUT, DEVICE)


def test_attention_spans_of_the_parts_exhaustively(L):
    """grad_q and grad_k as views of one buffer: refused exactly where they share an element (or, with odd strides, at least there)."""
    nb = ctypes.c_size_t(1 << 24)
    qs, kvs = (2, 3, 2, 4), (2, 3, 1, 4)
    args = [TT(i * T, s) for i, s in ((1, qs), (2, qs), (3, kvs), (4, kvs), (5, qs))]

    def elements(base, sizes, strides):
        out = {base}
        for n, s in zip(sizes, strides):
            out = {e + i * s for e in out for i in range(n)}
        return out

    for pitch in (8, 12, 13):
        for at in range(0, 30):
            sq, sk = (3 * pitch, pitch, 4, 1), (3 * pitch, pitch, 4, 1)
            rc = L.zr_attention_bwd(F32, *[a.desc for a in args], None, 6 * T, 0.5, None, 0, 7 * T, _i64(sq), 7 * T + 4 * at, _i64(sk), None, None,
                                    10 * T, ctypes.byref(nb), None)
            shares = bool(elements(0, qs, sq) & elements(at, kvs, sk))
            assert rc in (LAYOUT, DEVICE)
            assert not (shares and rc == DEVICE), (pitch, at)
            if at < pitch and not shares and at + 4 <= pitch:
                assert rc == DEVICE, (pitch, at)


def plan(L, part=64, inter=0, base=1e4, factor=1.0, original=0.0, low=1.0, high=32.0, magnitude=1.0):
    p = ZrRotary()
    return L.zr_rotary_plan(part, inter, base, factor, original, low, high, magnitude, ctypes.byref(p)), p


def test_rotary_plan(L):
    assert L.zr_rotary_plan(64, 0, 1e4, 1.0, 0.0, 1.0, 32.0, 1.0, None) == NULL
    for part in (0, -2, 3, 514):
        assert plan(L, part=part)[0] == SIZE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(base=0.5), dict(base=inf), dict(factor=0.0), dict(factor=-1.0), dict(factor=nan), dict(original=-1.0), dict(original=inf),
                dict(magnitude=nan), dict(original=8.0, low=-1.0), dict(original=8.0, low=2.0, high=2.0), dict(original=8.0, high=inf)):
        assert plan(L, **bad)[0] == VALUE, bad
    for part in (2, 64, 512):
        rc, p = plan(L, part=part, factor=3.0)
        assert rc == 0 and p.part == part and p.magnitude == 1
        for j in range(part // 2):
            want = 1e4 ** (-2 * j / part) / 3 / (2 * math.pi)
            assert abs(p.turns[j] / 2 ** 64 - want) <= 8 * 2.0 ** -53 * want + 2.0 ** -64
    rc, p = plan(L, part=64, factor=4.0, original=4096.0)
    for j in range(32):
        f = 1e4 ** (-2 * j / 64)
        w = min(1, max(0, (4096 * f / (2 * math.pi) - 1) / 31))
        want = f * (w + (1 - w) / 4) / (2 * math.pi)
        assert abs(p.turns[j] / 2 ** 64 - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -64
    assert plan(L, factor=0.125)[0] == 0  # more than a turn a position: the fraction is kept
    assert abs(plan(L, factor=0.125)[1].turns[0] / 2 ** 64 - (8 / (2 * math.pi) - 1)) < 2.0 ** -50


def test_rotary_refusals(L):
    good = plan(L)[1]

    def fwd(x=TT(T, (3, 5, 4, 64)), p=good, pt=I64, pos=TT(2 * T, (3, 5)).desc, out=3 * T, os=None, dt=F32, f=L.zr_rotary_fwd):
        return f(dt, x.desc, ctypes.byref(p) if p else None, pt, pos, 0, out, os, None)

    for f in (L.zr_rotary_fwd, L.zr_rotary_bwd):
        assert fwd(f=f) == DEVICE and fwd(pos=NONE, f=f) == DEVICE
        assert fwd(p=None, f=f) == NULL
        assert fwd(dt=4, f=f) == DTYPE and fwd(pt=3, f=f) == DTYPE
        assert fwd(x=TT(T, (64,)), pos=NONE, f=f) == RANK
        assert fwd(x=TT(T, (3, 5, 4, 63)), f=f) == SHAPE
        assert fwd(pos=TT(2 * T, (5, 3)).desc, f=f) == SHAPE and fwd(pos=TT(2 * T, (3, 5, 1)).desc, f=f) == SHAPE
        assert fwd(out=None, f=f) == NULL and fwd(x=TT(None, (3, 5, 4, 64)), f=f) == NULL
        assert fwd(out=T + 4, f=f) == LAYOUT and fwd(out=2 * T, f=f) == LAYOUT and fwd(out=T, f=f) == DEVICE
        assert fwd(os=_i64((1280, 0, 64, 1)), f=f) == LAYOUT
        assert fwd(pos=TT(2 * T + 4, (3, 5)).desc, f=f) == LAYOUT
        assert fwd(x=TT(T, (1 << 20, 1 << 12, 1, 64)), pos=NONE, out=1 << 50, f=f) == SIZE
        assert fwd(x=TT(T, (1, 1 << 20, 64)), pos=NONE, out=1 << 50, f=f) == SIZE
        assert fwd(x=TT(None, (0, 5, 4, 64)), pos=TT(None, (0, 5)).desc, out=None, f=f) == 0
    bad = plan(L)[1]
    bad.part = 7
    assert fwd(p=bad) == SIZE


def adam_tensor(at, n, bits=32, **kw):
    d = dict(param=at * T, copy=(at + 1) * T, grad=(at + 2) * T, m=(at + 3) * T, v=(at + 4) * T, n=n, weight_decay=0.1)
    if bits == 8:
        d |= dict(m_scale=(at + 5) * T, v_scale=(at + 6) * T)
    return ZrAdamwTensor(**{**d, **kw})


def test_adamw_refusals(L):
    good = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, seed=0)

    def step(tensors, bits=32, gt=F32, count=None, **kw):
        arr = (ZrAdamwTensor * max(1, len(tensors)))(*tensors)
        how = ZrAdamw(**{**good, **kw})
        return L.zr_adamw_step(gt, bits, len(tensors) if count is None else count, arr, ctypes.byref(how), None)

    one = [adam_tensor(1, 1000)]
    assert step(one) == DEVICE and step([adam_tensor(1, 1000, 8)], bits=8) == DEVICE
    assert step([]) == 0 and step([adam_tensor(1, 0)]) == 0 and step(one, count=-1) == SIZE
    assert L.zr_adamw_step(F32, 32, 1, None, ctypes.byref(ZrAdamw(**good)), None) == NULL
    assert L.zr_adamw_step(F32, 32, 0, None, None, None) == NULL
    assert step(one, gt=3) == DTYPE and step(one, bits=16) == DTYPE
    nan = float("nan")
    for bad in (dict(lr=nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1 - 1e-12), dict(eps=-1.0), dict(eps=nan), dict(step=0)):
        assert step(one, **bad) == VALUE, bad
    assert step([adam_tensor(1, 10, weight_decay=float("inf"))]) == VALUE
    assert step([adam_tensor(1, -1)]) == SIZE and step([adam_tensor(1, 1 << 34, 8)], bits=8) == SIZE and step([adam_tensor(1, 1 << 40)]) == SIZE
    for field in ("param", "grad", "m", "v"):
        assert step([adam_tensor(1, 10, **{field: None})]) == NULL
        assert step([adam_tensor(1, 10, **{field: 20 * T + 1})]) == LAYOUT
    assert step([adam_tensor(1, 10, 8, m_scale=None)], bits=8) == NULL and step([adam_tensor(1, 10, 8, v_scale=20 * T + 2)], bits=8) == LAYOUT
    assert step([adam_tensor(1, 10, copy=None)]) == DEVICE
    # Overlaps within a tensor and between two; a gradient may be shared.
    assert step([adam_tensor(1, 1000, m=T + 3996)]) == LAYOUT and step([adam_tensor(1, 1000, m=T + 4000)]) == DEVICE
    assert step([adam_tensor(1, 1000, grad=T)]) == LAYOUT
    two = lambda **kw: [adam_tensor(1, 1000), adam_tensor(10, 1000, **kw)]  # noqa: E731
    assert step(two()) == DEVICE and step(two(param=T)) == LAYOUT and step(two(v=3 * T)) == LAYOUT
    assert step(two(grad=3 * T)) == DEVICE and step(two(copy=T + 400)) == LAYOUT
    assert step(one, device_step=T) == LAYOUT and step(one, device_lr=20 * T + 2) == LAYOUT and step(one, device_step=20 * T + 4) == LAYOUT


def test_adamw_state_refusals(L):
    vp = ctypes.c_void_p

    def state(t, m=(30 * T,), v=(31 * T,), count=1):
        arr = (ZrAdamwTensor * 1)(t)
        return L.zr_adamw_state(count, arr, (vp * 1)(*m) if m else None, (vp * 1)(*v) if v else None, None)

    good = adam_tensor(1, 300, 8)
    assert state(good) == DEVICE and state(good, m=None) == DEVICE and state(good, m=None, v=None) == 0 and state(good, count=0) == 0
    assert state(good, count=-1) == SIZE and L.zr_adamw_state(1, None, None, None, None) == NULL
    assert state(adam_tensor(1, 300, 8, m=None)) == NULL and state(adam_tensor(1, 300, 8, m=None), m=None) == DEVICE
    assert state(adam_tensor(1, 300, 8, v_scale=None)) == NULL and state(adam_tensor(1, 1 << 34, 8)) == SIZE
    assert state(good, m=(4 * T,)) == LAYOUT and state(good, v=(30 * T,)) == LAYOUT and state(good, m=(30 * T + 1,)) == LAYOUT
