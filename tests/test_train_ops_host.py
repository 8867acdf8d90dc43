"""Host-side refusals and plans of the training operators (no GPU): every
argument error is returned before any device call, so made-up addresses do."""
import ctypes
import json

import pytest

import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrRng, ZrTensor, _i64

T = 1 << 32  # distance between made-up operands
NULL, RANK, SHAPE, SIZE, LAYOUT, WORKSPACE, DTYPE, VALUE = -1, -2, -3, -4, -5, -7, -9, -10
F32, BF16 = 0, 1


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


def test_layer_norm_forward_refusals(L):
    x = TT(T, (6, 40))
    ga, be = TT(2 * T, (40,)), TT(3 * T, (40,))

    def fwd(x=x.desc, ga=ga.desc, be=be.desc, eps=1e-5, y=4 * T, ys=None, mean=5 * T, rstd=6 * T, dt=F32):
        return L.zr_layer_norm_fwd(dt, x, ga, be, eps, y, ys, mean, rstd, None)

    assert fwd(dt=7) == DTYPE
    assert fwd(x=TT(T, ()).desc) == RANK
    assert fwd(x=TT(T, (1,) * 9).desc) == RANK
    assert fwd(x=TT(T, (6, 0)).desc) == SHAPE
    assert fwd(x=TT(T, (6, -1)).desc) == SIZE
    assert fwd(x=TT(T, (6, 40), (-1, 1)).desc) == SIZE
    assert fwd(ga=TT(2 * T, (39,)).desc) == SHAPE
    assert fwd(be=TT(2 * T, (1, 40)).desc) == SHAPE
    for eps in (-1e-6, float("nan"), float("inf")):
        assert fwd(eps=eps) == VALUE
    assert fwd(x=TT(None, (6, 40)).desc) == NULL
    assert fwd(y=None) == NULL
    assert fwd(ys=_i64((39, 1))) == LAYOUT                       # y overlaps itself
    assert fwd(y=T + 4) == LAYOUT                                # y partly over x
    assert fwd(y=2 * T) == LAYOUT and fwd(mean=T) == LAYOUT      # over gamma; mean over x
    assert fwd(mean=5 * T, rstd=5 * T + 8) == LAYOUT
    assert fwd(mean=4 * T) == LAYOUT
    assert fwd(x=TT(T, (1 << 31, 1)).desc, ga=NONE, be=NONE, y=1 << 40, mean=None, rstd=None) == SIZE
    assert fwd(x=TT(None, (0, 40)).desc, y=None) == 0            # no rows: nothing to do


def test_layer_norm_backward_refusals(L):
    g, x, ga = TT(T, (6, 40)), TT(2 * T, (6, 40)), TT(3 * T, (40,))
    nb = ctypes.c_size_t(0)

    def bwd(g=g.desc, x=x.desc, ga=ga.desc, mean=4 * T, rstd=5 * T, gx=6 * T, gxs=None, gg=7 * T, gb=8 * T,
            ws=None, n=None, dt=F32):
        nb.value = 0 if n is None else n
        return L.zr_layer_norm_bwd(dt, g, x, ga, mean, rstd, gx, gxs, gg, gb, ws, ctypes.byref(nb), None)

    assert bwd() == 0 and nb.value == 2 * 40 * 4  # one block, two sums of 40 floats
    assert bwd(gg=None) == 0 and nb.value == 40 * 4
    assert bwd(gg=None, gb=None) == 0 and nb.value == 0
    assert L.zr_layer_norm_bwd(F32, g.desc, x.desc, ga.desc, 4 * T, 5 * T, 6 * T, None, None, None, None,
                               None, None) == NULL
    assert bwd(ws=9 * T, n=2 * 40 * 4 - 1) == WORKSPACE
    assert bwd(ws=9 * T + 4, n=1 << 20) == WORKSPACE              # misaligned
    assert bwd(ws=T, n=1 << 20) == LAYOUT and bwd(ws=6 * T, n=1 << 20) == LAYOUT
    assert bwd(dt=-1) == DTYPE
    assert bwd(x=TT(2 * T, (6, 41)).desc) == SHAPE and bwd(x=TT(2 * T, (1, 6, 40)).desc) == SHAPE
    assert bwd(g=TT(T, (6, 0)).desc, x=TT(2 * T, (6, 0)).desc) == SHAPE
    assert bwd(ga=TT(3 * T, (41,)).desc) == SHAPE
    assert bwd(mean=None) == NULL and bwd(rstd=None) == NULL
    assert bwd(g=TT(None, (6, 40)).desc) == NULL and bwd(x=TT(None, (6, 40)).desc) == NULL
    assert bwd(gx=T + 4) == LAYOUT and bwd(gx=T) == 0 and bwd(gx=2 * T) == 0
    assert bwd(gx=4 * T) == LAYOUT and bwd(gg=T) == LAYOUT and bwd(gg=8 * T + 4) == LAYOUT
    assert bwd(gb=5 * T) == LAYOUT and bwd(gxs=_i64((0, 1))) == LAYOUT


def test_layer_norm_plans_cover_every_row_length(L):
    """Every row length fits its plan: a row group's lanes hold the row, and
    the workspace grows with the grid."""
    L.zr_test_describe_layer_norm.argtypes = [ctypes.c_int, ZrTensor, ZrTensor, ctypes.c_char_p,
                                              ctypes.c_size_t]
    buf = ctypes.create_string_buffer(1024)
    for dt in (F32, BF16):
        for dim in list(range(1, 200)) + [255, 256, 257, 768, 1000, 1001, 1024, 1025, 2048, 4096, 8191,
                                          8192, 8193, 8200, 50000]:
            for back in (False, True):
                g = TT(T, (100, dim)) if back else None
                x = TT(1 << 50, (100, dim))
                rc = L.zr_test_describe_layer_norm(dt, g.desc if back else NONE, x.desc, buf, 1024)
                assert rc == 0
                d = json.loads(buf.value)
                wide = 16 // (2 if dt == BF16 else 4)
                assert d["vec"] == (wide if dim % wide == 0 else 1)
                if d["group"]:
                    assert d["group"] * d["ni"] * d["vec"] >= dim and d["ni"] * d["vec"] <= 32
                else:
                    assert dim > 8192
                assert d["rows"] == 100 and (d["ws"] > 0) == back


def test_dropout_refusals(L):
    x, r = TT(T, (6, 40)), TT(2 * T, (6, 40))

    def fwd(x=x.desc, r=r.desc, p=0.1, rng=ZrRng(1, 2, None), out=3 * T, st=None, dt=F32):
        return L.zr_dropout_fwd(dt, x, r, p, rng, out, st, None)

    assert fwd(dt=2) == DTYPE
    for p in (-0.1, 1.5, float("nan")):
        assert fwd(p=p) == VALUE
        assert L.zr_dropout_bwd(F32, x.desc, p, ZrRng(1, 2, None), 3 * T, None, None) == VALUE
    assert fwd(r=TT(2 * T, (6, 41)).desc) == SHAPE and fwd(r=TT(2 * T, (40,)).desc) == SHAPE
    assert fwd(x=TT(T, (1,) * 9).desc) == RANK
    assert fwd(x=TT(None, (6, 40)).desc) == NULL and fwd(out=None) == NULL
    assert fwd(out=T + 4) == LAYOUT and fwd(out=2 * T - 8) == LAYOUT
    assert fwd(st=_i64((20, 1))) == LAYOUT
    assert fwd(rng=ZrRng(1, 2, 3 * T)) == LAYOUT and fwd(rng=ZrRng(1, 2, 9 * T + 4)) == LAYOUT
    assert fwd(x=TT(None, (0, 40)).desc, r=NONE, out=None) == 0


def test_binding_refusals():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        zr.zr_layer_norm_fwd(x)                        # not on a CUDA device
    with pytest.raises(ValueError):
        zr.zr_dropout_fwd(x, 0.1, 1)
    with pytest.raises(TypeError):
        zr.zr_layer_norm_fwd(x, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        zr.zr_dropout_fwd(x.double(), 0.1, 1)
    with pytest.raises(ValueError):
        zr.zr_dropout_fwd(x, 0.1, 1, residual=torch.zeros(4, 9))
    with pytest.raises(ValueError):
        zr.zr_layer_norm_fwd(x, out=torch.zeros(4, 9))
    with pytest.raises(TypeError):
        zr.zr_dropout_fwd(x, 0.1, 1, device_offset=torch.zeros(1))
    with pytest.raises(ValueError):
        zr.zr_layer_norm_bwd(x, x, None, torch.zeros(5), torch.zeros(4))
