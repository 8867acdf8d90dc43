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


def test_linear_xent_refusals(L):
    x, w, y = TT(T, (6, 64)), TT(2 * T, (50, 64)), TT(3 * T, (6,))
    nb = ctypes.c_size_t(0)
    MEAN, NONE_, SUM = 1, 0, 2

    def fwd(x=x.desc, w=w.desc, it=1, y=y.desc, red=MEAN, loss=4 * T, lse=5 * T, ws=None, n=0, dt=BF16):
        nb.value = n
        return L.zr_linear_xent_fwd(dt, x, w, it, y, -100, red, loss, lse, ws, ctypes.byref(nb), None)

    assert fwd() == 0 and nb.value > 0
    need = nb.value
    assert fwd(dt=2) == DTYPE and fwd(it=2) == DTYPE and fwd(red=3) == NULL
    assert fwd(x=TT(T, ()).desc) == RANK and fwd(w=TT(2 * T, (64,)).desc) == RANK
    assert fwd(w=TT(2 * T, (50, 63)).desc) == SHAPE and fwd(w=TT(2 * T, (0, 64)).desc) == SHAPE
    assert fwd(x=TT(T, (6, 0)).desc, w=TT(2 * T, (50, 0)).desc) == SHAPE
    assert fwd(y=TT(3 * T, (7,)).desc) == SHAPE and fwd(y=TT(3 * T, (6, 1)).desc) == SHAPE
    assert fwd(w=TT(2 * T, (1 << 30, 64)).desc) == SIZE
    assert fwd(x=TT(T, (1 << 30, 64)).desc, y=TT(3 * T, (1 << 30,)).desc) == SIZE
    assert fwd(x=TT(T, (6, 64), (-64, 1)).desc) == SIZE
    assert fwd(x=TT(T, (2, 3, 64)).desc, y=TT(3 * T, (2, 3), (1, 2)).desc) == LAYOUT  # labels out of order
    assert fwd(x=TT(None, (6, 64)).desc) == NULL and fwd(y=TT(None, (6,)).desc) == NULL
    assert fwd(loss=None) == NULL and fwd(lse=None) == NULL
    assert fwd(loss=5 * T) == LAYOUT and fwd(lse=T) == LAYOUT and fwd(loss=3 * T) == LAYOUT
    assert fwd(ws=6 * T, n=need - 1) == WORKSPACE and fwd(ws=6 * T + 8, n=need) == WORKSPACE
    assert fwd(ws=T, n=need) == LAYOUT and fwd(ws=5 * T, n=need) == LAYOUT
    assert fwd(red=NONE_, loss=None) == NULL
    assert L.zr_linear_xent_fwd(BF16, x.desc, w.desc, 1, y.desc, -100, MEAN, 4 * T, 5 * T, None, None, None) == NULL

    def bwd(gl=4 * T, x=x.desc, w=w.desc, y=y.desc, lse=5 * T, gx=7 * T, gw=8 * T, ws=None, n=0, red=MEAN, dt=BF16):
        nb.value = n
        return L.zr_linear_xent_bwd(dt, gl, x, w, 0, y, -100, red, lse, gx, gw, ws, ctypes.byref(nb), None)

    assert bwd() == 0 and nb.value > 6 * 64 * 2
    need = nb.value
    assert bwd(dt=9) == DTYPE and bwd(gl=None) == NULL and bwd(lse=None) == NULL
    assert bwd(gx=8 * T) == LAYOUT and bwd(gx=T) == LAYOUT and bwd(gw=2 * T + 16) == LAYOUT
    assert bwd(gx=5 * T) == LAYOUT and bwd(gw=4 * T) == LAYOUT
    assert bwd(ws=9 * T, n=need - 1) == WORKSPACE and bwd(ws=7 * T, n=need) == LAYOUT
    assert bwd(gx=None, gw=None, ws=9 * T, n=need) == 0          # nothing asked for
    assert bwd(x=TT(None, (0, 64)).desc, y=TT(None, (0,)).desc, gl=None, lse=None, gx=None, gw=None, ws=9 * T,
               n=0) == 0


def _xent_plan(L, dt, N, V, D, back, strides=None, base=T):
    L.zr_test_describe_linear_xent.argtypes = [ctypes.c_int, ZrTensor, ZrTensor, ctypes.c_int, ZrTensor,
                                               ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
    buf = ctypes.create_string_buffer(1024)
    x, w, y = TT(base, (N, D), strides), TT(1 << 50, (V, D)), TT(1 << 55, (N,))
    assert L.zr_test_describe_linear_xent(dt, x.desc, w.desc, 1, y.desc, back, buf, 1024) == 0
    return json.loads(buf.value)


def test_linear_xent_plans(L):
    """Operands go as they are only where the tensor maps can take them; the
    backward's pieces cover the vocabulary within the workspace's bound."""
    d = _xent_plan(L, BF16, 100, 1000, 128, 0)
    assert (d["parts"], d["pack_x"], d["pack_w"], d["kernel"]) == (1, 0, 0, "xent")
    assert _xent_plan(L, BF16, 100, 1000, 72, 0)["pack_w"] == 1           # whole blocks of 64
    assert _xent_plan(L, BF16, 100, 1000, 128, 0, strides=(132, 1))["pack_x"] == 1
    assert _xent_plan(L, BF16, 100, 1000, 128, 0, strides=(136, 1))["pack_x"] == 0
    assert _xent_plan(L, BF16, 100, 1000, 128, 0, base=T + 2)["pack_x"] == 1
    assert _xent_plan(L, BF16, 100, 1000, 128, 0, strides=(0, 1))["pack_x"] == 1
    assert _xent_plan(L, BF16, 100, 1000, 128, 1)["pack_x"] == 1          # rows left out become zero
    f = _xent_plan(L, F32, 100, 1000, 128, 0)
    assert (f["parts"], f["pack_x"], f["pack_w"]) == (3, 1, 1)
    for n in (1, 4):
        assert _xent_plan(L, BF16, n, 1000, 128, 0)["kernel"] == "xent_few"
    assert _xent_plan(L, BF16, 5, 1000, 128, 0)["kernel"] == "xent"
    assert _xent_plan(L, BF16, 4, 50001, 768, 0)["kernel"] == "xent"      # w as it is, and much of it
    assert _xent_plan(L, BF16, 4, 50001, 776, 0)["kernel"] == "xent_few"  # w would have to be copied
    for n, D, kernel in ((16, 1000, "xent_few"), (17, 1000, "xent"), (16, 6144, "xent_few"), (16, 6145, "xent"),
                         (4, 12288, "xent_few"), (4, 12289, "xent")):
        assert _xent_plan(L, F32, n, 1000, D, 0)["kernel"] == ("xent" if D % 4 else kernel)
    for dt, parts in ((BF16, 1), (F32, 3)):
        for N in (1, 7, 4096, 100000, 1000003):
            for V in (1, 255, 50001, 262144):
                d = _xent_plan(L, dt, N, V, 64, 1)
                assert d["piece"] % 256 == 0 and (d["n_piece"] - 1) * d["piece"] < V <= d["n_piece"] * d["piece"]
                g = N * min(d["piece"], (V + 63) // 64 * 64) * 2 * parts
                assert d["ws"] >= g and g <= max((1 << 30) + N * 512 * parts, N * 2304 * 2 * parts)


def test_linear_xent_slices(L):
    """A long sum over few tiles is cut into slices, none of them empty, whose
    planes the workspace holds; sums that fill the GPU stay whole."""
    for dt, N, V, D, cut in ((F32, 40, 100000, 384, 0), (BF16, 300, 32000, 1024, 0), (BF16, 1, 50001, 768, 0),
                             (BF16, 16384, 500, 1024, 1), (F32, 280, 650000, 24, 0)):
        d = _xent_plan(L, dt, N, V, D, 1)
        s = (d["slices_x"], d["slices_w"])
        assert s[cut] > 1 and s[1 - cut] == 1, (N, V, D, s)
        assert d["ws"] >= s[cut] * (N, V)[cut] * D * 4
    for dt, N, V, D in ((F32, 4080, 5003, 384), (BF16, 2048, 8192, 2048), (BF16, 4096, 32000, 1024), (F32, 1, 1, 1),
                        (BF16, 16384, 50001, 768), (F32, 64, 64, 64)):
        d = _xent_plan(L, dt, N, V, D, 1)
        assert (d["slices_x"], d["slices_w"]) == (1, 1), (N, V, D)
    for dt in (F32, BF16):
        for N in (1, 65, 129, 1000, 16384, 1000003):
            for V in (1, 64, 500, 50001, 1000000):
                for D in (1, 65, 2048):
                    d = _xent_plan(L, dt, N, V, D, 1)
                    for s, k, m in ((d["slices_x"], min(d["piece"], V), N), (d["slices_w"], N, min(d["piece"], V))):
                        kb = (k + 63) // 64
                        assert 1 <= s <= kb and -(-kb // -(-kb // s)) == s
                        assert s == 1 or s * m * D * 4 <= (1 << 30)


@pytest.mark.parametrize("cg", [1, 2])
def test_every_tile_is_dealt_out_once(L, cg):
    """All tiles of one and of two products, each to one worker, and no worker
    with more than a tile over the mean."""
    import random
    L.zr_test_gemm_walk.argtypes = [ctypes.c_uint32] * 4 + [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                                           ctypes.c_void_p]
    rng = random.Random(5)
    cases = [(1, 0, 1, 1), (76, 0, 3, 1), (1000, 0, 5, 1), (1, 1, 9, 2), (192, 588, 782, 256), (32, 40, 79, 64),
             (75, 1, 100, 1), (77, 400, 4, 300), (5, 1000, 900, 1)]
    cases += [(rng.randrange(1, 500), rng.randrange(0, 3000), rng.randrange(1, 800), rng.randrange(1, 800))
              for _ in range(300)]
    for t0, t1, k0, k1 in cases:
        visits = (ctypes.c_uint32 * (t0 + t1))()
        load = (ctypes.c_uint64 * 152)()
        workers = ctypes.c_uint32(0)
        assert L.zr_test_gemm_walk(t0, t1, k0, k1, cg, visits, load, ctypes.byref(workers)) == 0
        n = workers.value
        assert n == min(t0 + t1, 152 // cg)
        assert all(v == 1 for v in visits), (t0, t1, k0, k1)
        mean = (t0 * k0 + t1 * k1) / n
        assert max(load[:n]) <= mean + k0 + 2 * k1, (t0, t1, k0, k1)
