"""Host-side checks of the linear head's cross entropy (no GPU): made-up
addresses, the size query."""
import ctypes
import json

import pytest

import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrTensor, _i64

T = 1 << 32
LAYOUT = -5
F32, BF16, MEAN = 0, 1, 1


@pytest.fixture(scope="module")
def L():
    zr.build()
    return zr.lib()


class TT:
    def __init__(self, data, sizes, strides=None):
        self.sizes = _i64(sizes)
        self.strides = _i64(strides) if strides is not None else None
        self.desc = ZrTensor(data, len(sizes), self.sizes, self.strides)


def test_label_layouts(L):
    """Labels in the rows' order, whatever their pitch; permuted ones are refused."""
    w, nb = TT(2 * T, (50, 64)), ctypes.c_size_t(0)
    for sizes, strides, want in (((5, 7), (7, 1), 0), ((5, 7), (8, 1), 0), ((5, 7), (0, 1), 0), ((5, 7), (1, 0), 0),
                                 ((2, 3, 4), (24, 8, 2), 0), ((2, 3, 4), (100, 5, 1), 0), ((2, 3, 4), (0, 0, 0), 0),
                                 ((5, 1), (1, 9), 0), ((5, 7), (1, 5), LAYOUT), ((2, 3, 4), (4, 8, 1), LAYOUT),
                                 ((5, 7), (6, 1), LAYOUT)):
        x, y = TT(T, (*sizes, 64)), TT(3 * T, sizes, strides)
        assert L.zr_linear_xent_fwd(BF16, x.desc, w.desc, 1, y.desc, -100, MEAN, 4 * T, 5 * T, None,
                                    ctypes.byref(nb), None) == want, (sizes, strides)
        assert L.zr_linear_xent_bwd(F32, 4 * T, x.desc, w.desc, 0, y.desc, -100, MEAN, 5 * T, 6 * T, 7 * T, None,
                                    ctypes.byref(nb), None) == want, (sizes, strides)


def plan(L, dt, N, V, D, back=0):
    L.zr_test_describe_linear_xent.argtypes = [ctypes.c_int, ZrTensor, ZrTensor, ctypes.c_int, ZrTensor,
                                               ctypes.c_int, ctypes.c_char_p, ctypes.c_size_t]
    buf = ctypes.create_string_buffer(1024)
    x, w, y = TT(T, (N, D)), TT(1 << 50, (V, D)), TT(1 << 55, (N,))
    assert L.zr_test_describe_linear_xent(dt, x.desc, w.desc, 1, y.desc, back, buf, 1024) == 0
    return json.loads(buf.value)


def test_few_row_forward_limits(L):
    """Both sides of what x may take in shared memory, at widths whose rows of w
    start at 16-byte boundaries, so that this limit alone decides."""
    for dt, n, D, few in ((F32, 16, 6144, True), (F32, 16, 6148, False), (F32, 9, 6144, True), (F32, 9, 6148, False),
                          (F32, 4, 12288, True), (F32, 4, 12292, False), (F32, 2, 24576, True), (F32, 2, 24580, False),
                          (F32, 1, 49152, True), (F32, 1, 49156, False), (BF16, 4, 12288, True), (BF16, 4, 12296, False),
                          (BF16, 3, 12288, True), (BF16, 2, 24576, True), (BF16, 2, 24584, False),
                          (BF16, 1, 49152, True), (BF16, 1, 49160, False), (F32, 16, 512, True), (F32, 17, 512, False),
                          (BF16, 4, 512, True), (BF16, 5, 512, False)):
        assert plan(L, dt, n, 300, D)["kernel"] == ("xent_few" if few else "xent"), (dt, n, D)
