"""Host-side checks of the linear head's cross entropy (no GPU): made-up
addresses, the size query."""
import ctypes

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
