"""Host-side checks of layer norm (no GPU): made-up addresses."""
import ctypes

import pytest

import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrTensor, _i64

T = 1 << 32
LAYOUT = -5


@pytest.fixture(scope="module")
def L():
    zr.build()
    return zr.lib()


def test_workspace_meets_no_operand(L):
    sizes, width = _i64((6, 40)), _i64((40,))
    g, x = ZrTensor(T, 2, sizes, None), ZrTensor(2 * T, 2, sizes, None)
    gamma = ZrTensor(3 * T, 1, width, None)
    nb = ctypes.c_size_t(1 << 20)

    def bwd(ws):
        nb.value = 1 << 20
        return L.zr_layer_norm_bwd(0, g, x, gamma, 4 * T, 5 * T, 6 * T, None, 7 * T, 8 * T, ws, ctypes.byref(nb), None)

    for operand in (1, 2, 3, 4, 5, 6, 7, 8):
        assert bwd(operand * T) == LAYOUT, operand
        assert bwd(operand * T - 16) == LAYOUT, operand
    assert bwd(9 * T) != LAYOUT
