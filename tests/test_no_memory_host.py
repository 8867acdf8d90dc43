"""The C entry points raise nothing: a traced call without memory for its line
goes on (no GPU; a preloaded operator new fails on demand)."""
import os
import shutil
import subprocess
import sys

import pytest

import broadcast_elementwise_shape_gb300 as zr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = """
#include <cstdlib>
#include <new>
static bool failing = false;
extern "C" void shim_fail(int on) { failing = on; }
void* operator new(std::size_t n) {
  void* p = failing ? nullptr : std::malloc(n ? n : 1);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
"""

CALLS = """
import ctypes, sys
import broadcast_elementwise_shape_gb300 as zr
from broadcast_elementwise_shape_gb300 import ZrRng, ZrTensor, _i64
L, T = zr.lib(), 1 << 32
fail = ctypes.CDLL(None).shim_fail
sizes, nb = _i64((6, 64)), ctypes.c_size_t(1 << 30)
def t(k, s=sizes): return ZrTensor(k * T, len(s), s, None)
none, row, lab, strides = ZrTensor(None, 0, None, None), _i64((64,)), _i64((6,)), _i64((64, 1))
calls = {
  "binary_fwd": lambda: L.zr_binary_fwd(0, t(1), t(2), 3 * T, strides, None),
  "unary_fwd": lambda: L.zr_unary_fwd(0, 1.0, t(1), 3 * T, strides, None),
  "layer_norm_fwd": lambda: L.zr_layer_norm_fwd(0, t(1), none, none, 1e-5, 3 * T, None, None, None, None),
  "layer_norm_bwd": lambda: L.zr_layer_norm_bwd(0, t(1), t(2), none, 3 * T, 4 * T, 5 * T, None, 6 * T, 7 * T, 8 * T,
                                                ctypes.byref(nb), None),
  "dropout_fwd": lambda: L.zr_dropout_fwd(0, t(1), none, 0.5, ZrRng(1, 2, None), 3 * T, None, None),
  "linear_xent_fwd": lambda: L.zr_linear_xent_fwd(0, t(1), t(2), 1, t(3, lab), -100, 1, 4 * T, 5 * T, 6 * T,
                                                  ctypes.byref(nb), None),
  "linear_xent_bwd": lambda: L.zr_linear_xent_bwd(0, 7 * T, t(1), t(2), 1, t(3, lab), -100, 1, 4 * T, 5 * T, 9 * T,
                                                  12 * T, ctypes.byref(nb), None),
}
call = calls[sys.argv[1]]
first = call()      # what loads on first use has memory
fail(1)
again = call()
fail(0)
assert again == first == -6, (first, again)   # made-up addresses are no device memory
"""


@pytest.mark.parametrize("name", ["binary_fwd", "unary_fwd", "layer_norm_fwd", "layer_norm_bwd", "dropout_fwd",
                                  "linear_xent_fwd", "linear_xent_bwd"])
def test_traced_call_without_memory(tmp_path, name):
    if not shutil.which("g++"):
        pytest.skip("needs g++")
    zr.build()
    (tmp_path / "shim.cpp").write_text(SHIM)
    lib = str(tmp_path / "shim.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", lib, str(tmp_path / "shim.cpp")], check=True)
    env = dict(os.environ, LD_PRELOAD=lib, ZR_TRACE="1")
    r = subprocess.run([sys.executable, "-c", CALLS, name], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stderr.count("zr_trace") == 1, r.stderr   # the first call's
