"""The C library is built and the package imported without torch, and whatever
becomes of the torch binding (fake compilers, no GPU)."""
import os
import subprocess
import sys

import pytest

import broadcast_elementwise_shape_gb300.build  # noqa: F401

B = sys.modules["broadcast_elementwise_shape_gb300.build"]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _tool(path, body):
    path.parent.mkdir(parents=True, exist_ok=True)
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(0o755)


# Notes its arguments and creates what -o names.
WORKS = 'echo "$@" >> "$0.log"\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done\n'


@pytest.fixture
def box(tmp_path, monkeypatch):
    """A build folder of its own, nvcc and g++ that only note their arguments."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "_build" / "libzr.so"))
    monkeypatch.setattr(B, "TORCH_LIB", str(tmp_path / "_build" / "zr_torch.so"))
    monkeypatch.setattr(B, "TORCH_STAMP", str(tmp_path / "_build" / "zr_torch.version"))
    monkeypatch.setenv("CUDA_HOME", str(tmp_path / "nothing"))
    monkeypatch.setenv("PATH", f"{tmp_path / 'cuda' / 'bin'}:{os.environ['PATH']}")
    _tool(tmp_path / "cuda" / "bin" / "nvcc", WORKS)
    _tool(tmp_path / "cuda" / "bin" / "g++", WORKS)
    return tmp_path


def test_the_library_does_not_wait_for_the_binding(box):
    _tool(box / "cuda" / "bin" / "g++", "exit 1\n")
    with pytest.raises(RuntimeError, match="zr_torch"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.TORCH_LIB)
    assert B.stale()                                     # the binding is still to be built


def test_both_are_built_once(box):
    B.build()
    assert os.path.exists(B.LIB) and os.path.exists(B.TORCH_LIB) and not B.stale()
    calls = (box / "cuda" / "bin" / "nvcc.log").read_text()
    B.build()
    assert (box / "cuda" / "bin" / "nvcc.log").read_text() == calls
    with open(B.TORCH_STAMP, "w") as f:
        f.write("another torch")
    B.build()                                            # the binding alone
    assert (box / "cuda" / "bin" / "nvcc.log").read_text() == calls and not B.stale()


def test_cuda_headers_of_an_nvcc_on_path(box):
    B.build()
    compiled = (box / "cuda" / "bin" / "g++.log").read_text().splitlines()[0].split()
    assert os.path.realpath(box / "cuda" / "include") in compiled and "include" not in compiled


def test_without_torch(box, monkeypatch):
    find = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.stale()
    B.build()
    assert os.path.exists(B.LIB) and not B.stale() and not (box / "cuda" / "bin" / "g++.log").exists()


def test_import_without_torch():
    """-E -S: no site-packages, so neither torch nor numpy."""
    code = ("import broadcast_elementwise_shape_gb300 as zr, sys\n"
            "assert 'torch' not in sys.modules and 'zr_dropout_fwd' in dir(zr)\n"
            "try: zr.zr_layer_norm_fwd\n"
            "except ImportError: pass\n"
            "else: raise SystemExit('torch was found')\n"
            "try: zr.no_such_name\n"
            "except AttributeError: pass\n"
            "else: raise SystemExit('a name that is none')\n")
    r = subprocess.run([sys.executable, "-E", "-S", "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_import_does_not_load_torch():
    code = ("import broadcast_elementwise_shape_gb300 as zr, sys\nassert 'torch' not in sys.modules\n"
            "from broadcast_elementwise_shape_gb300 import zr_linear_xent_fwd\nassert 'torch' in sys.modules\n"
            "assert zr.zr_linear_xent_fwd is zr_linear_xent_fwd\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
