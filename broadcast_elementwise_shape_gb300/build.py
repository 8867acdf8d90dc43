"""Build the zr CUDA library in-tree: ``_build/libzr.so`` (sm_103a only), and the
training operators' torch binding beside it (``csrc/zr_torch.cpp``, one CPython
module linked against the library and the installed torch).

Each translation unit compiles in parallel with nvcc; the objects link into
one shared library with the CUDA runtime linked statically, so the library
has no dependency beyond the driver.  Arithmetic flags keep IEEE semantics:
no FMA contraction (``-fmad=false``), IEEE division and square root, and
subnormals preserved (``-ftz=false``).
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libzr.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["zr_api.cu", "zr_plan.cpp", "zr_launch_ew.cu", "zr_launch_red.cu", "zr_launch_sab.cu",
           "zr_launch_chain.cu", "zr_launch_bf16.cu", "zr_norm.cu", "zr_launch_norm_fwd.cu",
           "zr_launch_norm_bwd.cu", "zr_dropout.cu", "zr_xent.cu", "zr_launch_gemm.cu"]
TORCH_SOURCE = "zr_torch.cpp"
TORCH_LIB = os.path.join(BUILD, "zr_torch" + sysconfig.get_config_var("EXT_SUFFIX"))
TORCH_STAMP = os.path.join(BUILD, "zr_torch.version")  # the torch it was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-fmad=false", "-ftz=false",
         "-prec-div=true", "-prec-sqrt=true", "-I", INCLUDE]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return files + [os.path.abspath(__file__)]


def _torch_version() -> str:
    from importlib.metadata import version
    return version("torch")


def stale() -> bool:
    if not all(os.path.exists(f) for f in (LIB, TORCH_LIB, TORCH_STAMP)):
        return True
    with open(TORCH_STAMP) as f:
        if f.read() != _torch_version():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(TORCH_LIB))
    return any(os.path.getmtime(f) > t for f in _inputs())


def _build_binding(obj: str) -> None:
    """Link the binding's object against libzr.so and torch."""
    root = _torch_root()
    tmp = f"{TORCH_LIB}.{os.getpid()}.tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda", "-L", BUILD, "-l:libzr.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the torch binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch_version())


def _torch_root() -> str:
    """The installed torch package's folder, without importing it."""
    import importlib.util
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link ``libzr.so`` if missing or older than its sources."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if src == TORCH_SOURCE:
            inc = os.path.join(_torch_root(), "include")
            cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
            cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-I", inc, "-I",
                   os.path.join(inc, "torch", "csrc", "api", "include"), "-I",
                   sysconfig.get_paths()["include"], "-I", cuda, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiler failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        objs = list(ex.map(compile_one, [*SOURCES, TORCH_SOURCE]))
    binding = objs.pop()
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _build_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
