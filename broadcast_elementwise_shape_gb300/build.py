"""Build the zr CUDA library in-tree: ``_build/libzr.so`` (sm_103a only), and the
training operators' torch binding beside it (``csrc/zr_torch.cpp``, one CPython
module linked against the library and the installed torch; the library neither
needs it nor torch).

Each translation unit compiles in parallel with nvcc; the objects link into
one shared library with the CUDA runtime linked statically, so the library
has no dependency beyond the driver.  Arithmetic flags keep IEEE semantics:
no FMA contraction (``-fmad=false``), IEEE division and square root, and
subnormals preserved (``-ftz=false``).
"""
from __future__ import annotations

import importlib.util
import os
import shutil
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
           "zr_launch_norm_bwd.cu", "zr_dropout.cu", "zr_xent.cu", "zr_launch_gemm.cu",
           "zr_rotary.cu", "zr_adamw.cu", "zr_attn.cu", "zr_attn_any.cu",
           "zr_attn_fwd.cu", "zr_attn_bwd.cu",
           "zr_attn_f32.cu"]
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


def _torch_root():
    """The installed torch package's folder, without importing it; None if there is none."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _torch_version() -> str:
    from importlib.metadata import version
    return version("torch")


def _older(target: str) -> bool:
    """Whether `target` is missing or older than any source."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _binding_stale() -> bool:
    """The binding needs torch; without it there is none to build."""
    if _torch_root() is None:
        return False
    if not os.path.exists(TORCH_STAMP) or _older(TORCH_LIB):
        return True
    with open(TORCH_STAMP) as f:
        return f.read() != _torch_version()


def stale() -> bool:
    return _older(LIB) or _binding_stale()


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_binding(nvcc: str) -> str:
    """The binding's object file."""
    found = shutil.which(nvcc)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(found or nvcc)))
    inc = os.path.join(_torch_root(), "include")
    obj = os.path.join(BUILD, "zr_torch.o")
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-I", inc, "-I",
          os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
          "-I", os.path.join(cuda, "include"), "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj],
         f"compilation of {TORCH_SOURCE}")
    return obj


def _link_binding(obj: str) -> None:
    """Link the binding's object against libzr.so and torch."""
    tmp = f"{TORCH_LIB}.{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(_torch_root(), "lib"), "-ltorch_python",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda", "-L", BUILD, "-l:libzr.so",
          "-Wl,-rpath,$ORIGIN"], "link of the torch binding")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link ``libzr.so`` if missing or older than its sources, and
    where torch is installed the binding.  The library does not wait for the
    binding: it is in place when the binding's errors are raised."""
    lib, binding = force or _older(LIB), _torch_root() is not None and (force or _binding_stale())
    if not lib and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        said = _run([nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj],
                    f"compilation of {src}")
        if verbose or ptxas_info:
            sys.stderr.write(said)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        torch_obj = ex.submit(_compile_binding, nvcc) if binding else None
        objs = [ex.submit(compile_one, s) for s in SOURCES] if lib else []
    if lib:
        tmp = f"{LIB}.{os.getpid()}.tmp"
        _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *(o.result() for o in objs)], "link")
        os.replace(tmp, LIB)
    if binding:
        _link_binding(torch_obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
