"""Build libpbsa.so (sm_100a) in-tree with nvcc, and the Python binding of its request entry points.

    python -m block_sparse_attention_pbsa_b200.build

Each CUDA source is compiled to an object under ``_build/`` (in parallel), then linked
into ``block_sparse_attention_pbsa_b200/libpbsa.so`` with the static CUDA runtime.  The
driver API is reached through ``cudaGetDriverEntryPoint``, so nothing links libcuda.
The binding (``csrc/requests_binding.cpp``) is a Python module against the installed torch's headers, for this
interpreter; where it cannot be built the library is, and the build warns: only the calls that go through it are missing.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

from ._lib import binding_path

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpbsa.so")

SOURCES = ["api.cu", "blockify.cu", "score_select.cu", "blockify_select.cu", "attend_f32.cu", "attend_tc.cu",
           "memory_update.cu", "noalloc.cu", "attend_bwd.cu", "request_tables.cu", "q4_cache.cu", "attend_q4.cu", "attend_q4_tc.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    deps = [path] + [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".cuh", ".h"))]
    deps.append(os.path.join(ROOT, "include", "pbsa.h"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", path, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _binding() -> None:
    import torch

    out = binding_path()
    home = os.path.dirname(torch.__file__)
    src = os.path.join(CSRC, "requests_binding.cpp")
    deps = [src, os.path.join(ROOT, "include", "pbsa.h")]
    if os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(d) for d in deps):
        return
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found: set CXX or put it on PATH")
    inc = [os.path.join(ROOT, "include"), os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    lib = os.path.join(home, "lib")
    tmp = out + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in inc), src, "-o", tmp,
           f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on the binding:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _link(objs: list[str]) -> None:
    if os.path.exists(LIB) and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs):
        return
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_binding)
        _link(list(ex.map(lambda s: _compile(s, verbose), SOURCES)))
        try:
            binding.result()
        except Exception as e:   # (no torch, no compiler, headers that do not fit: nothing else needs them)
            warnings.warn(f"the binding of the request calls was not built, and they will raise: {e}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
