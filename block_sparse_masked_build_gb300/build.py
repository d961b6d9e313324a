"""Builds libbsm.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_bsm_torch.so (its calls from torch tensors; host code only) with g++.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file.  Run ``python -m block_sparse_masked_build_gb300.build``
or call :func:`build`.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbsm.so")
TORCH_SRC = os.path.join(CSRC, "bsm_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_bsm_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__])


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in _deps())


def _torch_stale() -> bool:
    deps = [TORCH_SRC, __file__, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    return not os.path.exists(TORCH_LIB) or any(
        os.path.getmtime(d) > os.path.getmtime(TORCH_LIB) for d in deps)


def _build_torch() -> None:
    """Compile _bsm_torch.so against the installed torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    if not os.path.exists(os.path.join(cuda, "include", "cuda_runtime_api.h")):
        cuda = "/usr/local/cuda"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [*cpp_extension.include_paths(), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"], INCLUDE]
    os.makedirs(OBJDIR, exist_ok=True)
    tmp = TORCH_LIB + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f for i in includes for f in ("-isystem", i)], TORCH_SRC, "-o",
           tmp, "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L",
           os.path.join(cuda, "lib64"), "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {TORCH_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is stale and return the path of libbsm.so."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        torch_lib = ex.submit(_build_torch) if force or _torch_stale() else None
        lib = _build_lib(verbose) if force or is_stale() else LIB
        if torch_lib is not None:
            torch_lib.result()
    return lib


def _build_lib(verbose: bool) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-c", src, "-o",
               obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=4) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
