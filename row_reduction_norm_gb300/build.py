"""Build the CUDA library in-tree: ``row_reduction_norm_gb300/librmsnorm_gb300.so``.

Every ``csrc/*.cu`` file is compiled for sm_103a only (one ``-gencode``) in
parallel, then linked into one shared library with the CUDA runtime linked
statically.  No cmake, no torch extension machinery: plain nvcc.  Beside it,
``csrc/fastcall.cpp`` becomes the Python module ``_fastcall`` (plain g++ against
the headers and libraries of the installed torch, whose version and Python's are
part of its file name: a module for another torch or Python is never loaded).

    python -m row_reduction_norm_gb300.build [--force]
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "librmsnorm_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build the library")
    return exe


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(INCLUDE, "rmsnorm.h")]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(d) > t for d in _deps())


def fastcall_path() -> str:
    """Where the native Python calls for the running torch and Python are."""
    import torch
    return os.path.join(PKG, f"_fastcall-torch{torch.__version__}" + sysconfig.get_config_var("EXT_SUFFIX"))


def build_fastcall(force: bool = False) -> str:
    """Compile the native Python calls if there are none for the running torch
    and Python, or older ones than their sources."""
    header, path = os.path.join(INCLUDE, "rmsnorm.h"), fastcall_path()
    if not force and os.path.exists(path) and os.path.getmtime(path) > max(
            os.path.getmtime(FAST_SRC), os.path.getmtime(header)):
        return path
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"), os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f for i in includes for f in ("-I", i)), FAST_SRC, "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fastcall.cpp:\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library, and the native Python calls, where they
    are missing or older than their sources."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        fast = ex.submit(build_fastcall, force)
        lib = _build_library(force, verbose, ptxas_info)
        fast.result()
    return lib


def _build_library(force: bool, verbose: bool, ptxas_info: bool) -> str:
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH_FLAGS, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def main():
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    main()
