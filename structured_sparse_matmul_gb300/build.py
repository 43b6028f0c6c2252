"""Build libvnm.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a.

Each translation unit compiles in parallel; the link uses nvcc's static CUDA
runtime, so the library needs only the driver at run time. Output:
``structured_sparse_matmul_gb300/_build/libvnm.so`` (git-ignored), and beside it
the Python binding's C part, ``_vnm_binding.*.so``, named after the Python it is for.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import List

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libvnm.so")
BINDING_PATH = os.path.join(BUILD_DIR, "_vnm_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cu", "compress.cu", "spmm_simt.cu", "spmm_tc.cu", "spmm_noalloc.cu", "gemm_compress.cu", "energy.cu", "bitmap.cu",
           "rmsnorm.cu", "fp8_quantize.cu", "fp8_linear.cu", "fp8_decode.cu", "dense_api.cu"]
HEADERS = ["vnm_internal.h", "vnm_ptx.cuh", "vnm_select.cuh", "vnm_dense.h", "vnm_fp8.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v"]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newer_than(path: str, names: List[str]) -> bool:
    """Whether `path` exists and is no older than these files of csrc and the public headers."""
    if not os.path.exists(path):
        return False
    files = [os.path.join(CSRC, s) for s in names]
    files += [os.path.join(ROOT, "include", h) for h in ("vnm.h", "vnm_testing.h")]
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in files)


def _library_up_to_date() -> bool:
    return _newer_than(LIB_PATH, SOURCES + HEADERS)


def _binding_up_to_date() -> bool:
    return _newer_than(BINDING_PATH, ["binding.c"])


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def build_binding() -> None:
    """Compile the binding's C part with the host compiler for the running Python. Without
    Python's headers it is left out: the library and the pruned calls do not need it."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        sys.stderr.write(f"no Python.h in {include}: the norm and 8-bit calls will not be available from Python\n")
        return
    tmp = BINDING_PATH + ".tmp"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-Wall", "-shared", "-fPIC", "-I", include,
           os.path.join(CSRC, "binding.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libvnm.so, then the binding, where any input is newer; return the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if force or not _library_up_to_date():
        build_library(verbose)
    if force or not _binding_up_to_date():
        build_binding()
    return LIB_PATH


def build_library(verbose: bool = False) -> None:
    """Compile and link libvnm.so."""
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        log = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".ptxas.txt")
        cmd = [nvcc, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(log, "w") as f:
            f.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stdout.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
