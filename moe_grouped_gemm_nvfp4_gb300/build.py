"""Builds the in-tree CUDA library `_lib/libnvfp4_gb300.so` for sm_103a and the
native Python binding `_lib/_binding-<torch version>.so` of its hot calls.

The translation units compile in parallel with nvcc, then link into
one shared object with the CUDA runtime linked statically; the binding is one
C++ file against torch's headers.  A build is skipped when its output is newer
than every source and header.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(OUT_DIR, "libnvfp4_gb300.so")
SOURCES = ["api.cu", "quantize.cu", "route.cu", "gemm.cu", "gemm_pair.cu", "gemm_pair_grouped.cu",
           "sparse.cu",
           "attention.cu", "attention_tc.cu", "attention_tc_wide.cu",
           "tokens.cu", "fp8_quantize.cu", "fp8_gemm.cu",
           "fp8_rows.cu", "norm.cu", "gate.cu", "fp8_moe.cu"]
HEADERS = [os.path.join(CSRC, h) for h in ("common.cuh", "kernels.h", "format.cuh", "attention.h",
                                                "attention_tc_common.cuh",
                                                "rows.cuh", "tokens.h", "fp8.h",
                                                "fp8_common.cuh", "fp8_quant.cuh", "norm.h",
                                                "gate.h", "gate.cuh", "fp8_moe.h")] + [
    os.path.join(ROOT, "include", "nvfp4.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(OUT_DIR, f"_binding-{torch.__version__}.so")


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_stale() -> bool:
    if not os.path.exists(BINDING_PATH):
        return True
    t = os.path.getmtime(BINDING_PATH)
    return any(os.path.getmtime(d) > t
               for d in (BINDING_SOURCE, os.path.join(ROOT, "include", "nvfp4.h")))


def _build_binding(verbose: bool) -> None:
    """g++ against torch's headers.  The C entry points stay undefined here: the
    library is loaded first, with its symbols visible."""
    base = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = BINDING_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           *(f"-I{d}" for d in (os.path.join(base, "include"),
                                os.path.join(base, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], os.path.join(cuda, "include"))),
           BINDING_SOURCE, "-o", tmp, f"-L{os.path.join(base, 'lib')}",
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on binding.cpp")
    os.replace(tmp, BINDING_PATH)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library if needed; returns its path."""
    if force or _stale():
        os.makedirs(OUT_DIR, exist_ok=True)
        _build_library(verbose)
    return LIB_PATH


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compiles the binding if needed; returns its path.  It alone needs g++ and the
    headers of Python and torch."""
    if force or _binding_stale():
        os.makedirs(OUT_DIR, exist_ok=True)
        _build_binding(verbose)
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library and, beside it, the binding if needed; returns the
    library's path."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        job = ex.submit(build_binding, force, verbose)
        build_library(force, verbose)
        job.result()
    return LIB_PATH


def _build_library(verbose: bool) -> None:
    nvcc = _nvcc()
    objs = [os.path.join(OUT_DIR, s.replace(".cu", ".o")) for s in SOURCES]

    def compile_one(i):
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, SOURCES[i]), "-o", objs[i]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, range(len(SOURCES))))
    for cmd, r in results:
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", tmp, *objs,
           "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
