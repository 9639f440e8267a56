"""Build ``libfp8attn.so`` in-tree with nvcc for sm_100a (B200), and beside it
the small CPython module ``_calls`` (gcc) through which the binding makes the
calls that take only microseconds.  The library needs nvcc alone; the module
needs Python's headers, and is left out with a warning where there are none.

    python -m quantization_amax_reduce_b200.build [--force] [--verbose]

The library links the CUDA runtime statically and resolves the driver's
tensor-map encoder at run time, so it needs no libcuda at link time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["api.cu", "quant.cu", "attention.cu", "regroup.cu", "scale_map.cu",
           "kv_cache.cu", "kv_tree.cu"]
HEADERS = ["kernels.h", "kv_tree.cuh", "sm100_ptx.cuh", "state.cuh"]
LIB = os.path.join(HERE, "libfp8attn.so")
CALLS_SRC = os.path.join(CSRC, "calls.c")
CALLS = os.path.join(HERE, "_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _older(target: str, deps) -> bool:
    return not os.path.exists(target) or \
        any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    return _older(LIB, deps + [os.path.join(ROOT, "include", "fp8attn.h")])


def _build_calls(force: bool) -> None:
    if not force and not _older(CALLS, [CALLS_SRC, os.path.join(ROOT, "include", "fp8attn.h")]):
        return
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        # (nothing but the paged cache's Python functions needs it)
        warnings.warn("no Python.h: _calls is not built; without it kv_assign_pages, kv_write, "
                      "kv_tree_fwd and kv_keep_path raise an error in Python")
        return
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if not cc:
        raise RuntimeError("no C compiler found")
    tmp = CALLS + ".tmp"
    subprocess.check_call([cc, "-O2", "-shared", "-fPIC", "-Wall", "-I",
                           sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"),
                           CALLS_SRC, "-o", tmp])
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library first: it needs neither Python's headers nor the module."""
    if force or _stale():
        _build_lib(verbose)
    _build_calls(force)
    return LIB


def _build_lib(verbose: bool) -> None:
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    common = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                     "-I", os.path.join(ROOT, "include")]
    if verbose:
        common += ["-Xptxas", "-v"]
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc()] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.check_call([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
