"""Builds libminf.so in-tree with nvcc for sm_100a.

Usage: ``python -m dynamic_sparse_attention_minf_b200.build [--verbose]``.
The library lands next to this file, where the Python binding loads it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["api.cu", "attn.cu", "bs_select.cu", "estimate.cu", "estimate_tc.cu", "grid.cu", "index.cu", "kv_cache.cu",
           "noalloc.cu", "rope.cu", "selftest.cu", "serve_api.cu", "tree_attn.cu", "tree_wide.cu"]
LIB = os.path.join(HERE, "libminf.so")
BINDING = os.path.join(HERE, "_binding.so")   # Python binding of the serving entry points (binding.cpp)
BUILD_DIR = os.path.join(ROOT, "_build")


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "minf.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = nvcc_path()
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-lineinfo",
             "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("nvcc link failed")
    os.replace(tmp, LIB)
    _build_binding(verbose)
    return LIB


def _build_binding(verbose: bool) -> None:
    """The extension module, linked against libminf.so beside it."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    tmp = BINDING + ".tmp"
    inc = [f for d in ext.include_paths() + [os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"),
                                             sysconfig.get_paths()["include"]] for f in ("-isystem", d)]
    libs = [f for d in ext.library_paths() for f in ("-L", d)]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_binding",
           *inc, os.path.join(CSRC, "binding.cpp"), "-o", tmp, *libs, "-L", HERE, "-l:libminf.so", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on binding.cpp")
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force=True))
