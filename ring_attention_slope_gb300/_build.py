"""Builds ``libslope.so`` (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a, and
``_marshal.so``, the Python binding's argument marshalling in C.

Translation units are compiled in parallel and linked into one shared
library next to this file.  The library is rebuilt only when a source or
header is newer than it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libslope.so")
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")

SOURCES = ["attn_partial.cu", "kv4_attn.cu", "api.cu", "lse_merge.cu", "qk_norm_rope.cu", "kv4_store.cu", "status.cu",
           "dck.cpp", "rope.cpp"]
HEADERS = ["host.cuh", "kernels.cuh", "kv4.cuh", "sm103_ptx.cuh", "waits.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libslope")
    return path


def _stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(MARSHAL_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(MARSHAL_PATH))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + ["marshal.c"]]
    deps += [os.path.join(INCLUDE, f) for f in ("slope.h", "slope_serving.h")] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit for sm_103a and link ``libslope.so``; returns its path."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    def compile_marshal():
        tmp = MARSHAL_PATH + f".tmp{os.getpid()}"
        cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-Wextra", "-shared", "-fPIC", "-fvisibility=hidden",
               "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, os.path.join(CSRC, "marshal.c"), "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for marshal.c:\n{r.stdout}\n{r.stderr}")
        return tmp

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        marshal = ex.submit(compile_marshal)
        objs = list(ex.map(compile_one, SOURCES))
    os.replace(marshal.result(), MARSHAL_PATH)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
