"""Builds ``libslope.so`` (the CUDA kernels and the C ABI) in-tree with nvcc for sm_103a, and
``_marshal``, the Python binding's argument marshalling in C.

Translation units are compiled in parallel and linked into one shared
library next to this file.  Each is rebuilt only when a source or
header is newer than it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libslope.so")
# named after the interpreter whose headers it is compiled with: another one finds none and builds its own
MARSHAL_PATH = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))

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


def _stale(path, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in deps)


def _include(*names):
    return [os.path.join(INCLUDE, f) for f in names]


def _compile_marshal():
    """Compiles marshal.c for this interpreter, which has to have its headers installed."""
    tmp = MARSHAL_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-Wall", "-Wextra", "-shared", "-fPIC", "-fvisibility=hidden",
           "-I", sysconfig.get_paths()["include"], "-I", INCLUDE, os.path.join(CSRC, "marshal.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for marshal.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL_PATH)


def _compile_library(verbose):
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

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit for sm_103a and link ``libslope.so``; returns its path.

    The library needs nothing of Python.  Where the argument marshalling cannot be compiled (no ``Python.h``, say),
    the library is built all the same, with a warning; the calls that go through the marshalling then raise."""
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + _include("slope.h", "slope_serving.h") + [__file__]
    if force or _stale(LIB_PATH, deps):
        _compile_library(verbose)
    deps = [os.path.join(CSRC, "marshal.c")] + _include("slope.h", "slope_serving.h") + [__file__]
    if force or _stale(MARSHAL_PATH, deps):
        try:
            _compile_marshal()
        except (OSError, RuntimeError) as e:
            if os.path.exists(MARSHAL_PATH):
                os.remove(MARSHAL_PATH)  # of older sources: not for this library
            warnings.warn(f"libslope is built without its Python marshalling: {e}", stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
