"""Build libmssm.so in-tree with nvcc for sm_100a.

    python selective_state_space_46_b200/build.py [--force] [--verbose] [extra nvcc flags]

Run this file directly (or load it by path): importing it through the package
would load the library it is meant to build.

Each .cu file is compiled to an object in parallel, then linked into a shared
library next to this file.  The CUDA runtime is linked statically, so loading
the library needs no GPU (only calling into it does).  The Python binding's
descriptor writer (csrc/marshal.cpp) becomes _marshal.so beside it; where that
cannot be built (it takes a C++ compiler and a torch with CUDA), the library still
is, and every operator that does not use it runs.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmssm.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", *ARCH,
              f"-I{INCLUDE}", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libmssm.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + [os.path.join(INCLUDE, "mssm.h"), os.path.abspath(__file__)]


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """The binding's descriptor writer: a CPython extension against the installed torch's headers."""
    import sysconfig
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    inputs = [MARSHAL_SRC, os.path.join(INCLUDE, "mssm.h"), os.path.abspath(__file__), os.path.join(base, "version.py")]
    if not force and os.path.exists(MARSHAL) and all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL) for p in inputs):
        return MARSHAL
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{INCLUDE}", f"-I{base}/include",
           f"-I{base}/include/torch/csrc/api/include", f"-I{os.path.dirname(os.path.dirname(_nvcc()))}/include",
           f"-I{sysconfig.get_paths()['include']}",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", MARSHAL_SRC, "-o", tmp,
           f"-L{base}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building _marshal.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    return MARSHAL


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def compile_objects(force: bool = False, verbose: bool = False, extra_flags=()) -> list:
    """Compiles every source whose object is missing or out of date; returns all objects."""
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    srcs = sources()
    headers = [p for p in _inputs() if not p.endswith(".cu")]
    newest_header = max((os.path.getmtime(p) for p in headers), default=0.0)

    def stale(src):
        # an object is rebuilt when its source, any header or this script is newer than it,
        # or when extra flags are given (they may change the code)
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        if force or extra_flags or not os.path.exists(obj):
            return True
        return os.path.getmtime(obj) < max(os.path.getmtime(src), newest_header)

    todo = [src for src in srcs if stale(src)]
    with ThreadPoolExecutor(max_workers=max(1, min(len(todo), os.cpu_count() or 1))) as ex:
        list(ex.map(compile_one, todo))
    return [os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o")) for src in srcs]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if force or not up_to_date():
        link(compile_objects(force, verbose, extra_flags), verbose)
    try:
        build_marshal(force, verbose)
    except (RuntimeError, ImportError, OSError) as e:  # no C++ compiler, or no torch with CUDA and its headers
        warnings.warn(f"the library is built, but the gated recurrence and the 4-bit linear map need _marshal.so from Python: {e}")
    return LIB


def link(objs, verbose: bool = False) -> str:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    args = sys.argv[1:]
    extra = [a for a in args if a not in ("--force", "--verbose")]
    print(build(force="--force" in args, verbose="--verbose" in args, extra_flags=extra))

