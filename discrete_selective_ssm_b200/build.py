"""Builds libnaju.so (the C-ABI CUDA library) in-tree for sm_100a.

    python -m discrete_selective_ssm_b200.build [--force]

nvcc compiles every ``csrc/*.cu`` to an object file (in parallel, under
``_build/`` at the repository root) and links them into one shared library
next to this file; the build is skipped when the library is newer than all
sources and headers, and an object is recompiled only when it is older than
its source or any header.  That needs nvcc alone: the C ABI has no part of
Python in it.  ``build_bind`` compiles ``csrc/naju_bind.cpp``, the compiled
part of the Python binding, with g++ against the running Python and the
installed torch, whose names the file carries.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libnaju.so")
BIND_SRC = os.path.join(CSRC, "naju_bind.cpp")
OBJDIR = os.path.join(ROOT, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the Naju CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return [f for d, pat in ((CSRC, "*.h*"), (CSRC, "*.cuh"), (INCLUDE, "*.h"))
            for f in glob.glob(os.path.join(d, pat))]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in sources() + _headers())


def _obj(src: str) -> str:
    return os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")


def _compile(src: str, force: bool, verbose: bool) -> str:
    obj = _obj(src)
    if not force and os.path.exists(obj):
        t = os.path.getmtime(obj)
        if all(os.path.getmtime(f) <= t for f in [src] + _headers()):
            return obj
    tmp = obj + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-c",
           "-I", INCLUDE, "-I", CSRC, "-o", tmp, src]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, obj)
    return obj


def bind_path() -> str:
    """Where the compiled part of the Python binding is kept: one file for each
    Python ABI and torch version, since it is of use to those alone."""
    torch = importlib.metadata.version("torch")
    return os.path.join(HERE, f"_naju_bind.{sysconfig.get_config_var('SOABI')}.torch{torch}.so")


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """The compiled part of the Python binding (an extension module)."""
    bind = bind_path()
    deps = [BIND_SRC, os.path.join(INCLUDE, "naju.h")]
    if not force and os.path.exists(bind) and all(
            os.path.getmtime(f) <= os.path.getmtime(bind) for f in deps):
        return bind
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = bind + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-I", os.path.join(torch, "include"),
           "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-o", tmp, BIND_SRC, "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, bind)
    return bind


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sources()
    # the largest translation units first, so they do not finish last
    srcs.sort(key=os.path.getsize, reverse=True)
    workers = max(1, min(len(srcs), os.cpu_count() or 1))
    with concurrent.futures.ThreadPoolExecutor(workers) as ex:
        objs = list(ex.map(lambda f: _compile(f, force, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([_nvcc(), *ARCH, "-shared", "-o", tmp, *sorted(objs)])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    how = {"force": "--force" in sys.argv, "verbose": "-v" in sys.argv}
    print(build(**how), flush=True)
    if importlib.util.find_spec("torch") is not None:
        print(build_bind(**how))
