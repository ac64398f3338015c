"""Build libkd.so (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: ``python -m chunked_kl_loss_chunk_b200.build`` (or ``build()``).
The library is written next to this file so it travels with the repository, and
beside it _kd_native.so, the C++ half of the Python binding (torch's headers, g++).
``--lib-only`` (``build(native=False)``) leaves that out, for programs in C: kd.py
then makes every call through ctypes.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libkd.so")
# Same sources with the device-side invariant checks on (-DKD_DEBUG=1): a failed
# check records KD_ERR_INTERNAL in the workspace's status word.
DEBUG_LIB_PATH = os.path.join(PKG_DIR, "libkd_debug.so")
NATIVE_SRC = os.path.join(CSRC, "kd_native.cpp")
NATIVE_PATH = os.path.join(PKG_DIR, "_kd_native.so")
# what the module was last built for: its file's time does not tell an upgrade of torch or Python
NATIVE_STAMP = os.path.join(ROOT, "_build", "_kd_native.built_for")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(INCLUDE, "kd.h")]


def up_to_date(debug: bool = False) -> bool:
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in deps())


def _built_for() -> str:
    """The Python and torch whose ABI the module is compiled against."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return f"python {'.'.join(map(str, sys.version_info[:3]))}, torch {torch.__version__}, cxx11 abi {abi}\n"


def native_up_to_date() -> bool:
    newest = max(os.path.getmtime(p) for p in (NATIVE_SRC, os.path.join(INCLUDE, "kd.h")))
    if not os.path.exists(NATIVE_PATH) or os.path.getmtime(NATIVE_PATH) < newest:
        return False
    if not os.path.exists(NATIVE_STAMP):
        return False
    with open(NATIVE_STAMP) as f:
        return f.read() == _built_for()


def build_native(force: bool = False, verbose: bool = False) -> str:
    """Compile _kd_native.so against the installed torch; returns its path."""
    if not force and native_up_to_date():
        return NATIVE_PATH
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = NATIVE_PATH + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in (INCLUDE, os.path.join(home, "include"), os.path.join(cuda, "include"),
                                sysconfig.get_paths()["include"])),
           NATIVE_SRC, "-o", tmp, "-L" + os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, NATIVE_PATH)
    os.makedirs(os.path.dirname(NATIVE_STAMP), exist_ok=True)
    with open(NATIVE_STAMP, "w") as f:
        f.write(_built_for())
    return NATIVE_PATH


def build(force: bool = False, verbose: bool = False, debug: bool = False, native: bool = True) -> str:
    """Compile every CUDA source into one shared library; returns its path.
    ``debug`` builds libkd_debug.so, with the device-side invariant checks;
    ``native=False`` leaves out the C++ half of the Python binding."""
    lib = _build_lib(force, verbose, debug)
    if native:
        build_native(force and not debug, verbose)
    return lib


def _build_lib(force: bool, verbose: bool, debug: bool) -> str:
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    if not force and up_to_date(debug):
        return lib
    nvcc = _nvcc()
    objdir = os.path.join(ROOT, "_build", "debug" if debug else "")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *(["-DKD_DEBUG=1"] if debug else []), "-I" + INCLUDE, "-c", src,
               "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = lib + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-cudart", "static"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv,
                native="--lib-only" not in sys.argv))
