"""Build the in-tree C-ABI library ``libflce.so`` for sm_100a with nvcc, and ``_marshal.so``, the
binding's host helper, with g++ against torch's headers.

    python -m lm_head_linear_gemm_b200.build [--verbose-ptxas]
    FLCE_BUILD_DEFINES="-DFLCE_DW_GROUPS=2" python -m lm_head_linear_gemm_b200.build --force

The library is written next to this file so that it travels with the source tree;
nothing is installed into site-packages.
"""
from __future__ import annotations

import argparse
import os
import shlex
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libflce.so")
SOURCES = [os.path.join(CSRC, f) for f in ("flce_api.cu", "flce_train.cu")]
HEADERS = [os.path.join(CSRC, f) for f in ("sm100.cuh", "gemm.cuh", "rowwise.cuh", "host.h",
                                           "packed.cuh", "qk_norm.cuh", "optim.cuh")] + [
    os.path.join(ROOT, "include", f) for f in ("flce.h", "flce_train.h")]

MARSHAL_PATH = os.path.join(HERE, "_marshal.so")
MARSHAL_SOURCES = [os.path.join(CSRC, "marshal.cpp"), os.path.join(ROOT, "include", "flce.h"),
                   os.path.join(ROOT, "include", "flce_train.h")]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA 12.9 toolkit is required to build libflce.so")


def nvcc_flags(verbose_ptxas: bool = False) -> list[str]:
    flags = [
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-O3", "-lineinfo", "-std=c++17",
        "-Xcompiler", "-fPIC", "-shared",
        "--expt-relaxed-constexpr",
        "--threads", "0",                      # the sources side by side
        "-I", os.path.join(ROOT, "include"),
    ]
    if verbose_ptxas:
        flags += ["-Xptxas", "-v"]
    # build-time tuning constants of flce_api.cu (e.g. "-DFLCE_DW_GROUPS=2"), for measurements
    flags += os.environ.get("FLCE_BUILD_DEFINES", "").split()
    return flags


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in SOURCES + HEADERS)


def marshal_built_for() -> str:
    """What the helper is good for: it uses torch's C++ interface (internal parts of it too, tried
    with torch 2.11), which no other version need share, and Python's."""
    import torch
    return f"built for torch {torch.__version__}, {sys.implementation.cache_tag}"


def marshal_is_stale() -> bool:
    if not os.path.exists(MARSHAL_PATH) or \
            os.path.getmtime(MARSHAL_PATH) < max(map(os.path.getmtime, MARSHAL_SOURCES)):
        return True
    with open(MARSHAL_PATH, "rb") as f:                  # the module's attribute `built_for`
        return marshal_built_for().encode() + b"\0" not in f.read()


def build_marshal(force: bool = False, quiet: bool = False) -> str:
    """The host helper of the binding: a CPython module on torch's C++ headers (no kernels)."""
    if not force and not marshal_is_stale():
        return MARSHAL_PATH
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cxx = shlex.split(os.environ.get("CXX", "")) or ["g++"]  # may be several words ("ccache g++")
    if shutil.which(cxx[0]) is None:
        raise RuntimeError(f"{cxx[0]}: compiler not found; g++ (or CXX) builds _marshal.so")
    tmp = MARSHAL_PATH + ".tmp"
    cmd = [*cxx, "-O2", "-std=c++17", "-fPIC", "-shared",
           f'-DFLCE_MARSHAL_BUILT_FOR="{marshal_built_for()}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(base, "include"),
           "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"),
           MARSHAL_SOURCES[0], "-o", tmp, "-L", os.path.join(base, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    if not quiet:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MARSHAL_PATH)
    return MARSHAL_PATH


def build_library(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    """``libflce.so``: needs nvcc alone."""
    if not force and not is_stale():
        return LIB_PATH
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc_path()] + nvcc_flags(verbose_ptxas) + ["-o", tmp] + SOURCES
    if not quiet:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas or (res.stderr.strip() and not quiet):
        print(res.stderr, file=sys.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    """Both.  The library comes first: C callers use it without the binding's helper, which needs
    torch's C++ headers."""
    path = build_library(force, verbose_ptxas, quiet)
    build_marshal(force, quiet)
    return path


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
