"""Build the CUDA library ``libmoe_b200.so`` in-tree with nvcc for sm_100a.

Usage: ``python -m mixture_experts_ffn_14_b200.build [--force] [--verbose] [--debug-bounds]``.
Objects go to ``mixture_experts_ffn_14_b200/_build/`` and are rebuilt when a
source or header is newer than the object. Cross-compiles without a GPU.

``--debug-bounds`` builds ``libmoe_b200_debug.so`` from the same sources with
``-DMOE_DEBUG_BOUNDS`` (objects in ``_build_debug/``): every index that one kernel of
the sublayer or of its expert-parallel pieces computes and another uses is checked
before the access, a failed check sets status bit 0x40 and skips the access. (The
kernels of the top-k routing, combine and int8 calls have no such checks; what a caller
gives them is checked in every build.) Load it with
``MOE_B200_LIBRARY=libmoe_b200_debug.so``.

``build_torch_calls`` compiles ``_torch_calls.so`` (csrc/torch_calls.cpp), the binding of
the routing, combine and int8 calls, against the installed torch's headers; again when
torch or Python is another one than it was compiled for.
"""

from __future__ import annotations

import argparse
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libmoe_b200_debug.so")
TORCH_CALLS = os.path.join(PKG, "_torch_calls.so")
TORCH_CALLS_TAG = os.path.join(BUILD, "torch_calls.tag")  # torch and Python that it was compiled for

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_b200.so")
    return cand


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, debug_bounds: bool = False) -> str:
    build_dir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug_bounds else (BUILD, LIB)
    flags = NVCC_FLAGS + (["-DMOE_DEBUG_BOUNDS"] if debug_bounds else [])
    os.makedirs(build_dir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    objs = []
    for src in srcs:
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or ptxas_info or _stale(obj, [src] + hdrs):
            cmd = [nvcc()] + flags + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
    if force or _stale(lib, objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", lib] + objs + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    return lib


def _torch_tag() -> str:
    return f"torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('SOABI')}"


def build_torch_calls(force: bool = False, verbose: bool = False) -> str:
    src = os.path.join(CSRC, "torch_calls.cpp")
    built_for = ""
    if os.path.exists(TORCH_CALLS_TAG):
        with open(TORCH_CALLS_TAG) as f:
            built_for = f.read().strip()
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: its headers are required to build _torch_calls.so")
    if not force and built_for == _torch_tag() and not _stale(TORCH_CALLS, [src] + _headers()):
        return TORCH_CALLS
    import torch

    home = os.path.dirname(spec.origin)
    include = os.path.join(home, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    cmd += ["-I" + d for d in (os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], include,
                               os.path.join(include, "torch", "csrc", "api", "include"), cuda)]
    cmd += [src, "-o", TORCH_CALLS, "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.makedirs(os.path.dirname(TORCH_CALLS_TAG), exist_ok=True)
    with open(TORCH_CALLS_TAG, "w") as f:
        f.write(_torch_tag() + "\n")
    return TORCH_CALLS


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    ap.add_argument("--debug-bounds", action="store_true",
                    help="build libmoe_b200_debug.so with the device-side index checks")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info, debug_bounds=a.debug_bounds))
    print(build_torch_calls(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
