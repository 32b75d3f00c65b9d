"""Build the CUDA library libdiffattn_v2.so in place (sm_100a).

    python -m differential_attention_v2_b200.build [--force] [--verbose] [--debug-bounds]

Compiles every kernel and the C ABI with nvcc for sm_100a into one shared library that
sits next to this file, where the Python binding loads it. nvcc cross-compiles, so this
runs on machines without a GPU. Rebuilds only when a source is newer than the library.

--debug-bounds also builds libdiffattn_v2_debug.so: the same library compiled with
-DDA2_DEBUG_BOUNDS, in which the kernels check their shared-memory, tensor-memory and global
indices against the extents they address and report a violation through the device error
word (code 4) instead of making the access. The tests load it directly.

The library's Python binding has a native half, _native.so (csrc/binding.cpp, compiled with g++
against torch's headers), which the same command builds after the library. The library itself needs
neither torch nor Python's headers: where the native half cannot be built, a warning says so, the
library is there, and the binding's entry points that do not go through the native half work.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_NAME = "libdiffattn_v2.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
DEBUG_LIB_PATH = os.path.join(PKG, "libdiffattn_v2_debug.so")
NATIVE_PATH = os.path.join(PKG, "_native.so")
NATIVE_STAMP_PATH = os.path.join(PKG, "_native.stamp")  # what _native.so was built for
NATIVE_SOURCE = os.path.join(CSRC, "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + [
        os.path.join(ROOT, "include", "diffattn_v2.h"), os.path.abspath(__file__)]


def up_to_date(path=LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libdiffattn_v2.so")
    return exe


def build(force: bool = False, verbose: bool = False, extra_flags=None, debug_bounds: bool = False) -> str:
    """Build the library (or, with debug_bounds, its bounds-checking twin); returns its path."""
    out = DEBUG_LIB_PATH if debug_bounds else LIB_PATH
    if debug_bounds:
        extra_flags = list(extra_flags or []) + ["-DDA2_DEBUG_BOUNDS"]
    if force or not up_to_date(out):
        _compile(out, verbose, extra_flags)
    if not debug_bounds:
        try:
            build_native(force=force, verbose=verbose)
        except (RuntimeError, ImportError, OSError) as e:
            warnings.warn(f"{out} is built, but not the Python binding's native half, which its sink, rotary and cache "
                          f"calls need: {e}", stacklevel=2)
    return out


def _compile(out, verbose, extra_flags):
    tmp = out + ".tmp"
    cmd = [nvcc()] + NVCC_FLAGS + list(extra_flags or []) + ["-I", os.path.join(ROOT, "include"), "-o", tmp] + _sources()
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr)
    os.replace(tmp, out)


def native_stamp() -> str:
    """The interpreter and torch whose ABIs _native.so has to match."""
    import torch

    return f"python {sys.implementation.cache_tag} {sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def native_built_for() -> str:
    """native_stamp() of the build that made _native.so ("": there is none, or it does not say)."""
    if not os.path.exists(NATIVE_PATH) or not os.path.exists(NATIVE_STAMP_PATH):
        return ""
    with open(NATIVE_STAMP_PATH) as f:
        return f.read()


def build_native(force: bool = False, verbose: bool = False) -> str:
    """Build _native.so, the native half of the Python binding (g++ against torch's headers), if a
    source is newer or it was built for another interpreter or torch."""
    made_from = (NATIVE_SOURCE, os.path.abspath(__file__))
    stamp = native_stamp()
    if not force and native_built_for() == stamp and all(
            os.path.getmtime(p) <= os.path.getmtime(NATIVE_PATH) for p in made_from):
        return NATIVE_PATH
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    tmp = NATIVE_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for p in include for x in ("-isystem", p)] + [NATIVE_SOURCE, "-o", tmp, "-L", os.path.join(torch_dir, "lib")]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, NATIVE_PATH)
    with open(NATIVE_STAMP_PATH, "w") as f:
        f.write(stamp)
    return NATIVE_PATH


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true", help="print register and spill counts")
    ap.add_argument("--debug-bounds", action="store_true", help="also build the bounds-checking library")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_verbose else []
    path = build(force=a.force or a.ptxas_verbose, verbose=a.verbose or a.ptxas_verbose, extra_flags=extra)
    print(path)
    if a.debug_bounds:
        print(build(force=a.force, verbose=a.verbose, extra_flags=extra, debug_bounds=True))


if __name__ == "__main__":
    sys.exit(main())
