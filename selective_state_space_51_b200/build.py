"""Build libssmscan.so in-tree with nvcc for sm_100a (B200).

Run as ``python -m selective_state_space_51_b200.build`` or call ``build()``.
The library is written next to this file so that it travels with the source
tree; nothing is installed elsewhere. Every .cu file is compiled into an
object of its own, at the same time, and only if it or a header it includes
has changed.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJECTS = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libssmscan.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-cudart", "static",
]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))
    return any(os.path.getmtime(d) > t for d in deps)


def _included(path, seen=None):
    """`path` and every file it includes by a quoted name."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    with open(path) as f:
        names = re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M)
    for n in names:
        _included(os.path.join(os.path.dirname(path), n), seen)
    return seen


def _object(src, force, verbose, extra):
    obj = os.path.join(OBJECTS, os.path.basename(src)[:-3] + ".o")
    if not force and not extra and os.path.exists(obj) and all(
            os.path.getmtime(d) <= os.path.getmtime(obj)
            for d in _included(src)):
        return obj
    tmp = obj + ".tmp.%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", "-o", tmp, src]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every .cu under csrc/ and link one shared library."""
    if not force and not _stale():
        return LIB
    os.makedirs(OBJECTS, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objects = list(pool.map(
            lambda s: _object(s, force, verbose, tuple(extra)), sources()))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objects]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
