"""Build libssmscan.so in-tree with nvcc for sm_100a (B200).

Run as ``python -m selective_state_space_51_b200.build`` or call ``build()``.
The library is written next to this file so that it travels with the source
tree; nothing is installed elsewhere. Every .cu file is compiled into an
object of its own, at the same time, and only if it, a header it includes, the
flags or the compiler have changed.
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


def _key(extra=()):
    """What an object or the library is built with, apart from its sources:
    kept in a file of its name among the objects. None without a compiler
    (what is there is then taken by its date)."""
    try:
        nvcc = _nvcc()
    except RuntimeError:
        return None
    version = subprocess.run([nvcc, "--version"], check=True, text=True,
                             capture_output=True).stdout
    return "\n".join([nvcc, version, *NVCC_FLAGS, *extra])


def _key_file(path):
    return os.path.join(OBJECTS, os.path.basename(path) + ".key")


def _built_with(path, key) -> bool:
    if key is None:
        return True
    try:
        with open(_key_file(path)) as f:
            return f.read() == key
    except OSError:
        return False


def _place(tmp, path, key) -> None:
    """Moves a finished file to its place. It has its key last: a build that
    ends in between leaves none."""
    if os.path.exists(_key_file(path)):
        os.remove(_key_file(path))
    os.replace(tmp, path)
    with open(_key_file(path), "w") as f:
        f.write(key)


def _stale(key) -> bool:
    if not os.path.exists(LIB) or not _built_with(LIB, key):
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


def _object(src, force, verbose, extra, key):
    obj = os.path.join(OBJECTS, os.path.basename(src)[:-3] + ".o")
    if not force and os.path.exists(obj) and _built_with(obj, key) and all(
            os.path.getmtime(d) <= os.path.getmtime(obj)
            for d in _included(src)):
        return obj
    tmp = obj + ".tmp.%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-I", INCLUDE, "-c", "-o", tmp, src]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    _place(tmp, obj, key)
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Compile every .cu under csrc/ and link one shared library; `extra`:
    more flags for the compiler."""
    key = _key(extra)
    if not force and not _stale(key):
        return LIB
    os.makedirs(OBJECTS, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        objects = list(pool.map(
            lambda s: _object(s, force, verbose, tuple(extra), key),
            sources()))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objects]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    _place(tmp, LIB, key)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
