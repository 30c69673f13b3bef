"""Build libdgb200.so in-tree with nvcc for sm_100a.

    python -m moe_grouped_gemm_tcgen05_b200.build [--force]

Every .cu file is compiled to an object of its own under _build/ (in parallel,
and only when a source it may include is newer), and the objects are linked.
The library is rebuilt only when a source or the public header is newer than
the shared object.
"""

from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdgb200.so")
OBJECTS = os.path.join(PKG, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdgb200.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + _headers()


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [
        os.path.join(INCLUDE, "dgb200.h")
    ]


def _included(path):
    """The files that a source includes with quotes, itself and those they include among them."""
    found, todo = set(), [path]
    by_name = {os.path.basename(h): h for h in _headers()}
    while todo:
        p = todo.pop()
        if p in found:
            continue
        found.add(p)
        with open(p, encoding="utf-8") as f:
            todo += [by_name[n] for n in re.findall(r'#include "([^"]+)"', f.read()) if n in by_name]
    return found


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    objects, running = [], []
    os.makedirs(OBJECTS, exist_ok=True)
    for cu in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(OBJECTS, os.path.basename(cu)[:-3] + ".o")
        objects.append(obj)
        if not force and os.path.exists(obj) and all(os.path.getmtime(s) <= os.path.getmtime(obj) for s in _included(cu)):
            continue
        cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", cu, "-o", obj + ".tmp"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        running.append((subprocess.Popen(cmd), cmd, obj))
    failed = [cmd for p, cmd, _ in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, obj in running:
        os.replace(obj + ".tmp", obj)
    tmp = LIB + ".tmp"
    subprocess.run([_nvcc(), *NVCC_FLAGS, "-shared", *objects, "-o", tmp], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
