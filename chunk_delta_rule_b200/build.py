"""Builds the in-tree CUDA library ``libcomba.so`` for sm_100a with nvcc.

``python -m chunk_delta_rule_b200.build`` (or ``build()``) recompiles when any
source or the public header is newer than the library.  The library links the
CUDA runtime statically and resolves driver entry points at run time, so it
loads on a machine without a GPU driver (compute calls then fail with
COMBA_ECUDA)."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcomba.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    # each .cu is a translation unit of its own; they compile side by side
    cmds, objs = [], []
    for cu in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        objs.append(f"{tmp}.{os.path.basename(cu)}.o")
        cmd = [_nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", "-o", objs[-1], cu]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        cmds.append(cmd)
    try:
        running = [subprocess.Popen(cmd) for cmd in cmds]
        for cmd, rc in zip(cmds, [p.wait() for p in running]):
            if rc != 0:
                raise subprocess.CalledProcessError(rc, cmd)
        subprocess.check_call([_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
