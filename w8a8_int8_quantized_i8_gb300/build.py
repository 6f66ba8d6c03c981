"""Builds libi8.so (the CUDA library behind include/i8.h) in-tree with nvcc,
and beside it libi8probe.so, a measurement helper for the benchmark (the
legacy warp MMA's int8 and fp16 rates; not part of the W8A8 path).

libi8.so is two translation units (the linear layer, the serving operators),
the probe one; one ``-gencode`` target (sm_103a), no cmake; all three compile
in parallel.  The outputs are git-ignored and rebuilt whenever a source is
newer than them.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libi8.so")
UNITS = [os.path.join(CSRC, "i8_api.cu"), os.path.join(CSRC, "serving_api.cu")]
PROBE_LIB = os.path.join(PKG, "libi8probe.so")
PROBE_SRC = os.path.join(CSRC, "engine_probe.cu")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    # IEEE fp32 behaviour (nvcc's defaults, stated so no flag set can drop
    # them): no flush to zero, correctly rounded division and square root
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libi8")


def _sources():
    return ([s for s in glob.glob(os.path.join(CSRC, "*.cu")) if s != PROBE_SRC]
            + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "i8.h")])


def _stale(lib, sources) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(s) > t for s in sources)


def stale() -> bool:
    return _stale(LIB, _sources()) or _stale(PROBE_LIB, [PROBE_SRC])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libi8.so and libi8probe.so if missing or older than their sources."""
    targets = []
    if force or _stale(LIB, _sources()):
        targets.append((LIB, UNITS))
    if force or _stale(PROBE_LIB, [PROBE_SRC]):
        targets.append((PROBE_LIB, [PROBE_SRC]))

    def start(cmd):
        if verbose:
            print(" ".join(cmd))
        return subprocess.Popen(cmd)

    jobs = []
    for lib, units in targets:
        objects = [f"{lib}.{os.path.basename(u)}.tmp{os.getpid()}.o" for u in units]
        jobs.append((lib, objects, [start([nvcc(), *NVCC_FLAGS, "-c", "-o", o, u])
                                    for o, u in zip(objects, units)]))
    failed = []
    for lib, objects, procs in jobs:
        ok = all([p.wait() == 0 for p in procs])
        tmp = f"{lib}.tmp{os.getpid()}"
        if ok and start([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objects]).wait() == 0:
            os.replace(tmp, lib)
        else:
            failed.append(os.path.basename(lib))
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    if failed:
        raise RuntimeError(f"nvcc failed building {', '.join(failed)}")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
