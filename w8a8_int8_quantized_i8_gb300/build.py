"""Builds libi8.so (the CUDA library behind include/i8.h) in-tree with nvcc,
and beside it libi8probe.so, a measurement helper for the benchmark (the
legacy warp MMA's int8 and fp16 rates; not part of the W8A8 path), and _calls.*.so,
the CPython extension that hands torch tensors to libi8 where a small call's time
is the host's (csrc/torch_calls.cpp).  Only the calls that go through the extension
need it, and g++ and torch's headers with it.

libi8.so is three translation units (the linear layer, the serving operators,
the 4-bit route), the probe and the extension one each; one ``-gencode`` target
(sm_103a), no cmake; all of them compile in parallel.  The outputs are git-ignored and rebuilt whenever a source is
newer than them.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libi8.so")
UNITS = [os.path.join(CSRC, name) for name in ("i8_api.cu", "serving_api.cu", "fp4_api.cu")]
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
# (its name has what its binary interface depends on: another Python or torch builds its own)
CALLS_LIB = os.path.join(PKG, f"_calls.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")
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


def _calls_sources():
    return [CALLS_SRC, os.path.join(ROOT, "include", "i8.h")]


def stale(calls: bool = True) -> bool:
    return (_stale(LIB, _sources()) or _stale(PROBE_LIB, [PROBE_SRC])
            or (calls and _stale(CALLS_LIB, _calls_sources())))


def _calls_compile(obj: str) -> list[str]:
    """Compiles the extension against this torch and this Python."""
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-c", "-o", obj, CALLS_SRC]


def _calls_link(out: str, obj: str) -> list[str]:
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L", PKG, "-l:libi8.so", "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, calls: bool = True) -> str:
    """Compile libi8.so, libi8probe.so and, with ``calls``, the extension if missing or older
    than their sources.  An extension that does not compile leaves the libraries built."""
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
    obj = proc = None
    if calls and (force or _stale(CALLS_LIB, _calls_sources())):
        obj = f"{CALLS_LIB}.tmp{os.getpid()}.o"
        try:
            proc = start(_calls_compile(obj))
        except OSError as e:    # no compiler
            print(e, file=sys.stderr)
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
    if obj:
        tmp = f"{CALLS_LIB}.tmp{os.getpid()}"
        if proc and proc.wait() == 0 and not failed and start(_calls_link(tmp, obj)).wait() == 0:
            os.replace(tmp, CALLS_LIB)
        else:
            failed.append(os.path.basename(CALLS_LIB))
        if os.path.exists(obj):
            os.remove(obj)
    if failed:
        raise RuntimeError(f"the compiler failed building {', '.join(failed)}")
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
