"""Builds libfa_gb300.so (the C-ABI library of include/fa.h) for sm_103a.

Each CUDA source is compiled by nvcc in parallel into ``_build/``, then linked
into ``libfa_gb300.so`` next to this file (in-tree; git-ignored).  Usage:
``python -m attention_backward_preprocess_gb300.build`` or ``build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa_gb300.so")
SOURCES = ["fa_api.cu", "fa_bwd_main.cu", "fa_bwd_wide.cu", "fa_fwd_tc.cu", "fa_fwd_split.cu",
           "fa_fwd_duo.cu",
           "fa_kernels.cu", "fa_ranges.cu", "fa_kvcache.cu",
           "fa_selftest.cu", "fa_noalloc.cu"]
HEADERS = ["fa_device.cuh", "fa_params.h", "fa_fwd_common.h", "fa_bwd_units.cuh", "fa_ranges.h",
           "fa_fwd_ranges.cuh", "fa_kvcache.h"]
PUBLIC_HEADERS = [os.path.join(ROOT, "include", h) for h in ("fa.h", "fa_selftest.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = [os.path.join(CSRC, h) for h in HEADERS] + PUBLIC_HEADERS
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + common):
            jobs.append((s, o))

    def compile_one(job):
        s, o = job
        cmd = [cc] + ARCH + FLAGS + ["-c", s, "-o", o]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s" % (s, r.stderr))
        return r.stderr

    with ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        logs = list(ex.map(compile_one, jobs))
    if verbose:
        for log in logs:
            sys.stderr.write(log)
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        # static CUDA runtime, no link against the driver library: the .so
        # loads on a machine without a GPU (the tensor-map encoder is fetched
        # through the runtime's driver entry-point query at run time)
        cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s" % r.stderr)
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
