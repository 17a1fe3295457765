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
BINDING = os.path.join(PKG, "_fa_torch.so")   # the short way in for torch tensors (fa_torch.cpp)
SOURCES = ["fa_api.cu", "fa_bwd_main.cu", "fa_bwd_wide.cu", "fa_fwd_tc.cu", "fa_fwd_split.cu",
           "fa_fwd_duo.cu",
           "fa_kernels.cu", "fa_ranges.cu", "fa_kvcache.cu", "fa_kvcache4.cu", "fa_rope.cu",
           "fa_selftest.cu", "fa_noalloc.cu"]
HEADERS = ["fa_device.cuh", "fa_params.h", "fa_fwd_common.h", "fa_bwd_units.cuh", "fa_ranges.h",
           "fa_fwd_ranges.cuh", "fa_kvcache.h", "fa_kvwork.cuh", "fa_epilogue.h", "fa_rope.h"]
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

    def compile_binding():
        """fa_torch.cpp against the installed torch's and Python's headers."""
        import sysconfig

        import torch
        t = os.path.dirname(torch.__file__)
        s, o = os.path.join(CSRC, "fa_torch.cpp"), os.path.join(BUILD, "fa_torch.o")
        if not (force or _stale(o, [s] + PUBLIC_HEADERS + [os.path.join(t, "version.py")])):
            return
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
        for d in (sysconfig.get_paths()["include"], os.path.join(t, "include"),
                  os.path.join(t, "include", "torch", "csrc", "api", "include"),
                  os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")):
            cmd += ["-isystem", d]
        r = subprocess.run(cmd + ["-I" + os.path.join(ROOT, "include"), "-c", s, "-o", o], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed on %s:\n%s" % (s, r.stderr))

    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        binding = ex.submit(compile_binding)
        logs = list(ex.map(compile_one, jobs))
        binding.result()
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
    o = os.path.join(BUILD, "fa_torch.o")
    if force or _stale(BINDING, [o]):
        import torch
        t = os.path.join(os.path.dirname(torch.__file__), "lib")
        tmp = BINDING + ".tmp.%d" % os.getpid()
        cmd = ["g++", "-shared", "-o", tmp, o, "-L" + PKG, "-l:libfa_gb300.so", "-Wl,-rpath,$ORIGIN", "-L" + t,
               "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s" % r.stderr)
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
