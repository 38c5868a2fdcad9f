"""Builds the CUDA library in-tree: io_aware_exact_12_gb300/libattn.so.

Each translation unit under csrc/ is compiled for sm_103a only
(-gencode arch=compute_103a,code=sm_103a) in parallel, then linked as a
shared library against the shared CUDA runtime.  Beside it, compiled at the
same time by the C++ compiler, _paged.so: the Python binding of the paged and windowed calls
(CPython and torch's C++ headers).  No cmake; a few seconds per file.  Run ``python -m io_aware_exact_12_gb300.build`` (or call ``build()``).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libattn.so")
SOURCES = ["attn_api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_noalloc.cu", "attn_diag.cu", "attn_decode.cu", "attn_fwd_fp8.cu",
           "attn_paged_append.cu", "attn_paged_decode.cu", "attn_paged_select.cu", "attn_paged_assign.cu",
           "attn_window_fwd.cu", "attn_window_bwd.cu"]
HEADERS = ["attn_internal.h", "block_order.h", "tc_sm103.cuh", "dropout.cuh", "attn_paged.h", "attn_window.h", "attn_window_tiles.cuh"]
BINDING = "paged_binding.cpp"
BINDING_PATH = os.path.join(PKG, "_paged.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _cuda_dir() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))


def _binding_compile(src: str, obj: str):
    import torch
    t = _torch_dir()
    return [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
            "-isystem", os.path.join(t, "include"), "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(_cuda_dir(), "include"), "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj]


def _binding_link(obj: str, out: str):
    lib = os.path.join(_torch_dir(), "lib")
    return [os.environ.get("CXX", "g++"), "-shared", "-o", out, obj, "-L", PKG, "-l:libattn.so", "-L", lib, "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, h) for h in ("attn.h", "attn_diag.h")] + [__file__]
    objs = []
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or verbose_ptxas or _stale(o, [s] + headers):
            jobs.append([nvcc()] + _flags(verbose_ptxas) + ["-c", s, "-o", o])

    bind_src, bind_obj = os.path.join(CSRC, BINDING), os.path.join(BUILD_DIR, "paged_binding.o")
    if force or _stale(bind_obj, [bind_src, os.path.join(INCLUDE, "attn.h"), __file__]):
        jobs.append(_binding_compile(bind_src, bind_obj))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for cmd, r in ex.map(run, jobs):
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError("compilation failed: " + " ".join(cmd))
            if not quiet or verbose_ptxas:
                sys.stderr.write(r.stdout + r.stderr)
    if force or jobs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + ".tmp.%d" % os.getpid()
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed: " + " ".join(cmd))
        os.replace(tmp, LIB_PATH)
    if force or _stale(BINDING_PATH, [bind_obj, LIB_PATH]):
        tmp = BINDING_PATH + ".tmp.%d" % os.getpid()
        cmd, r = run(_binding_link(bind_obj, tmp))
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed: " + " ".join(cmd))
        os.replace(tmp, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, quiet=False))
