"""Build the CUDA library in-tree with nvcc for sm_103a.

Produces ``bit_rotated_kv_decode_gb300/_lib/liboscar_gb300.so`` (CUDA runtime
linked statically).  Translation units are compiled in parallel; a unit is
rebuilt when its source or a header is newer than its object.  Beside it goes
``_oscar_calls.so``, the Python extension that marshals the arguments of the paged calls.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "liboscar_gb300.so")
CALLS = os.path.join(LIBDIR, "_oscar_calls.so")   # argument marshalling for Python (csrc/calls.cpp)
SOURCES = ["host.cpp", "write_kernels.cu", "decode_kernels.cu", "decode_scratch.cu", "bf16_decode.cu",
           "paged_host.cpp", "paged_append.cu", "paged_decode.cu", "paged_prefill.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src + ".o")
        objs.append(obj)
        if force or _stale(obj, [path] + headers):
            extra = ["-Xptxas", "-v"] if verbose and src.endswith(".cu") else []
            jobs.append([nvcc, *ARCH, *FLAGS, *extra, "-c", path, "-o", obj])

    calls_src = os.path.join(CSRC, "calls.cpp")
    if force or _stale(CALLS, [calls_src] + headers):
        torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)   # (importing it takes longer than the build)
        torch_lib = os.path.join(torch_dir, "lib")
        dirs = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
                sysconfig.get_paths()["include"]]
        jobs.append([shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + d for d in dirs),
                     calls_src, "-o", CALLS, "-L" + torch_lib, "-Wl,-rpath," + torch_lib, "-ltorch_python", "-ltorch_cpu",
                     "-lc10", "-lc10_cuda"])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(jobs) or 1) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                print(out)
    if force or jobs or _stale(LIB, objs):
        run([nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"])
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
