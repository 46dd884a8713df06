"""Build the CUDA library in-tree with nvcc for sm_103a.

Produces ``bit_rotated_kv_decode_gb300/_lib/liboscar_gb300.so`` (CUDA runtime
linked statically).  Translation units are compiled in parallel; a unit is
rebuilt when its source or a header is newer than its object.  Beside it goes
``_oscar_calls.*.so``, the Python extension that marshals the arguments of the paged
calls (csrc/calls.cpp); without torch it is left out, and they are marshalled in Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "liboscar_gb300.so")
SOURCES = ["host.cpp", "write_kernels.cu", "decode_kernels.cu", "decode_scratch.cu", "bf16_decode.cu",
           "paged_host.cpp", "paged_append.cu", "paged_decode.cu", "paged_prefill.cu", "prompt_attention.cu",
           "extend.cu", "chunk_read.cu", "chunk_attention.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def calls_path() -> str:
    """The extension for this interpreter and this torch: it reads tensors by torch's own layout, so that one built for
    another version must not be found."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "unknown"
    return os.path.join(LIBDIR, f"_oscar_calls.{sysconfig.get_config_var('SOABI')}.torch-{torch}.so")


CALLS = calls_path()


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


def _extension(nvcc: str):
    """The command that compiles the extension, or None and why there is none."""
    spec = importlib.util.find_spec("torch")   # (importing it takes longer than the build)
    if spec is None or not spec.origin:
        return None, "torch is not installed"
    torch_dir = os.path.dirname(spec.origin)
    torch_lib, python = os.path.join(torch_dir, "lib"), sysconfig.get_paths()["include"]
    for need in (os.path.join(torch_lib, "libc10_cuda.so"), os.path.join(python, "Python.h")):
        if not os.path.exists(need):
            return None, f"{need} is missing"
    dirs = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
            os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"), python]
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + d for d in dirs),
            os.path.join(CSRC, "calls.cpp"), "-o", calls_path(), "-L" + torch_lib, "-Wl,-rpath," + torch_lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], None


# Kernels that split their registers at run time (setmaxnreg) count on what they are launched
# with: a file, a pattern of the kernels' names, how many of them, and the registers.
REGISTERS = {"paged_prefill.cu": (r"paged_prefill_kernelI", 4, 168),
             "prompt_attention.cu": (r"paged_prefill_kernelI", 6, 168),
             "chunk_attention.cu": (r"chunk_scan_kernelI", 6, 128)}


def check_registers(src: str, log: str) -> None:
    """Checks a file's kernels in what ptxas -v says."""
    if src not in REGISTERS:
        return
    pattern, count, want = REGISTERS[src]
    used = [int(n) for name, n in re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, re.S)
            if re.search(pattern, name)]
    if used != [want] * count:
        raise RuntimeError(f"build failed: {src}: {count} kernels of {want} registers are wanted, the compiler has {used}")


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
            extra = ["-Xptxas", "-v"] if src.endswith(".cu") else []
            jobs.append((src, obj, [nvcc, *ARCH, *FLAGS, *extra, "-c", path, "-o", obj]))

    extension, why = _extension(nvcc)
    if why:
        print(f"{why}: the paged calls are marshalled in Python", file=sys.stderr)
    elif not force and not _stale(calls_path(), [os.path.join(CSRC, "calls.cpp")] + headers):
        extension = None

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    def compiled(job):
        src, obj, cmd = job
        out = run(cmd)
        try:
            check_registers(src, out)
        except RuntimeError:
            os.remove(obj)
            raise
        return out

    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        late = ex.submit(run, extension) if extension else None
        for out in ex.map(compiled, jobs):
            if verbose and out:
                print(out)
    if force or jobs or _stale(LIB, objs):
        run([nvcc, *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"])
    if late:
        late.result()   # (an error in it leaves the library built)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
