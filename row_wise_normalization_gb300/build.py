"""Build the CUDA library ``librownorm.so`` in-tree with nvcc for sm_103a, and beside it
``_binding.so``, which marshals the head operators' plain calls from Python (C++ against the
installed PyTorch; where that cannot be compiled, the package does the same in Python).

Each ``csrc/*.cu`` translation unit is compiled to an object in
``_build/`` (in parallel), then linked into ``librownorm.so`` next to this
file. Rebuilds only what is older than its sources. ``-Xptxas -v`` output
(registers, spills, shared memory per kernel) is kept in
``_build/ptxas.log``.

Usage: ``python -m row_wise_normalization_gb300.build [--force] [--verbose]``
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librownorm.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xptxas", "-v",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps)


def build_binding(force: bool = False) -> bool:
    """Compile ``_binding.so``; False (and no such file) where that does not succeed."""
    src = os.path.join(CSRC, "binding.cpp")
    stamp = os.path.join(BUILD, "binding.stamp")
    try:
        import torch

        made_for = f"{torch.__version__} {sys.version}"
        if (not force and not _stale(BINDING, [src] + _headers()) and os.path.exists(stamp)
                and open(stamp).read() == made_for):
            return True
        root = os.path.dirname(torch.__file__)
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
        inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
               "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src, "-o",
               tmp, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
               f"-Wl,-rpath,{lib}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stderr if r.returncode else ""
    except (ImportError, OSError) as e:
        why = str(e)
    if why:
        print(f"[build] _binding.so: not built, calls are marshalled in Python\n{why[-2000:]}",
              file=sys.stderr, flush=True)
        if os.path.exists(BINDING):
            os.remove(BINDING)
        return False
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(made_for)
    return True


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link the library; returns its path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    objs = []
    todo = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            todo.append((src, obj))

    def compile_one(item):
        src, obj = item
        cmd = [nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj + ".tmp"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        os.replace(obj + ".tmp", obj)
        with open(obj + ".ptxas.log", "w") as f:
            f.write(r.stderr)
        if verbose:
            print(f"[build] {os.path.basename(src)}", flush=True)

    n = jobs or min(len(todo) + 1, os.cpu_count() or 1)
    with ThreadPoolExecutor(n) as ex:
        binding = ex.submit(build_binding, force)
        list(ex.map(compile_one, todo))
        binding.result()
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            for obj in objs:
                p = obj + ".ptxas.log"
                if os.path.exists(p):
                    f.write(open(p).read())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
