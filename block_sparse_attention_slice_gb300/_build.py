"""Builds ``libattn_slice.so`` in-tree with nvcc for sm_103a, and the
marshalling module ``_paging.so`` with g++ against PyTorch's headers.

Each ``csrc/*.cu`` translation unit is compiled in parallel, then linked
into one shared library next to this file; ``csrc/paging_module.cpp`` compiles
beside them.  Rebuilds only when a source or header is newer than what is
built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn_slice.so")
MODULE = os.path.join(HERE, "_paging.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _module_flags(nvcc):
    """Compile and link flags of the marshalling module: PyTorch's own, for its version here."""
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
           "/usr/local/cuda/include"]
    cc = ["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    ld = ["-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
          "-L" + HERE, "-l:libattn_slice.so", "-Wl,-rpath,$ORIGIN"]
    return cc + ["-I" + i for i in inc], ld


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr[-4000:]}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library if needed and returns its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-Xptxas", "-v", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(obj + ".log", "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
        return obj

    cc, ld = _module_flags(nvcc)
    cxx = os.environ.get("CXX") or "g++"
    module_obj = os.path.join(BUILD, "paging_module.o")
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        module = ex.submit(_run, [cxx, *cc, "-c", os.path.join(CSRC, "paging_module.cpp"), "-o", module_obj],
                           "compiling paging_module.cpp failed")
        objs = list(ex.map(compile_one, srcs))
        module.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)
    _run([cxx, "-shared", "-o", MODULE + ".tmp", module_obj, *ld], "linking _paging.so failed")
    os.replace(MODULE + ".tmp", MODULE)
    if verbose:
        for o in objs:
            sys.stdout.write(open(o + ".log").read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
