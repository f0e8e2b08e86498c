"""Builds ``libattn_slice.so`` in-tree with nvcc for sm_103a, and the
marshalling module ``_paging.so`` with g++ against PyTorch's headers.

Each ``csrc/*.cu`` translation unit is compiled in parallel, then linked
into one shared library next to this file; ``csrc/paging_module.cpp`` compiles
beside them.  The library needs nvcc alone.  Rebuilds only when a source or
header is newer than what is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
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
MODULE_SRC = os.path.join(CSRC, "paging_module.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build the library")
    return cand


def _cxx():
    return os.environ.get("CXX") or "g++"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(built, deps) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(p) <= os.path.getmtime(built) for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def module_up_to_date() -> bool:
    return _newer(MODULE, [MODULE_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    return library_up_to_date() and module_up_to_date()


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
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{what}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr[-4000:]}")
    return r


def _has_torch() -> bool:
    try:
        return importlib.util.find_spec("torch") is not None
    except ValueError:          # sys.modules holds None for it
        return False


def build_library(force: bool = False) -> str:
    """Compiles the C library if needed, with nvcc alone, and returns its path."""
    if not force and library_up_to_date():
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

    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(compile_one, srcs))
    _run([nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs], "linking libattn_slice.so failed")
    os.replace(LIB + ".tmp", LIB)
    return LIB


def _compile_module() -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc, _ = _module_flags(_nvcc())
    obj = os.path.join(BUILD, "paging_module.o")
    _run([_cxx(), *cc, "-c", MODULE_SRC, "-o", obj], "compiling paging_module.cpp failed")
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles what is needed, the library first, and returns its path.

    The module needs a C++ compiler and the headers of PyTorch and Python: it is
    left out where there is no PyTorch, whose tensors alone it serves, and what
    goes wrong with it is raised once the library stands."""
    todo = _has_torch() and (force or not module_up_to_date())
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_compile_module) if todo else None
        build_library(force)
        if module:
            obj = module.result()
            _, ld = _module_flags(_nvcc())
            _run([_cxx(), "-shared", "-o", MODULE + ".tmp", obj, *ld], "linking _paging.so failed")
            os.replace(MODULE + ".tmp", MODULE)
    if verbose:
        for log in sorted(glob.glob(os.path.join(BUILD, "*.log"))):
            sys.stdout.write(open(log).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
