"""Build libmoe.so (the C-ABI library) for sm_103a with nvcc, in-tree, and _paged.so, the Python
side of the paged serving path, with g++ against the installed torch.

Each .cu translation unit is compiled in parallel, then linked into a shared
library against the shared CUDA runtime. The build is skipped when the libraries
are newer than every source and header.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
PY_SOURCE = os.path.join(CSRC, "py_paged.cpp")
PY_LIB = os.path.join(PKG, "_paged.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [PY_SOURCE] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "**", "*.h"), recursive=True) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(PY_LIB)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(PY_LIB))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        py_obj = ex.submit(_compile_py)
        objs = list(ex.map(compile_one, sources()))
        py_obj = py_obj.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_py(py_obj)
    return LIB


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_py() -> str:
    import torch
    obj = os.path.join(BUILD, "py_paged.cpp.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    _run(f"g++ on {PY_SOURCE}", [
        "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-isystem", inc, "-isystem",
        os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-I", sysconfig.get_path("include"),
        "-I", INCLUDE, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", PY_SOURCE, "-o", obj])
    return obj


def _link_py(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = PY_LIB + f".tmp{os.getpid()}"
    _run("linking _paged.so", [
        "g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libmoe.so", "-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu",
        "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"])
    os.replace(tmp, PY_LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
