"""Build libmoe.so (the C-ABI library) for sm_103a with nvcc, in-tree, and _paged.so, the Python
side of the paged serving path, with g++ against the installed torch.

Each .cu translation unit is compiled in parallel, then linked into a shared
library against the shared CUDA runtime. libmoe.so needs nothing of torch and comes first: where the
torch headers that _paged.so is built against are missing, build() raises after libmoe.so is in
place. Either library is built again when a source or header of its own is newer, _paged.so also when
the installed torch or the interpreter is another one than it was built for.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
PY_SOURCE = os.path.join(CSRC, "py_paged.cpp")
PY_LIB = os.path.join(PKG, "_paged.so")
PY_STAMP = os.path.join(BUILD, "py_paged.stamp")  # what _paged.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-v,-warn-spills"]
# Kernels whose warps share out their registers: source, kernel, and the constant in the source that counts what a thread
# has at launch. With another count their launch is refused.
REGISTERS = (("gqa_rows.cu", "gqa_rows_kernel", "kRegsLaunch"),
             ("kv4_decode.cu", "kv4_decode_kernelILi1E", "kRegsLaunch"), ("kv4_decode.cu", "kv4_decode_kernelILi2E", "kRegsLaunch"))


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(INCLUDE, "**", "*.h"), recursive=True) + [os.path.abspath(__file__)]


def _newer(lib: str, deps) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps)


def lib_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _py_target() -> str:
    import torch
    return f"{torch.__version__} in {os.path.dirname(torch.__file__)}, Python {sys.version}"


def py_up_to_date() -> bool:
    if not (_newer(PY_LIB, [PY_SOURCE] + _headers()) and os.path.exists(PY_STAMP)):
        return False
    with open(PY_STAMP, encoding="utf-8") as f:
        return f.read() == _py_target()


def up_to_date() -> bool:
    return lib_up_to_date() and py_up_to_date()


def check_registers(src: str, log: str) -> None:
    """Raises when ptxas (its -v output in `log`) gave a kernel of REGISTERS another number than its source counts on."""
    for name, kernel, constant in REGISTERS:
        if os.path.basename(src) != name:
            continue
        with open(src, encoding="utf-8") as f:
            want = re.search(rf"\bconstexpr int {constant} = (\d+);", f.read())
        used = re.search(rf"Compiling entry function '[^']*{kernel}[^']*'.*?Used (\d+) registers", log, flags=re.S)
        if not (want and used and want[1] == used[1]):
            raise RuntimeError(f"{name}: {kernel} counts on {want and want[1]} registers a thread at launch, "
                               f"the compiler gave it {used and used[1]}")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    lib_stale, py_stale = force or not lib_up_to_date(), force or not py_up_to_date()
    if not (lib_stale or py_stale):
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        check_registers(src, r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        py_obj = ex.submit(_compile_py) if py_stale else None
        if lib_stale:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            _run("linking libmoe.so", [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
            os.replace(tmp, LIB)
        if py_obj is not None:
            _link_py(py_obj.result())
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
    with open(PY_STAMP, "w", encoding="utf-8") as f:
        f.write(_py_target())


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
