"""The in-tree build: the C library does not depend on torch's headers, the Python side is built again for another torch,
and a kernel that did not get the registers it counts on stops it (no GPU needed)."""
import ctypes
import os

import pytest
import torch

from routed_expert_ffn_softmax_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build with one small C function in place of the library's sources, in a folder of its own."""
    src = tmp_path / "small.cu"
    src.write_text('extern "C" int three() { return 3; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    for name, file in (("BUILD", "_build"), ("LIB", "libmoe.so"), ("PY_LIB", "_paged.so"), ("PY_STAMP", "_build/stamp")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return tmp_path


def test_the_c_library_is_built_without_torch_headers(small, monkeypatch):
    def no_headers():
        raise RuntimeError("g++ on py_paged.cpp failed: ATen/core/TensorBody.h: No such file")
    monkeypatch.setattr(build, "_compile_py", no_headers)
    with pytest.raises(RuntimeError, match="TensorBody"):
        build.build()
    assert ctypes.CDLL(build.LIB).three() == 3
    assert build.lib_up_to_date() and not build.py_up_to_date() and not build.up_to_date()
    at = os.path.getmtime(build.LIB)
    with pytest.raises(RuntimeError):  # the next call tries the Python side alone
        build.build()
    assert os.path.getmtime(build.LIB) == at


def test_a_missing_or_older_library_is_not_current(small, monkeypatch):
    monkeypatch.setattr(build, "_compile_py", lambda: "")
    monkeypatch.setattr(build, "_link_py", lambda obj: None)
    assert not build.lib_up_to_date()
    build.build()
    assert build.lib_up_to_date()
    os.utime(build.LIB, (1, 1))
    assert not build.lib_up_to_date()


@pytest.mark.parametrize("what", ["torch", "python"])
def test_the_python_side_is_built_again_for_another_torch_or_interpreter(what, monkeypatch):
    build.build()
    assert build.up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.1")
    else:
        monkeypatch.setattr(build.sys, "version", "2.7")
    assert build.lib_up_to_date() and not build.py_up_to_date() and not build.up_to_date()


def ptxas(kernel, registers):
    return f"""ptxas info    : Compiling entry function '_ZN3moe4rows18rows_tables_kernelENS0_6ParamsE' for 'sm_103a'
ptxas info    : Used 32 registers, used 1 barriers, 9216 bytes smem
ptxas info    : Compiling entry function '_ZN3moe4rows15{kernel}E14CUtensorMap_stS1_S1_NS0_6ParamsE' for 'sm_103a'
ptxas info    : Function properties for _ZN3moe4rows15{kernel}E14CUtensorMap_stS1_S1_NS0_6ParamsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {registers} registers, used 16 barriers
"""


def test_a_kernel_without_its_registers_stops_the_build():
    src = os.path.join(build.CSRC, "gqa_rows.cu")
    build.check_registers(src, ptxas("gqa_rows_kernel", 168))
    for log in (ptxas("gqa_rows_kernel", 166), ptxas("another_kernel", 168), ""):
        with pytest.raises(RuntimeError, match="gqa_rows_kernel counts on 168 registers"):
            build.check_registers(src, log)
    build.check_registers(os.path.join(build.CSRC, "paged_plan.cu"), "")


def test_the_build_looks_at_the_registers(small, monkeypatch):
    src = small / "gqa_rows.cu"
    src.write_text("constexpr int kRegsLaunch = 255;\n__global__ void gqa_rows_kernel(int* p) { *p = 1; }\n")
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "_compile_py", lambda: "")
    with pytest.raises(RuntimeError, match="counts on 255 registers"):
        build.build()
    assert not os.path.exists(build.LIB)
