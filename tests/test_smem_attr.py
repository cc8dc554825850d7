"""The table of the kernels' shared memory limits (hs_smem_attr.h), on the CPU:
the header is compiled against a stand-in of the CUDA runtime that counts the
attribute calls.  A kernel launched with ever larger sizes once filled the
table with one entry a size, after which every other kernel's call paid for it."""
import os
import pathlib
import shutil
import subprocess

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]
CUDA = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


def test_a_kernel_takes_one_entry_whatever_its_sizes(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists(os.path.join(CUDA, "cuda_runtime.h")):
        pytest.skip("g++ or the CUDA headers are not available")
    exe = tmp_path / "smem_attr_check"
    subprocess.run([cxx, "-O1", "-std=c++17", "-I", str(ROOT / "activation_sparse_moe_gb300" / "csrc"), "-I", str(ROOT / "include"),
                    "-I", CUDA, str(ROOT / "tests" / "smem_attr_check.cpp"), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    # 101 sizes; 40 kernels once; nothing; the largest size; the other device once; 100 kernels, of which 64 - 42 find a
    # place and 78 are set again; their size
    assert got == [101, 40, 0, 50000 + 100 * 16, 1, 100 + 78, 70000]
