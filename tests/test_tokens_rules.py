"""The token operators' host rules, compiled as plain C++ (no GPU, no CUDA call): what is
prepared once in a context."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "row_wise_normalization_gb300", "csrc")


def _cuda_include():
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")


def _run(tmp_path, body):
    """Compiles and runs a program of the rules' header; returns what it prints."""
    if shutil.which("g++") is None or not os.path.exists(
            os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("needs g++ and CUDA's headers")
    src, exe = tmp_path / "rules.cpp", tmp_path / "rules"
    src.write_text('#include <cstdio>\n#include <cstdint>\n#include "rn_tokens.h"\n'
                   "using namespace rn;\nint main() {\n" + body + "\nreturn 0; }\n")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-I",
                           _cuda_include(), str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout


def test_a_failed_preparation_is_tried_again(tmp_path):
    out = _run(tmp_path, r"""
    unsigned long long done = 0;
    int calls = 0;
    cudaError_t answer = cudaErrorMemoryAllocation;
    auto set = [&] { ++calls; return answer; };
    printf("%d ", once_in_context(7, done, set) == cudaErrorMemoryAllocation);
    printf("%d ", once_in_context(7, done, set) == cudaErrorMemoryAllocation);
    answer = cudaSuccess;
    for (int k = 0; k < 3; ++k) printf("%d ", once_in_context(7, done, set) == cudaSuccess);
    printf("%d ", calls);                       // two failures and one success
    once_in_context(8, done, set);              // another context
    once_in_context(8, done, set);
    printf("%d ", calls);
    once_in_context(0, done, set);              // none current: never taken as done
    once_in_context(0, done, set);
    printf("%d", calls);
    """)
    assert out.split() == ["1", "1", "1", "1", "1", "3", "4", "6"]
