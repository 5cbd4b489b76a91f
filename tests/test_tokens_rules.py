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


def test_clusters_follow_what_the_gpu_places(tmp_path):
    out = _run(tmp_path, r"""
    // the largest power of two that fits, down to one CTA
    for (int limit : {16, 15, 8, 5, 2, 1, 0})
        printf("%d ", placeable_cluster(16, [&](int c) { return c <= limit ? 3 : 0; }));
    // the sort: what each CTA holds, and the sort in global memory beyond that
    bool ok = true;
    for (int most = 1; most <= 16; most *= 2)
        for (int64_t n = 1; n < 400000; n += n < 3000 ? 1 : 97) {
            const int c = sort_cluster(n, most);
            if (c == 0) {
                ok = ok && n > (int64_t)most * kSortMaxShare && sort_may_use_memory(n);
                continue;
            }
            const int64_t per = (n + c - 1) / c;
            ok = ok && c <= most && (c & (c - 1)) == 0 &&
                 (per + kSortThreads - 1) / kSortThreads * kSortThreads <= kSortMaxShare;
        }
    printf("%d ", ok);
    printf("%d %d %d %d ", sort_cluster(163840, 16), sort_cluster(163841, 16),
           sort_cluster(81920, 8), sort_cluster(81921, 8));
    // a row's CTAs
    printf("%d %d %d %d", logprob_split(1, 128000, 4, 152, 16), logprob_split(1, 128000, 4, 152, 8),
           logprob_split(1, 128000, 4, 152, 1), logprob_split(700, 128000, 8, 152, 16));
    """)
    assert out.split() == ["16", "8", "8", "4", "2", "1", "1", "1", "16", "0", "8", "0",
                           "16", "8", "1", "1"]


@pytest.mark.parametrize("n", [10241, 16383, 163840, 163841])
def test_workspace_holds_the_sort_in_memory(n):
    """Whatever cluster a GPU places, the workspace of a call is one size."""
    from row_wise_normalization_gb300 import capi

    small = capi.embed_bwd_workspace_size(10240, 1000, 8)
    assert small < 10240 * 8 + (10240 // 8) * (2 * 8 * 4 + 2) + 4096
    # keys and positions twice, counts of 512 digits for each 4096 ids, sums of the chunks
    chunks = -(-n // 32)
    assert capi.embed_bwd_workspace_size(n, 1000, 8) >= 16 * n + -(-n // 4096) * 2048 + 64 * chunks


def test_realigned_rows_read_nothing_beside_the_row(tmp_path):
    """Every phase of both rows: the aligned vectors that are read lie within the source row,
    every element is written once, and what is left over is at most a warp's."""
    out = _run(tmp_path, r"""
    long bad = 0, rows = 0, vectors = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int64_t d = 1; d <= 100; ++d)
            for (uintptr_t o = 4096; o < 4112; o += es)
                for (uintptr_t s = 8192; s < 8208; s += es) {
                    const ShiftSpan p = shift_span(o, s, d, es);
                    const int64_t vec = 16 / es, tail = p.head + p.nv * vec;
                    const uintptr_t first = s + p.head * es - p.phase;
                    const uintptr_t last = first + p.nv * 16 + (p.phase ? 16 : 0);
                    ++rows;
                    vectors += p.nv;
                    bad += p.head < 0 || p.nv < 0 || tail > d || p.head + (d - tail) > 32;
                    if (p.nv > 0) {
                        bad += (o + p.head * es) % 16 != 0 || first % 16 != 0;
                        bad += first < s || last > s + d * es;
                    }
                    // an end leaves at most one vector, and fewer elements than one, behind
                    bad += p.head >= 2 * vec || d - tail >= 2 * vec;
                }
    printf("%ld %d", bad, rows > 0 && vectors > 0);
    """)
    assert out.split() == ["0", "1"]
