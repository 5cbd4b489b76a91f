"""The head operators' rules that need no GPU; those of the host code are compiled as plain C++."""
import os
import re
import shutil
import subprocess
from fractions import Fraction

import pytest

from test_tokens_rules import CSRC, _cuda_include


def run_rules(tmp_path, body):
    """Compiles and runs a program of the rules' header, with overflows of signed numbers that end
    it; returns what it prints."""
    if shutil.which("g++") is None or not os.path.exists(
            os.path.join(_cuda_include(), "cuda_runtime.h")):
        pytest.skip("needs g++ and CUDA's headers")
    src, exe = tmp_path / "rules.cpp", tmp_path / "rules"
    src.write_text('#include <cstdio>\n#include <cstdint>\n#include "rn_heads.h"\n'
                   "using namespace rn;\nint main() {\n" + body + "\nreturn 0; }\n")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", "-I", CSRC, "-I",
                           _cuda_include(), str(src), "-o", str(exe)])
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout


E4M3_TIES = range(16, 33)        # five significant bits: every tie of e4m3, subnormal ones too


def _rounded(x):
    """A positive fraction to 24 significant bits, ties to even."""
    e = x.numerator.bit_length() - x.denominator.bit_length() - 24
    step = Fraction(2) ** e
    while x / step >= 2 ** 24:
        step *= 2
    while x / step < 2 ** 23:
        step /= 2
    return round(x / step) * step          # (round() of a fraction: ties to even)


def close_quotients():
    """All pairs of 24-bit numbers (a, b), b with all of them, whose quotient is within 9 2^-49 of the
    middle between a tie of e4m3 and an FP32 number beside it.

    The middle is n = 2^20 t +- 1 of 25 bits, t of five, and a 2^l = n b + d with |d| <= 9, as n b <
    2^49. As a < 2^24 and n b >= 2^47, l > 23, so that 2^20 divides +-b + d: b is within 9 of a
    multiple of 2^20."""
    for b in sorted({c * 2 ** 20 + e for c in range(8, 17) for e in range(-9, 10)}):
        if not 2 ** 23 <= b < 2 ** 24:
            continue
        for t in E4M3_TIES:
            for n in (2 ** 20 * t - 1, 2 ** 20 * t + 1):
                if not 2 ** 24 <= n < 2 ** 25:
                    continue
                for d in range(-9, 10):
                    a = n * b + d
                    a //= a & -a
                    if a < 2 ** 24:
                        yield a, b


def test_a_corrected_product_is_the_quotient_beside_ties():
    """t - (t b - a) / b with t = a / b by the reciprocal, each operation rounded once: its relative
    error before the last rounding is at most 2^-46 = 8 2^-49, so that only these pairs, where that
    could pass the middle of two FP32 numbers, need to be tried."""
    pairs = set(close_quotients())
    assert len(pairs) > 100
    for a, b in pairs:
        inverse = _rounded(Fraction(1, b))
        t = _rounded(a * inverse)
        rest = t * b - a                                   # (fused: one rounding)
        rest = _rounded(rest) if rest > 0 else -_rounded(-rest) if rest else rest
        assert _rounded(t - rest * inverse) == _rounded(Fraction(a, b)), (a, b)


# ---- host code -------------------------------------------------------------
def test_bisection_stays_within_the_offsets(tmp_path):
    """Every entry that is looked at is one of 1 .. seqs, for as many sequences as are taken, and
    the answer is the first end beyond the token."""
    out = run_rules(tmp_path, r"""
    long wrong = 0, looked = 0;
    for (int seqs : {0, 1, 2, 3, 61, 4096, (1 << 29) + 1, (1 << 30) - 1, 1 << 30})
        for (int64_t t : {(int64_t)-1, (int64_t)0, (int64_t)seqs / 2, (int64_t)seqs - 1, (int64_t)seqs,
                          (int64_t)1 << 31}) {
            // sequences of one token each: entry i is i
            const int got = first_beyond(
                [&](int i) {
                    ++looked;
                    if (i < 1 || i > seqs) ++wrong;
                    return (int64_t)i;
                },
                seqs, t);
            const int64_t want = t < 1 ? 1 : t >= seqs ? (int64_t)seqs + 1 : t + 1;
            wrong += got != want;
        }
    printf("%ld %d", wrong, looked > 100);
    """)
    assert out.split() == ["0", "1"]


# ---- what is compiled ------------------------------------------------------
def test_kernels_that_are_compiled_are_those_that_calls_reach(tmp_path):
    """Every shape that some width and access gives has its kernels in the library, and no other."""
    lib = os.path.join(os.path.dirname(CSRC), "librownorm.so")
    if shutil.which("nm") is None or not os.path.exists(lib):
        pytest.skip("needs nm and the library")
    out = run_rules(tmp_path, r"""
    for (int vec : {4, 8})
        for (int v : {vec, 4, 2, 1})
            for (int64_t d = 2; d <= kMaxHeadDim; d += 2)
                for (int bwd = 0; bwd < 2 && d % (2 * v) == 0; ++bwd) {
                    const HeadShape s = head_shape(v, vec, d, bwd);
                    printf("%d %d %d %d %d\n", vec, bwd, s.v, s.lpr, s.ch);
                }
    """)
    want = set()
    for line in set(out.split("\n")) - {""}:
        vec, bwd, v, lpr, ch = map(int, line.split())
        for t in ["f"] if vec == 4 else ["13__nv_bfloat16", "6__half"]:
            if not bwd:          # (into a cache or not, of 8 bits or not)
                want |= {("fwd", t, v, lpr, ch, *kind) for kind in ((0, 0), (1, 0), (1, 1))}
            else:                # (neighbours or not, several tokens to a warp where it holds several rows)
                want |= {("bwd", t, v, lpr, ch, inter, pack) for inter in (0, 1)
                         for pack in ((0, 1) if lpr <= 16 else (0,))}
    names = subprocess.run(["nm", lib], capture_output=True, text=True, check=True).stdout
    got = {(m[0], m[1], *map(int, m[2:])) for m in re.findall(
        r"heads_(fwd|bwd)_kernelI(f|13__nv_bfloat16|6__half)Li(\d+)ELi(\d+)ELi(\d+)ELb([01])ELb([01])E",
        names)}
    assert want - got == set() and got - want == set()
