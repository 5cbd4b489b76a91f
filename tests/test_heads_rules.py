"""The head operators' rules that need no GPU; those of the host code are compiled as plain C++."""
import os
import re
import shutil
import subprocess
from fractions import Fraction

import numpy as np
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


# ---- 8 bits ----------------------------------------------------------------
def e4m3_values():
    """The non-negative e4m3 values in the order of their codes."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e4m3_codes(q):
    """The e4m3 codes of FP32 numbers: nearest, ties to the even code, at most 448 in size; NaN 127."""
    q = np.asarray(q, np.float32)
    a, held = np.minimum(np.abs(q.astype(np.float64)), 448.0), e4m3_values()
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.searchsorted(held, a).clip(1, 126)
    lo = hi - 1
    down, up = a - held[lo], held[hi] - a           # (exact: few bits of 64)
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return np.where(nan, 127, c + np.where(np.signbit(q), 128, 0)).astype(np.uint8)


def test_codes_of_exact_values_and_ties():
    held = e4m3_values().astype(np.float32)
    assert np.array_equal(e4m3_codes(held), np.arange(127)) and held[-1] == 448
    assert np.array_equal(e4m3_codes(-held), np.arange(127) + 128)
    ties = (held[1:] + held[:-1]) / 2
    assert np.array_equal(e4m3_codes(ties) % 2, np.zeros(126))
    assert e4m3_codes([np.inf, -np.inf, np.nan, 464, 1e-4]).tolist() == [126, 254, 127, 126, 0]


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
    middle between a number t of five bits, as every tie of e4m3 is, and an FP32 number beside it.

    The middle is n = 2^20 t +- 1 of 25 bits, and a 2^l = n b + d with |d| <= 9, as n b < 2^49. As
    a < 2^24 and n b >= 2^47, l > 23, so that 2^20 divides +-b + d: b is within 9 of a multiple of
    2^20."""
    for b in sorted({c * 2 ** 20 + e for c in range(8, 17) for e in range(-9, 10)}):
        if not 2 ** 23 <= b < 2 ** 24:
            continue
        for t in range(16, 33):
            for n in (2 ** 20 * t - 1, 2 ** 20 * t + 1):
                if not 2 ** 24 <= n < 2 ** 25:
                    continue
                for d in range(-9, 10):
                    a = n * b + d
                    a //= a & -a
                    if a < 2 ** 24:
                        yield a, b


def _reciprocals(tmp_path, scales):
    """(hi, lo, power) of each scale, as the host code gives them."""
    out = run_rules(tmp_path, "for (float s : {" + ", ".join(float(s).hex() + "f" for s in scales) +
                    '}) {\n    const E4m3Scale e = e4m3_scale(s);\n'
                    '    printf("%a %a %a\\n", e.hi, e.lo, e.power);\n}')
    return [tuple(Fraction(float.fromhex(x)) for x in line.split()) for line in out.split("\n") if line]


def test_reciprocals_of_scales(tmp_path):
    """Both parts are positive, hi at most the reciprocal, and their sum is off by lo's rounding alone:
    2^-47 of it. With as much for the product's that leaves h below 9 2^-49."""
    rng = np.random.default_rng(5)
    scales = rng.integers(0x00200008, 0x7f800000, 400).astype(np.uint32).view(np.float32)
    scales = [*scales, 1.0, 3.0, 7.0, 2.0 ** -126, 2.0 ** 64, 2.0 ** 96, 2.0 ** 96 * 1.25, 2.0 ** 127,
              float(np.float32(3.4028235e38)), *(
                  b * 2.0 ** e for _, b in set(close_quotients()) for e in (0, 72, 104))]
    for s, (hi, lo, power) in zip(scales, _reciprocals(tmp_path, scales)):
        exact = 1 / (Fraction(float(s)) * power)
        assert lo > 0 and hi <= exact and power in (1, Fraction(1, 2 ** 64)), float(s)
        assert exact - hi < exact / 2 ** 22
        assert abs(hi + lo - exact) <= (exact - hi) / 2 ** 24 + exact * Fraction(1, 2 ** 52), float(s)


def test_the_product_by_a_reciprocal_of_two_parts_rounds_as_the_quotient(tmp_path):
    """RN(a hi + RN(a lo)) is RN(x (1 + h)) of the quotient x = a / b, |h| < 9 2^-49. It can lie on another
    side of a tie than the FP32 quotient only where x is that close to a middle beside the tie."""
    pairs = sorted(set(close_quotients()))
    assert len(pairs) > 100
    bs = sorted({b for _, b in pairs})
    parts = dict(zip(bs, _reciprocals(tmp_path, bs)))
    differ = 0
    for a, b in pairs:
        hi, lo, _ = parts[b]
        got, want = _rounded(a * hi + _rounded(a * lo)), _rounded(Fraction(a, b))
        differ += got != want
        e = np.arange(-12, 36.0)                        # (quotients from 2^-36 on)
        assert np.array_equal(e4m3_codes(float(got) * 2 ** e), e4m3_codes(float(want) * 2 ** e)), (a, b)
    assert differ < 3                                   # (the search is for real)


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
