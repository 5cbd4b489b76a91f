"""The head operators' rules that need no GPU."""
from fractions import Fraction

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
