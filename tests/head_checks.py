"""Tolerances of the head operators' tests, derived from the arithmetic.

u = 2^-24 is FP32's half step, uT the storage type's (2^-8 BF16, 2^-11 FP16, 2^-4 e4m3).

* r = (sum / d + eps)^-1/2: a lane adds at most 16 squares of its row in a chain (fused, one
  rounding each), 5 shuffles join lanes, one division or product and eps follow, whose
  constant 1 / d may be rounded too: 24 u relative of a sum of positive terms, half of that in r,
  and 2 units in the last place (4 u) of the reciprocal root: 16 u.
* y: n = x r w adds two roundings (18 u); y_a = n_a c - n_b s two more at most for each term
  and the difference: 21 u of the terms' absolute sum. Without a norm n = x: 3 u.
* dx: g = dy_a c + dy_b s is off by 3 u of its terms. r w g: 3 + 1 + 1 (the difference) + 16 + 1
  = 22 u of its magnitude. The second term x r^3 mean(w g x): its terms 3 + 2, their sum 24, the
  products with 1 / d and r twice 3 + 32, with x and r 2 + 16 and the difference 1: 83 u.
* dw: terms g x r 3 + 2 + 16 = 21 u, their sum one u for each addition of the longest chain:
  a lane's rows, 5 shuffles, 8 warps, then the CTAs' rows.
* storage adds uT of the result, half the smallest subnormal step at least.
* e4m3: 2 u more (the quotient by the scale takes one of them), then uT = 2^-4, half of 2^-9 at least.
"""
from __future__ import annotations

import numpy as np

from token_checks import TINY, U, UT, _near

E4M3_U, E4M3_TINY = 2.0 ** -4, 2.0 ** -10


def _stored(tol, want, dtype):
    return tol + UT[dtype] * (np.abs(want) + tol) + TINY[dtype]


def check_rope(got, want, mag, norm, dtype, what="y"):
    with np.errstate(invalid="ignore"):
        tol = _stored((21 if norm else 3) * U * mag, want, dtype)
    _near(got, want, tol, what)


def check_rope_e4m3(got, want, mag, norm, scale, what="cache"):
    """got: the stored values; want: divided by the scale and held within +-448."""
    tol = (23 if norm else 5) * U * mag / scale
    _near(got, want, tol + E4M3_U * (np.abs(want) + tol) + E4M3_TINY, what)


def check_rope_bwd(got, want, norm, dtype, what="dx"):
    tol = ((22 if norm else 3) * want["mag1"] + 83 * want["mag2"]) * U
    _near(got, want["dx"], _stored(tol, want["dx"], dtype), what)


def check_dw(got, want, tokens, heads, dtype, what="dw"):
    """heads: of queries and keys together. CTAs of 6 or 8 warps, at least 304 of them where there is
    work for as many, share the rows of both about evenly: queries' and keys' CTAs are rounded from
    their shares, at worst one where one and a half were due, and 1.5 rows / (304 * 6) is
    2 rows / (304 * 8). A lane adds at most one of a warp's rows at once, and a warp's unit is 16 of
    them at most. At most 2432 CTAs are joined: 19 a thread, 2 shuffles, 32 warps."""
    chain = 2 * -(-tokens * heads // (304 * 8)) + 16 + 5 + 8 + 19 + 2 + 32
    tol = (21 + chain) * U * want["dw_abs"]
    _near(got, want["dw"], _stored(tol, want["dw"], dtype), what)
