"""Tolerances of the token operators' tests, derived from the arithmetic.

u = 2^-24 is FP32's half step, uT the storage type's (2^-8 BF16, 2^-11 FP16).

* Embedding rows: one FP32 product, one rounding: compared bit for bit.
* Embedding gradient: m terms added in any order err by at most (m - 1) u times
  the sum of their absolute values; the scale's product (and the sum onto an
  existing value) add one rounding each, storage uT.
* lse = m + log S: z_j is rounded by its subtraction, its product and the
  product's constant (scale * log2 e, itself two roundings), so e_j is off by
  4 u |z_j| relative, and by 2 units in the last place (4 u) of the exponential;
  S adds at most DEPTH values in a row along its longest chain (a thread's
  batches of 32, its rescalings, the merge of threads), all of them positive:
      dS = u (DEPTH + 4 + 4 E|z|),  E the mean under p.
  lse adds the roundings of its logarithm and sum and of m's scaling.
* entropy = log S - W / S with W summed along the same chain:
      dS + u (|W/S| (2 DEPTH + 12) + 8 E z^2) + 4 u |log S|.
* gradient: p_j is off by u (4 |z_j| + 6) relative; the terms' magnitudes and
  (1 + |z|) come from the oracle, so 8 u covers them, with one rounding of the
  stored value; the exponential's results below 2^-126 are zero.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
UT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
# half of the smallest subnormal step of each type
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


def depth(vocab):
    """The longest chain of additions of a row's sum: 32 in a batch, then one
    for each batch of a thread (at least 4096 columns a round), then 5 in a
    warp and up to 32 warps and 16 CTAs."""
    return 32 + vocab // 4096 + 5 + 32 + 16 + 4


def _near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    # (outputs are FP32 or narrower: what FP32 cannot hold is infinite)
    with np.errstate(over="ignore"):
        narrow = want.astype(np.float32).astype(np.float64)
    special = ~np.isfinite(narrow)
    ok = np.where(special, (got == narrow) | (np.isnan(got) & np.isnan(narrow)), False)
    with np.errstate(invalid="ignore"):
        ok |= ~special & (np.abs(got - want) <= tol)
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} off; first {i}: got {got[i]!r}, want "
                             f"{want[i]!r}, tolerance {np.broadcast_to(tol, want.shape)[i]:.3e}")


def check_embed_bwd(got, want, absum, terms, dtype, old=None, what="dtable"):
    """old: the values accumulated onto."""
    m = np.asarray(terms)[:, None]
    tol = U * (np.maximum(m - 1, 0) + 2) * absum
    if old is not None:
        want = want + old
        tol = tol + U * np.abs(want)
    tol = tol * (1 + UT[dtype]) + UT[dtype] * np.abs(want) + TINY[dtype]
    _near(got, want, tol, what)


def check_logprob(out, want, logits, scale, what=""):
    """out, want: dicts as oracle.tokens.logprob gives (out's entries may be
    missing)."""
    x = scale * np.asarray(logits, np.float64)
    lse = want["lse"]
    fine = np.isfinite(lse)
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.where(fine, np.max(x, axis=1), 0.0)
        z = x - m[:, None]
        p = np.where(fine[:, None], np.exp(x - lse[:, None]), 0.0)
        az = np.where(p > 0, np.abs(z), 0.0)
    ez, ez2 = (p * az).sum(1), (p * az * az).sum(1)
    ls = np.where(fine, lse - m, 0.0)
    D = depth(x.shape[1])
    ds = U * (D + 4 + 4 * ez)
    base = ds + 4 * U * np.abs(ls)
    _near(out["lse"], lse, base + 4 * U * (np.abs(m) + np.where(fine, np.abs(lse), 0)),
          what + "lse")
    if out.get("entropy") is not None:
        _near(out["entropy"], want["entropy"],
              base + U * (ez * (2 * D + 12) + 8 * ez2), what + "entropy")
    if out.get("logp") is not None:
        w = want["logp"]
        _near(out["logp"], w, base + 6 * U * np.where(np.isfinite(w), np.abs(w), 0)
              + 6 * U * np.abs(ls), what + "logp")
    if out.get("top_ids") is not None:
        assert np.array_equal(np.asarray(out["top_ids"]), want["top_ids"]), what + "top_ids"
    if out.get("top_logp") is not None:
        w = want["top_logp"]
        _near(out["top_logp"], w, (base + 6 * U * np.abs(ls))[:, None]
              + 6 * U * np.where(np.isfinite(w), np.abs(w), 0), what + "top_logp")


def check_logprob_bwd(got, want, mag, factor, dtype, what="dlogits"):
    with np.errstate(invalid="ignore"):
        tol = 8 * U * mag + UT[dtype] * (np.abs(want) + 8 * U * mag) + TINY[dtype]
        # Probabilities below 2^-126 are taken as zero: what is lost is at most that times
        # scale (|g| + |h| (|log p| + H)), and |log p| < 104 down to FP32's last subnormal
        # number (beyond, p |log p| only falls). One more rounding of each.
        tol = tol + 2.0 ** -126 * factor * (1 + 8 * U)
    _near(got, want, tol, what)
