"""Float64 definitions of the token operators: embedding rows and their
gradient, log probabilities with entropies and alternatives, and their
gradient. NumPy, row by row, sharing nothing with the CUDA sources.
"""
from __future__ import annotations

import numpy as np


def embed(tokens, table, scale):
    """scale * table[tokens]; rows of zeros for ids outside the table."""
    table = np.asarray(table, np.float64)
    tokens = np.asarray(tokens).reshape(-1)
    out = np.zeros((tokens.size, table.shape[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[i] = scale * table[t]
    return out


def embed_backward(dout, tokens, vocab, scale):
    """(gradient, sum of the absolute terms, terms of each row)."""
    dout = np.asarray(dout, np.float64)
    g = np.zeros((vocab, dout.shape[1]))
    a = np.zeros_like(g)
    m = np.zeros(vocab, np.int64)
    for i, t in enumerate(np.asarray(tokens).reshape(-1)):
        if 0 <= t < vocab:
            g[t] += dout[i]
            a[t] += np.abs(dout[i])
            m[t] += 1
    return scale * g, abs(scale) * a, m


def log_softmax(logits, scale):
    """(log p, lse) of each row; a row of nothing but -inf: (-inf, -inf); a row
    with a NaN or a +inf: NaN."""
    x = scale * np.asarray(logits, np.float64)
    lq = np.empty_like(x)
    lse = np.empty(x.shape[0])
    for i, r in enumerate(x):
        if np.isnan(r).any() or (r == np.inf).any():
            lq[i], lse[i] = np.nan, np.nan
            continue
        m = r.max()
        if m == -np.inf:
            lq[i], lse[i] = -np.inf, -np.inf
            continue
        ls = np.log(np.exp(r - m).sum())
        lse[i] = m + ls
        lq[i] = (r - m) - ls      # (m may be too large to hold log S beside it)
    return lq, lse


def _plogp(lq):
    with np.errstate(invalid="ignore"):
        return np.where(lq == -np.inf, 0.0, np.exp(lq) * lq)


def logprob(logits, targets, scale, top=0):
    """dict of logp, entropy, lse, top_ids, top_logp."""
    lq, lse = log_softmax(logits, scale)
    rows, vocab = lq.shape
    out = {"lse": lse, "entropy": -_plogp(lq).sum(1) + 0.0}
    if targets is not None:
        lp = np.zeros(rows)
        for i, t in enumerate(np.asarray(targets).reshape(-1)):
            if 0 <= t < vocab:
                lp[i] = lq[i, t]
        out["logp"] = lp
    x = np.asarray(logits, np.float64)
    order = np.where(np.isnan(x), np.inf, x + 0.0)
    first = np.isnan(x)
    ids = np.stack([np.lexsort((np.arange(vocab), -order[i], ~first[i]))[:top]
                    for i in range(rows)]) if rows else np.zeros((0, top), np.int64)
    out["top_ids"] = ids
    out["top_logp"] = np.take_along_axis(lq, ids, 1)
    return out


def logprob_backward(dlogp, dentropy, logits, targets, lse, entropy, scale):
    """(gradient, magnitude, factor): magnitude bounds each term of the sum that
    makes an element, factor what a probability below 2^-126 is multiplied by in it (its
    logarithm taken as -104, that of FP32's last subnormal number). lse None: log
    probabilities from the logits themselves."""
    x = scale * np.asarray(logits, np.float64)
    lq = None
    if lse is None:
        lq, lse = log_softmax(logits, scale)
    d = np.zeros_like(x)
    mag = np.zeros_like(x)
    factor = np.zeros((x.shape[0], 1))
    for i in range(x.shape[0]):
        t = -1 if targets is None else int(targets[i])
        there = 0 <= t < x.shape[1]
        g = float(dlogp[i]) if dlogp is not None and there else 0.0
        h = float(dentropy[i]) if dentropy is not None else 0.0
        if (g == 0 and h == 0) or lse[i] == -np.inf:
            continue
        z = x[i] - lse[i] if lq is None else lq[i]
        p = np.exp(z)
        zp = np.where(p > 0, z, 0.0)
        H = float(entropy[i]) if dentropy is not None else 0.0
        d[i] = -scale * p * (g + h * (zp + H))
        factor[i] = scale * (abs(g) + abs(h) * (104 + abs(H)))
        mag[i] = scale * p * (abs(g) + abs(h) * (np.abs(zp) + abs(H))) * (1 + np.abs(zp))
        if there:
            d[i, t] += scale * g
            mag[i, t] += scale * abs(g)
    return d, mag, factor
