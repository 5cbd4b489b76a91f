"""Float64 definitions of the head operators: norms of queries and keys with the
position rotation and their gradient, slots of a paged cache, appending to it and
gathering from it. NumPy, sharing nothing with the CUDA sources.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def turn_matrix(d, rot, cos, sin, interleaved):
    """The rotation of one token as a [d, d] matrix."""
    m = np.eye(d)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        m[a, a], m[a, b], m[b, a], m[b, b] = cos[i], -sin[i], sin[i], cos[i]
    return m


def _turns(positions, table, n, d, interleaved):
    """([n, d, d] rotations, [n] whether the token has a position)."""
    if table is None or np.shape(table)[1] == 0:
        return np.broadcast_to(np.eye(d), (n, d, d)), np.ones(n, bool)
    table = np.asarray(table, np.float64)
    rot = table.shape[1]
    there = np.array([0 <= p < table.shape[0] for p in positions], bool)
    out = np.zeros((n, d, d))
    for t in range(n):
        if there[t]:
            row = table[int(positions[t])]
            out[t] = turn_matrix(d, rot, row[:rot // 2], row[rot // 2:], interleaved)
    return out, there


def rope(x, w, positions, table, eps, norm, interleaved):
    """(y, magnitude) of rows x [n, heads, d]: the magnitude is the sum of the absolute
    terms of each value."""
    x = np.asarray(x, np.float64)
    n, _, d = x.shape
    if norm:
        with np.errstate(divide="ignore", invalid="ignore"):
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if w is not None:
            x = x * np.asarray(w, np.float64)
    m, there = _turns(positions, table, n, d, interleaved)
    with np.errstate(invalid="ignore"):
        y = np.einsum("tij,thj->thi", m, x)
        mag = np.einsum("tij,thj->thi", np.abs(m), np.abs(x))
    y[~there], mag[~there] = 0, 0
    return y, mag


def rope_backward(dy, x, w, positions, table, eps, norm, interleaved):
    """dict of dx, its magnitudes (of the first term, of the second), and with a norm dw and
    the sum of its absolute terms."""
    dy = np.asarray(dy, np.float64)
    n, _, d = dy.shape
    m, there = _turns(positions, table, n, d, interleaved)
    dy = np.where(there[:, None, None], dy, 0)
    g = np.einsum("tij,thi->thj", m, dy)
    gm = np.einsum("tij,thi->thj", np.abs(m), np.abs(dy))
    if not norm:
        return {"dx": g, "mag1": gm, "mag2": np.zeros_like(g)}
    x = np.where(there[:, None, None], np.asarray(x, np.float64), 0)
    w = np.ones(d) if w is None else np.asarray(w, np.float64)
    with np.errstate(divide="ignore"):
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    r = np.where(there[:, None, None], r, 0)
    mean = (w * g * x).mean(-1, keepdims=True)
    mabs = (np.abs(w) * gm * np.abs(x)).mean(-1, keepdims=True)
    return {"dx": r * (w * g - x * r * r * mean), "mag1": r * np.abs(w) * gm,
            "mag2": r ** 3 * np.abs(x) * mabs, "dw": (g * x * r).sum((0, 1)),
            "dw_abs": (gm * np.abs(x) * r).sum((0, 1))}


def slots(page_table, starts, offsets, n, page_size):
    """(slots, positions) of a ragged batch, one token at a time."""
    s, p = np.full(n, -1, np.int64), np.full(n, -1, np.int64)
    limit = 2 ** 31 - 1
    for b in range(len(starts)):
        for t in range(max(0, int(offsets[b])), min(n, int(offsets[b + 1]))):
            pos = int(starts[b]) + t - int(offsets[b])
            if not 0 <= pos <= limit:
                continue
            p[t] = pos
            col = pos // page_size
            if col < page_table.shape[1]:
                page = int(page_table[b, col])
                if page >= 0 and (page + 1) * page_size <= limit:
                    s[t] = page * page_size + pos % page_size
    return s, p


def append(cache, rows, slot_ids, scale=1.0, eight=False):
    """The cache [pages, page_size, heads, d] with rows [n, heads, d] in their slots, before
    any rounding; and which of it was written."""
    out = np.array(cache, np.float64)
    hit = np.zeros(out.shape[:2], bool)
    page = out.shape[1]
    for t, s in enumerate(np.asarray(slot_ids).reshape(-1)):
        if 0 <= s < out.shape[0] * page:
            y = np.asarray(rows[t], np.float64) / scale
            out[s // page, s % page] = np.clip(y, -E4M3_MAX, E4M3_MAX) if eight else y
            hit[s // page, s % page] = True
    return out, hit


def gather(cache, slot_ids, scale=1.0):
    """Rows of slots, zeros outside the cache."""
    cache = np.asarray(cache, np.float64)
    page = cache.shape[1]
    ids = np.asarray(slot_ids).reshape(-1)
    out = np.zeros((ids.size, *cache.shape[2:]))
    for t, s in enumerate(ids):
        if 0 <= s < cache.shape[0] * page:
            out[t] = cache[s // page, s % page] * scale
    return out
