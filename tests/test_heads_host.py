"""The head operators on the host: the oracle against closed forms and differences,
argument checks before any CUDA call, the binding's refusals, and the rule on overlapping
rows (no GPU needed)."""
import math
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
from oracle import heads as oh
from row_wise_normalization_gb300 import capi
from test_tokens_rules import CSRC

A = 1 << 32          # fake, aligned addresses; never dereferenced
STEP = 1 << 32
SIZE, NULL, ALIGN = capi.RN_ERR_SIZE, capi.RN_ERR_NULL, capi.RN_ERR_ALIGN
ALIAS, DTYPE, SCALE, EPS = capi.RN_ERR_ALIAS, capi.RN_ERR_DTYPE, capi.RN_ERR_SCALE, capi.RN_ERR_EPS


# ---- the oracle ------------------------------------------------------------
def _table(rng, rows, rot):
    a = rng.uniform(-3, 3, (rows, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_turns_pairs_and_keeps_lengths(interleaved):
    rng = np.random.default_rng(0)
    d, rot, n = 10, 6, 4
    x, table = rng.standard_normal((n, 3, d)), _table(rng, 9, rot)
    pos = np.array([8, 0, 3, 9])
    y, _ = oh.rope(x, None, pos, table, 0.0, False, interleaved)
    assert not y[3].any()                       # no such position
    assert np.array_equal(y[..., rot:][:3], x[..., rot:][:3])
    for t in range(3):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            z = (x[t, :, a] + 1j * x[t, :, b]) * complex(table[pos[t], i],
                                                         table[pos[t], rot // 2 + i])
            assert np.allclose(y[t, :, a] + 1j * y[t, :, b], z, rtol=0, atol=1e-14)
    yn, _ = oh.rope(x[:3], np.ones(d), pos[:3], table, 0.0, True, interleaved)
    assert np.allclose((yn ** 2).mean(-1), 1, rtol=1e-12)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradient_against_differences(norm, interleaved):
    rng = np.random.default_rng(1)
    n, h, d, rot = 3, 2, 8, 6
    x, w = rng.standard_normal((n, h, d)), rng.standard_normal(d)
    dy, table = rng.standard_normal((n, h, d)), _table(rng, 5, rot)
    pos = np.array([4, 7, 1])
    f = lambda x, w: (dy * oh.rope(x, w, pos, table, 1e-3, norm, interleaved)[0]).sum()  # noqa: E731
    got = oh.rope_backward(dy, x, w, pos, table, 1e-3, norm, interleaved)
    e = 1e-6
    for at in np.ndindex(n, h, d):
        p, m = x.copy(), x.copy()
        p[at] += e
        m[at] -= e
        assert abs((f(p, w) - f(m, w)) / (2 * e) - got["dx"][at]) < 1e-7
    if norm:
        for j in range(d):
            p, m = w.copy(), w.copy()
            p[j] += e
            m[j] -= e
            assert abs((f(x, p) - f(x, m)) / (2 * e) - got["dw"][j]) < 1e-7
    assert not got["dx"][1].any()


def test_oracle_cache_holds_what_was_appended():
    rng = np.random.default_rng(2)
    table = np.array([[2, 0, 5], [1, 4, -1]])
    s, p = oh.slots(table, [3, 0], [0, 4, 7], 9, 4)
    assert s.tolist() == [11, 0, 1, 2, 4, 5, 6, -1, -1] and p.tolist() == [3, 4, 5, 6, 0, 1, 2, -1, -1]
    s2, p2 = oh.slots(table, [8], [0, 3], 3, 4)
    assert s2.tolist() == [20, 21, 22] and p2.tolist() == [8, 9, 10]
    s3, p3 = oh.slots(table[1:], [7, ], [0, 2], 2, 4)
    assert s3.tolist() == [19, -1] and p3.tolist() == [7, 8]
    cache = rng.standard_normal((6, 4, 2, 3))
    rows = rng.standard_normal((9, 2, 3))
    new, hit = oh.append(cache, rows, s)
    assert np.array_equal(new[~hit], cache[~hit]) and hit.sum() == 7
    got = oh.gather(new, s)
    assert np.array_equal(got[:7], rows[:7]) and not got[7:].any()


# ---- argument checks -------------------------------------------------------
def _h(at, heads=4, bs=0, ts=32, hs=8):
    return capi.heads(at, heads, bs, ts, hs)


_PARTS = struct.Struct("Q4q").unpack


def _qk(**kw):
    a = dict(q=_h(A), k=_h(A + STEP), wq=A + 2 * STEP, wk=A + 3 * STEP, positions=A + 4 * STEP,
             table=A + 5 * STEP, table_rows=100, table_stride=8, rot=8, batch=1, len=5, d=8, dtype=0,
             itype=1, norm=1, interleaved=0, eps=1e-5, zero=0)
    a.update(kw)
    return capi.qk(*_PARTS(a.pop("q")), *_PARTS(a.pop("k")), *a.values())


_IN = set("q k wq wk positions table table_rows table_stride rot batch len d dtype itype norm "
          "interleaved eps".split())


def _split(kw):
    return {k: v for k, v in kw.items() if k in _IN}, {k: v for k, v in kw.items() if k not in _IN}


def _fwd(**kw):
    i, o = _split(kw)
    a = dict(q_out=_h(A + 6 * STEP), k_out=_h(A + 7 * STEP))
    a.update(o)
    return capi.qk_rope_fwd(_qk(**i), **a)


def _bwd(**kw):
    i, o = _split(kw)
    a = dict(dq_out=_h(A + 6 * STEP), dk_out=_h(A + 7 * STEP), dq=_h(A + 8 * STEP),
             dk=_h(A + 9 * STEP), dwq=A + 10 * STEP, dwk=A + 11 * STEP, workspace=A + 12 * STEP,
             workspace_bytes=1 << 20)
    a.update(o)
    return capi.qk_rope_bwd(_qk(**i), **a)


def _cache(**kw):
    a = dict(k=A + 13 * STEP, v=A + 14 * STEP, kp=128, ks=32, kh=8, vp=128, vs=32, vh=8, pages=10,
             page=4, dv=8, dtype=0, k_scale=1.0, v_scale=1.0, zero=0)
    a.update(kw)
    return capi.cache(*a.values())


def _app(**kw):
    i, o = _split(kw)
    a = dict(q_out=_h(A + 6 * STEP), v=_h(A + 7 * STEP), cache=_cache(), slots=A + 8 * STEP)
    a.update(o)
    return capi.kv_append(_qk(**i), **a)


def _gat(**kw):
    a = dict(cache=_cache(), d=8, slots=A, itype=1, n=5, dtype=0, k_out=_h(A + STEP),
             v_out=_h(A + 2 * STEP))
    a.update(kw)
    return capi.kv_gather(**a)


def _slo(**kw):
    a = dict(itype=0, page_table=A, ld=6, width=6, starts=A + STEP, offsets=A + 2 * STEP, seqs=3,
             page_size=16, slots=A + 3 * STEP, positions=A + 4 * STEP, n=7)
    a.update(kw)
    return capi.kv_slots(**a)


# of q, k and their description, for every call that takes them
COMMON = [
    (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE), (dict(itype=2), DTYPE), (dict(d=0), SIZE),
    (dict(d=7), SIZE), (dict(d=514), SIZE), (dict(rot=3), SIZE), (dict(rot=10), SIZE),
    (dict(rot=-2), SIZE), (dict(batch=-1), SIZE), (dict(len=-1), SIZE), (dict(len=1 << 31), SIZE),
    (dict(batch=1 << 20, len=1 << 12), SIZE), (dict(table_rows=0), SIZE),
    (dict(table_stride=7), SIZE), (dict(eps=-1.0), EPS), (dict(eps=math.nan), EPS),
    (dict(eps=math.inf), EPS), (dict(positions=0), NULL), (dict(table=0), NULL),
    (dict(positions=A + 4 * STEP + 4), ALIGN), (dict(table=A + 5 * STEP + 2), ALIGN),
    (dict(wq=A + 1), ALIGN), (dict(wk=A + 2), ALIGN), (dict(q=_h(A, ts=-1)), SIZE),
    (dict(q=_h(A, hs=1 << 60)), SIZE), (dict(q=_h(A, heads=-1)), SIZE),
    (dict(k=_h(A + STEP, heads=65536)), SIZE), (dict(q=_h(0)), NULL), (dict(k=_h(0)), NULL),
    (dict(q=_h(A + 2)), ALIGN), (dict(k=_h(A + STEP + 1)), ALIGN),
]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(q=_h(0, 0), k=_h(0, 0)), SIZE), (dict(q_out=_h(A + 6 * STEP, heads=3)), SIZE),
    (dict(k_out=None), NULL), (dict(q_out=_h(0)), NULL), (dict(q_out=_h(A + 6 * STEP + 2)), ALIGN),
    (dict(q_out=_h(A + 4)), ALIAS), (dict(q_out=_h(A, ts=64)), ALIAS),
    (dict(q_out=_h(A + STEP)), ALIAS), (dict(k_out=_h(A + 6 * STEP + 16)), ALIAS),
    (dict(q_out=_h(A + 2 * STEP)), ALIAS), (dict(k_out=_h(A + 4 * STEP)), ALIAS),
    (dict(k_out=_h(A + 5 * STEP + 128)), ALIAS), (dict(q_out=_h(A + 6 * STEP, ts=0)), ALIAS),
    (dict(q_out=_h(A + 6 * STEP, hs=4)), ALIAS), (dict(q_out=_h(A + 6 * STEP, ts=28)), ALIAS),
    (dict(len=0, q=_h(0), k=_h(0), q_out=None, k_out=None), capi.RN_OK),
    (dict(batch=0, positions=0), capi.RN_OK),
])
def test_qk_rope_fwd_checks(kw, want):
    assert _fwd(**kw) == want


def test_null_struct():
    assert capi.qk_rope_fwd(None, None, None) == NULL
    assert capi.qk_rope_bwd(None, None, None, None, None, 0, 0, 0, 0) == NULL
    assert capi.kv_append(None, None, None, None, 0) == NULL
    assert capi.kv_gather(None, 8, A, 1, 4, 0, None, None) == NULL


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(dq_out=_h(A + 6 * STEP, heads=5)), SIZE), (dict(dk=None), NULL),
    (dict(dk_out=_h(0)), NULL), (dict(dq=_h(A + 8 * STEP + 2)), ALIGN),
    (dict(dwq=A + 10 * STEP + 2), ALIGN), (dict(wq=0), NULL), (dict(wk=0), NULL),
    (dict(norm=0), NULL), (dict(workspace=0), NULL), (dict(workspace=A + 12 * STEP + 8), ALIGN),
    (dict(workspace_bytes=100), SIZE), (dict(dq=_h(A + 4)), ALIAS), (dict(dq=_h(A + STEP)), ALIAS),
    (dict(dq=_h(A + 7 * STEP)), ALIAS), (dict(dk=_h(A + 6 * STEP)), ALIAS),
    (dict(dk=_h(A + 8 * STEP)), ALIAS), (dict(dwq=A + 8 * STEP), ALIAS),
    (dict(dwk=A + 10 * STEP + 4), ALIAS), (dict(workspace=A + 9 * STEP), ALIAS),
    (dict(workspace=A + 6 * STEP), ALIAS), (dict(workspace=A + 11 * STEP), ALIAS),
    (dict(dwq=A), ALIAS), (dict(dq=_h(A + 8 * STEP, hs=0)), ALIAS),
    (dict(len=0, dwq=0, dwk=0, workspace=0), capi.RN_OK),
])
def test_qk_rope_bwd_checks(kw, want):
    assert _bwd(**kw) == want


def test_workspace_size():
    assert capi.qk_rope_bwd_workspace_size(128) == 2432 * 128 * 4
    for bad in (0, 3, -2, 514):
        with pytest.raises(capi.RowNormError):
            capi.qk_rope_bwd_workspace_size(bad)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(rot=0, itype=7), DTYPE), (dict(k=_h(0, 0)), SIZE), (dict(v=_h(A + 7 * STEP, heads=3)), SIZE),
    (dict(v=None), NULL), (dict(cache=None), NULL), (dict(slots=0), NULL), (dict(q_out=None), NULL),
    (dict(v=_h(0)), NULL), (dict(slots=A + 8 * STEP + 4), ALIGN), (dict(v=_h(A + 7 * STEP + 2)), ALIGN),
    (dict(cache=_cache(dtype=1)), DTYPE), (dict(cache=_cache(dtype=4)), DTYPE),
    (dict(cache=_cache(pages=-1)), SIZE), (dict(cache=_cache(page=0)), SIZE),
    (dict(cache=_cache(pages=1 << 20, page=1 << 12)), SIZE), (dict(cache=_cache(dv=7)), SIZE),
    (dict(cache=_cache(dv=514)), SIZE), (dict(cache=_cache(kp=-1)), SIZE),
    (dict(cache=_cache(k=0)), NULL), (dict(cache=_cache(v=A + 14 * STEP + 2)), ALIGN),
    (dict(cache=_cache(k_scale=2.0)), SCALE), (dict(cache=_cache(dtype=3, k_scale=0.0)), SCALE),
    (dict(cache=_cache(dtype=3, v_scale=math.inf)), SCALE),
    (dict(cache=_cache(dtype=3, v_scale=-1.0)), SCALE),
    (dict(cache=_cache(dtype=3, v_scale=1e-40)), SCALE),
    (dict(cache=_cache(dtype=3, k_scale=math.nan)), SCALE),
    (dict(cache=_cache(v=A + 13 * STEP + 64)), ALIAS), (dict(cache=_cache(kp=64)), ALIAS),
    (dict(cache=_cache(kh=4)), ALIAS), (dict(cache=_cache(k=A + 64)), ALIAS),
    (dict(cache=_cache(v=A + STEP)), ALIAS), (dict(cache=_cache(v=A + 7 * STEP)), ALIAS),
    (dict(cache=_cache(k=A + 8 * STEP)), ALIAS), (dict(q_out=_h(A + 13 * STEP)), ALIAS),
    (dict(q_out=_h(A + 4)), ALIAS), (dict(q_out=_h(A + STEP)), ALIAS),
    (dict(len=0, slots=0, v=_h(0)), capi.RN_OK),
])
def test_kv_append_checks(kw, want):
    assert _app(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(dtype=1), DTYPE), (dict(itype=2), DTYPE), (dict(n=-1), SIZE),
    (dict(n=1 << 31), SIZE), (dict(d=9), SIZE), (dict(d=514), SIZE), (dict(k_out=_h(A, heads=0)), SIZE),
    (dict(v_out=_h(A + 2 * STEP, heads=3)), SIZE), (dict(k_out=None), NULL), (dict(k_out=_h(0)), NULL),
    (dict(slots=0), NULL), (dict(slots=A + 4), ALIGN), (dict(v_out=_h(A + 2 * STEP + 2)), ALIGN),
    (dict(k_out=_h(A + 2 * STEP + 64)), ALIAS), (dict(k_out=_h(A + 13 * STEP)), ALIAS),
    (dict(v_out=_h(A)), ALIAS), (dict(v_out=_h(A + 2 * STEP, ts=24)), ALIAS),
    (dict(cache=_cache(dtype=3, k_scale=-1.0)), SCALE), (dict(cache=_cache(v_scale=3.0)), SCALE),
    (dict(n=0, slots=0, k_out=_h(0), v_out=_h(0)), capi.RN_OK),
])
def test_kv_gather_checks(kw, want):
    assert _gat(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(itype=2), DTYPE), (dict(n=-1), SIZE), (dict(n=1 << 31), SIZE), (dict(seqs=-1), SIZE),
    (dict(width=-1), SIZE), (dict(ld=5), SIZE), (dict(page_size=0), SIZE),
    (dict(page_size=1 << 31), SIZE), (dict(page_table=0), NULL), (dict(starts=0), NULL),
    (dict(offsets=0), NULL), (dict(slots=0), NULL), (dict(page_table=A + 2), ALIGN),
    (dict(starts=A + STEP + 1), ALIGN), (dict(positions=A + 4 * STEP + 2), ALIGN),
    (dict(slots=A + 8), ALIAS), (dict(slots=A + 4 * STEP + 4), ALIAS),
    (dict(positions=A + 2 * STEP + 4), ALIAS), (dict(positions=A + STEP), ALIAS),
    (dict(n=0, slots=0, offsets=0), capi.RN_OK),
])
def test_kv_slots_checks(kw, want):
    assert _slo(**kw) == want


def test_binding_refusals():
    q, k = torch.zeros(4, 2, 8), torch.zeros(4, 1, 8)
    pos, table = torch.zeros(4, dtype=torch.int64), torch.zeros(9, 8)
    w = torch.zeros(8)
    kc = torch.zeros(3, 4, 1, 8)
    for bad, kind in [
        (lambda: rn.qk_rope_fwd([1], k), TypeError),
        (lambda: rn.qk_rope_fwd(q.double(), k), TypeError),
        (lambda: rn.qk_rope_fwd(q[0], k), ValueError),
        (lambda: rn.qk_rope_fwd(q, k, pos, table.double()), (TypeError, ValueError)),
        (lambda: rn.qk_rope_fwd(q, k, pos.float(), table), (TypeError, ValueError)),
        (lambda: rn.kv_append(k, k, pos.to(torch.int16), kc, kc), TypeError),
        (lambda: rn.kv_append(k, k, [0], kc, kc), TypeError),
        (lambda: rn.kv_gather([0], kc, pos), TypeError),
        (lambda: rn.kv_gather(kc, kc, pos, dtype=torch.float64), TypeError),
        (lambda: rn.kv_slots(pos, pos, pos, 4, 16), (TypeError, ValueError)),
        (lambda: rn.kv_slots([[0]], pos, pos, 4, 16), TypeError),
        (lambda: rn.qk_rope_bwd(q.int(), k, q, k, wq=w), TypeError),
    ]:
        with pytest.raises(kind):
            bad()


# ---- overlapping rows ------------------------------------------------------
def test_boxes_that_are_called_apart_share_nothing(tmp_path):
    """Every pair of small boxes, byte by byte: none called apart shares a byte, none whose
    runs are called apart meets itself; blocks of one matrix are told apart."""
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src, exe = tmp_path / "boxes.cpp", tmp_path / "boxes"
    src.write_text(r"""
#include <cstdio>
#include <map>
#include <random>
#include "rn_boxes.h"
using namespace rn;
static std::map<long, int> bytes(const Box& b) {
    std::map<long, int> m;
    for (long i = 0; i < b.count[0]; ++i)
        for (long j = 0; j < b.count[1]; ++j)
            for (long k = 0; k < b.count[2]; ++k)
                for (long r = 0; r < b.run; ++r)
                    ++m[(long)(uintptr_t)b.p + i * b.stride[0] + j * b.stride[1] + k * b.stride[2] + r];
    return m;
}
int main() {
    std::mt19937 g(7);
    auto pick = [&](int a, int b) { return (long)(a + g() % (b - a + 1)); };
    long wrong = 0, told = 0, close = 0;
    for (int t = 0; t < 60000; ++t) {
        Box x[2];
        const long m = pick(4, 40);
        for (Box& b : x) {
            b.p = (const void*)(uintptr_t)pick(100, 160);
            b.run = pick(1, 6);
            for (int i = 0; i < 3; ++i) {
                b.count[i] = pick(1, 4);
                b.stride[i] = pick(0, 2) == 0 ? m * pick(1, 3) : pick(0, 12);
            }
        }
        const auto a = bytes(x[0]), b = bytes(x[1]);
        bool meet = false, self = false;
        for (auto& e : a) meet |= b.count(e.first) > 0, self |= e.second > 1;
        const bool said = apart(x[0], x[1]);
        wrong += (said && meet) || (said != apart(x[1], x[0]) && meet);
        wrong += runs_apart(x[0]) && self;
        const bool ranges = (uintptr_t)x[0].p + extent(x[0]) <= (uintptr_t)x[1].p ||
                            (uintptr_t)x[1].p + extent(x[1]) <= (uintptr_t)x[0].p;
        told += said && !ranges;
        close += !said && !meet;
    }
    // queries, keys and values as column blocks; keys and values as halves of every page
    char* const p = (char*)(1 << 20);
    const Box q = {p, {1, 50, 8}, {0, 640, 32}, 32}, k = {p + 256, {1, 50, 2}, {0, 640, 32}, 32},
              v = {p + 320, {1, 50, 2}, {0, 640, 32}, 32};
    const Box kc = {p, {9, 4, 2}, {512, 64, 32}, 32}, vc = {p + 256, {9, 4, 2}, {512, 64, 32}, 32};
    printf("%ld %d %d %d %d %d", wrong, told > 100, apart(q, k) && apart(k, v) && apart(v, q),
           apart(kc, vc), apart(q, q), apart(Box{}, q));
    return 0;
}
""")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                           str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split() == ["0", "1", "1", "1", "0", "1"]
