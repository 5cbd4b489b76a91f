"""Slots of a paged cache, appending to it with norm and rotation, gathering from it, against
the float64 definitions; and the head operators together, as a served and a trained layer."""
import threading

import numpy as np
import pytest
import torch

import head_checks
import row_wise_normalization_gb300 as rn
from oracle import heads as oh
from test_gpu_heads import EPS, IT, TYPES, Case, _bits, table_of
from token_util import DT, f64, rounded

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


# ---- slots -----------------------------------------------------------------
def _slots(table, starts, offsets, n, page, itype, **kw):
    t = [torch.as_tensor(np.asarray(a, np.int64)).to(IT[itype]).cuda() for a in (table, starts, offsets)]
    s, p = rn.kv_slots(*t, n, page, **kw)
    assert s.dtype is IT[itype] and p.dtype is IT[itype]
    return s.cpu().numpy().astype(np.int64), p.cpu().numpy().astype(np.int64)


@pytest.mark.parametrize("itype", ["i32", "i64"])
@pytest.mark.parametrize("seqs,most,context,page,pad,first", [
    (1, 1, 0, 1, 0, 0), (1, 300, 7, 16, 0, 0), (61, 1, 500, 16, 3, 0), (9, 40, 90, 7, 5, 0),
    (255, 9, 33, 64, 0, 0), (700, 3, 10, 5, 600, 2), (4095, 2, 4, 3, 1, 0), (4096, 2, 4, 3, 0, 0),
    (6000, 3, 4, 128, 9, 1), (3, 0, 4, 16, 10, 0),
])
def test_slots(seqs, most, context, page, pad, first, itype):
    rng = np.random.default_rng([seqs, most, page])
    new = rng.integers(0, most + 1, seqs)
    if most == 1:
        new[:] = 1
    offsets = first + np.concatenate([[0], new.cumsum()])
    starts = rng.integers(0, context + 1, seqs)
    width = (context + most) // page + 1
    table = rng.permutation(seqs * width).reshape(seqs, width)
    n = int(offsets[-1]) + pad
    want = oh.slots(table, starts, offsets, n, page)
    got = _slots(table, starts, offsets, n, page, itype)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("itype", ["i32", "i64"])
def test_slots_that_do_not_exist(itype):
    big = 2 ** 31 - 1
    table = np.array([[3, -1, big, 2], [0, big // 16 - 1, 5, big // 16]])
    starts, offsets = [10, -20], [0, 60, 110]
    want = oh.slots(table, starts, offsets, 112, 16)
    got = _slots(table, starts, offsets, 112, 16, itype)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert (want[0] >= 0).any() and (want[1][60:80] == -1).all()
    starts = [big - 3, 0]
    want = oh.slots(table, starts, [0, 8, 9], 9, 1)
    got = _slots(table, starts, [0, 8, 9], 9, 1, itype)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    if itype == "i64":
        got = _slots(np.full((2, 4), 2 ** 62), [2 ** 40, 3], [0, 2, 4], 4, 16, itype)
        assert (got[0] == -1).all() and got[1].tolist() == [-1, -1, 3, 4]
    # no sequence, no page, no token
    assert (_slots(np.zeros((0, 3)), [], [0], 4, 16, itype)[0] == -1).all()
    got = _slots(np.zeros((1, 0)), [2], [0, 3], 3, 16, itype)
    assert (got[0] == -1).all() and got[1].tolist() == [2, 3, 4]
    assert _slots(table, starts, [0, 0, 0], 0, 16, itype)[0].size == 0


def test_slots_from_a_wider_table_into_given_memory():
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.permutation(5 * 40).reshape(5, 40)).int().cuda()
    starts, offsets = torch.arange(5).int().cuda(), (torch.arange(6) * 30).int().cuda()
    slots = torch.full((160,), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((160,), 77, dtype=torch.int32, device="cuda")
    got = rn.kv_slots(wide[:, 5:14], starts, offsets, 153, 4, slots=slots[3:156], positions=pos[4:157])
    want = oh.slots(wide[:, 5:14].cpu().numpy(), starts.cpu(), offsets.cpu(), 153, 4)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    assert bool((slots[:3] == 77).all()) and bool((slots[156:] == 77).all())
    assert bool((pos[:4] == 77).all()) and bool((pos[157:] == 77).all())
    with pytest.raises(TypeError):
        rn.kv_slots(wide, starts.long(), offsets, 10, 4)
    with pytest.raises(ValueError):
        rn.kv_slots(wide, starts, offsets[1:], 10, 4)
    with pytest.raises(ValueError):
        rn.kv_slots(wide.t(), starts, offsets, 10, 4)
    with pytest.raises(rn.RowNormError):
        rn.kv_slots(wide, starts, offsets, 10, 0)


# ---- the cache -------------------------------------------------------------
def make_cache(rng, layout, pages, page, heads, d, dv, dtype):
    """(whole tensors, k_cache, v_cache) full of values; what neither holds is part of the
    whole tensors."""
    def new(*shape):
        a = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
        return a.to(dtype)

    if layout == "by_token":
        w = new(pages, page, heads, d), new(pages, page, heads, dv)
        return w, w[0], w[1]
    if layout == "by_head":
        w = new(pages, heads, page, d), new(pages, heads, page, dv)
        return w, w[0].transpose(1, 2), w[1].transpose(1, 2)
    if layout == "halves":                    # keys and values as halves of every page
        w = new(pages, 2, page, heads, max(d, dv))
        return (w,), w[:, 0, :, :, :d], w[:, 1, :, :, :dv]
    if layout == "side_by_side":              # a head's key and value in one row
        w = new(pages, page, heads, d + dv)
        return (w,), w[..., :d], w[..., d:]
    w = new(3, pages, page + 1, heads, d + 1), new(pages, page, heads, dv)
    return w, w[0][1, :, :page, :, :d], w[1]  # a layer of many, ragged in every direction


LAYOUTS = ["by_token", "by_head", "halves", "side_by_side", "ragged"]


def _marked(whole, k, v, hit):
    """Which elements of the whole tensors slots of `hit` cover."""
    out = []
    for w in whole:
        m = torch.zeros(w.shape, dtype=torch.bool, device="cuda")
        for c in (k, v):
            if c.untyped_storage().data_ptr() == w.untyped_storage().data_ptr():
                view = m.as_strided(c.shape, c.stride(), c.storage_offset() - w.storage_offset())
                view[torch.from_numpy(hit).cuda()] = True
        out.append(m)
    return out


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "e4m3"),
                                         ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,hq,hk,d,dv,rot,page,norm,itype", [
    (1, 4, 1, 64, 64, 64, 16, True, "i64"), (37, 8, 2, 128, 128, 128, 7, True, "i32"),
    (20, 0, 3, 80, 80, 20, 1, False, "i64"), (33, 6, 3, 34, 34, 34, 16, True, "i32"),
    (19, 2, 2, 64, 128, 32, 5, True, "i64"), (23, 0, 4, 128, 32, 0, 64, False, "i32"),
    (9, 3, 1, 512, 512, 64, 4, True, "i32"), (14, 5, 1, 256, 18, 256, 3, True, "i64"),
])
def test_append(n, hq, hk, d, dv, rot, page, norm, itype, layout, dtype, cache):
    c = Case(n, hq or 1, hk, d, rot, dtype, norm, n % 2 == 1, itype)
    v = rounded(c.rng, (n, hk, dv), dtype, 2.0)
    pages = n // page + 3
    eight = cache == "e4m3"
    ks, vs = (float(np.float32(0.013)), 0.25) if eight else (1.0, 1.0)
    whole, kc, vc = make_cache(c.rng, layout, pages, page, hk, d, dv, E4M3 if eight else DT[dtype])
    ids = c.rng.permutation(pages * page)[:n]
    if n > 5:
        ids[[0, 3, n - 1]] = [-1, pages * page, -7]
    slots = torch.from_numpy(ids).to(IT[itype]).cuda()
    before = [w.clone() for w in whole]
    k0, v0 = f64(kc.float()), f64(vc.float())
    q = rn.kv_append(c.k, v, slots, kc, vc, c.pos, c.table, c.wk, EPS, q=c.q if hq else None,
                     wq=c.wq if hq else None, k_scale=ks, v_scale=vs, **c.kw)
    wk, mk = c.want("k")
    want_k, hit = oh.append(k0, wk, ids, ks, eight)
    want_v, _ = oh.append(v0, f64(v), ids, vs, eight)
    mag = np.zeros_like(want_k)
    live = [t for t in range(n) if 0 <= ids[t] < pages * page]
    for t in live:
        mag[ids[t] // page, ids[t] % page] = mk[t]
    if eight:
        head_checks.check_rope_e4m3(f64(kc.float())[hit], want_k[hit], mag[hit], norm, ks, "k")
        head_checks.check_rope_e4m3(f64(vc.float())[hit], want_v[hit],
                                    np.abs(want_v[hit]) * vs, False, vs, "v")
    else:
        head_checks.check_rope(f64(kc)[hit], want_k[hit], mag[hit], norm, dtype, "k")
        assert np.array_equal(f64(vc)[hit], want_v[hit])
    for w, b, m in zip(whole, before, _marked(whole, kc, vc, hit)):
        same = w.view(torch.uint8).view(*w.shape[:-1], w.shape[-1], -1) == \
            b.view(torch.uint8).view(*w.shape[:-1], w.shape[-1], -1)
        assert bool((same.all(-1) | m).all()), "another slot was written"
    if hq:
        ref = rn.qk_rope_fwd(c.q, None, c.pos, c.table, c.wq, None, EPS, **c.kw)[0]
        head_checks.check_rope(f64(q), *c.want("q"), norm, dtype, "q")
        assert norm is False or q.shape == ref.shape
    else:
        assert q is None
    # out again: the rows as they are held, zeros for those that are not
    for out_t in ([DT[dtype]] if not eight else [torch.float32, torch.bfloat16, torch.float16]):
        gk, gv = rn.kv_gather(kc, vc, slots, dtype=out_t, k_scale=ks, v_scale=vs)
        for got, cc, sc in ((gk, kc, ks), (gv, vc, vs)):
            want = torch.zeros(n, hk, cc.shape[-1], device="cuda")
            at = torch.tensor([ids[t] for t in live], device="cuda", dtype=torch.int64)
            want[torch.tensor(live, device="cuda", dtype=torch.int64)] = \
                cc.float()[at // page, at % page] * sc
            assert torch.equal(got, want.to(out_t))


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "e4m3"), ("f16", "f16")])
@pytest.mark.parametrize("hq,hk,d,rot,interleaved", [(2, 1, 64, 64, False), (1, 1, 128, 128, True), (3, 2, 64, 32, False),
                                                     (4, 1, 32, 32, False), (2, 1, 80, 40, True), (8, 2, 16, 16, False),
                                                     (5, 3, 64, 64, False), (2, 2, 256, 256, False)])
def test_many_tokens_of_few_heads(hq, hk, d, rot, interleaved, dtype, cache):
    """Long batches, whose warps take rows of several tokens: the same bits as in short ones, padding
    and tokens without a slot among them."""
    n = 20011
    rng = np.random.default_rng([n, hq, d])
    x = rounded(rng, (n, hq + 2 * hk, d), dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    w = rounded(rng, (d,), dtype)
    table = table_of(rng, 60, rot)
    pos = torch.from_numpy(rng.integers(-2, 62, n)).cuda()
    ids = rng.permutation(24000)[:n]
    ids[rng.random(n) < 0.05] = -1
    slots = torch.from_numpy(ids).cuda()
    t = E4M3 if cache == "e4m3" else DT[dtype]
    kw = dict(interleaved=interleaved)
    sc = dict(k_scale=0.25, v_scale=0.5) if cache == "e4m3" else {}

    def caches():
        return [torch.full((1500, 16, hk, d), 3.0, device="cuda").to(t) for _ in range(2)]

    whole, parts = caches(), caches()
    qa = rn.kv_append(k, v, slots, *whole, pos, table, w, q=q, wq=w, **kw, **sc)
    qf, kf = rn.qk_rope_fwd(q, k, pos, table, w, w, **kw)
    assert torch.equal(qa, qf)
    for a in range(0, n, 501):
        s = slice(a, a + 501)
        rn.kv_append(k[s], v[s], slots[s], *parts, pos[s], table, w, **kw, **sc)
        q1, k1 = rn.qk_rope_fwd(q[s], k[s], pos[s], table, w, w, **kw)
        assert torch.equal(q1, qf[s]) and torch.equal(k1, kf[s])
    for a, b in zip(whole, parts):
        assert torch.equal(_bits(a), _bits(b))
    # the gradient: the same bits again, and the weights' against its definition in 64 bits
    g = rounded(rng, (n, hq + hk, d), dtype)
    dq, dk, dwq, dwk = rn.qk_rope_bwd(g[:, :hq], g[:, hq:], q, k, pos, table, w, w, **kw)
    for a in range(0, n, 501):
        s = slice(a, a + 501)
        part = rn.qk_rope_bwd(g[s, :hq], g[s, hq:], q[s], k[s], pos[s], table, w, w, **kw)
        assert torch.equal(part[0], dq[s]) and torch.equal(part[1], dk[s])
    live = ((pos >= 0) & (pos < 60)).double()[:, None, None]
    row = table[pos.clamp(0, 59)].double()[:, None]
    cs, sn = row[..., :rot // 2], row[..., rot // 2:]
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    gd, xd = g.double() * live, x[:, :hq + hk].double()
    turn, mag = gd.clone(), gd.abs()
    turn[..., first] = gd[..., first] * cs + gd[..., second] * sn
    turn[..., second] = gd[..., second] * cs - gd[..., first] * sn
    mag[..., first] = (gd[..., first] * cs).abs() + (gd[..., second] * sn).abs()
    mag[..., second] = (gd[..., second] * cs).abs() + (gd[..., first] * sn).abs()
    r = (xd.square().mean(-1, keepdim=True) + EPS).rsqrt()
    for sl, dw in ((slice(0, hq), dwq), (slice(hq, None), dwk)):
        want = {"dw": f64((turn * xd * r)[:, sl].sum((0, 1))),
                "dw_abs": f64((mag * xd.abs() * r)[:, sl].sum((0, 1)))}
        head_checks.check_dw(f64(dw), want, n, hq + hk, dtype)
    # a batch of sequences, head by head
    b4 = lambda z: z[:20000].reshape(8, 2500, z.shape[1], d).transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    q4, k4 = rn.qk_rope_fwd(b4(q), b4(k), pos[:20000], table, w, w, **kw)
    assert torch.equal(q4.reshape(20000, hq, d), qf[:20000]) and torch.equal(k4.reshape(20000, hk, d), kf[:20000])
    # the rotation alone, and back
    r, _ = rn.qk_rope_fwd(q, None, pos, table, **kw)
    back = rn.qk_rope_bwd(r, None, None, None, pos, table, **kw)[0]
    there = (pos >= 0) & (pos < 60)
    assert not bool(back[~there].any())
    # two rotations of FP32 values with their roundings, cosines and sines of unit length to 2^-23
    far = (back - q)[there].double().abs().max()
    assert float(far) <= (4 * torch.finfo(DT[dtype]).eps + 2.0 ** -20) * float(q.double().abs().max())


def test_append_saturates_and_keeps_nan():
    k = torch.tensor([1e6, -1e6, 448.0, 465.0, float("inf"), -float("inf"), float("nan"), 0.0],
                     device="cuda").view(1, 1, 8).repeat(1, 1, 2)
    kc = torch.zeros(1, 1, 1, 16, device="cuda").to(E4M3)
    vc = torch.zeros(1, 1, 1, 16, device="cuda").to(E4M3)
    rn.kv_append(k, k, torch.zeros(1, dtype=torch.int32, device="cuda"), kc, vc, k_scale=1.0, v_scale=0.5)
    want = [448.0, -448.0, 448.0, 448.0, 448.0, -448.0]
    for c in (kc, vc):
        got = c.float().flatten()[:8].tolist()
        assert got[:6] == want and got[6] != got[6] and got[7] == 0


def test_append_turns_the_largest_values_without_nan():
    """The rotation comes before the scale: what it leaves finite is held at 448, not as NaN."""
    big = torch.finfo(torch.bfloat16).max * 0.5
    k = torch.full((1, 1, 64), big, dtype=torch.bfloat16, device="cuda")
    table = torch.cat([torch.full((1, 32), 0.6), torch.full((1, 32), 0.8)], 1).cuda()
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    kc, vc = (torch.zeros(1, 1, 1, 64, device="cuda").to(E4M3) for _ in range(2))
    rn.kv_append(k, -k, pos, kc, vc, pos, table, k_scale=0.001, v_scale=0.001)
    got = kc.float().flatten()
    assert bool((got[:32] == -448).all()) and bool((got[32:] == 448).all())
    assert bool((vc.float() == -448).all())
    # a norm's factor comes before the weights: a row beyond the squares' range gives zeros
    w = torch.full((64,), 1e30, dtype=torch.bfloat16, device="cuda")
    q, _ = rn.qk_rope_fwd(k, None, pos, table, w)
    assert not bool(q.any())


def test_every_e4m3_value_comes_out():
    bits = torch.arange(256, dtype=torch.uint8, device="cuda")
    kc = bits.view(E4M3).view(8, 1, 1, 32)
    vc = bits.flip(0).view(E4M3).view(8, 1, 1, 32)
    slots = torch.arange(8, device="cuda")
    for t in (torch.float32, torch.bfloat16, torch.float16):
        for d in (32, 30, 6):                 # every access width
            k, v = rn.kv_gather(kc[..., :d], vc[..., :d], slots, dtype=t, k_scale=0.375, v_scale=3.0)
            wk = (kc[..., :d].float() * 0.375).to(t).view(8, 1, d)
            wv = (vc[..., :d].float() * 3.0).to(t).view(8, 1, d)
            assert torch.equal(k.nan_to_num(7e4 if t != torch.float16 else 6e4),
                               wk.nan_to_num(7e4 if t != torch.float16 else 6e4))
            assert torch.equal(v.nan_to_num(6e4), wv.nan_to_num(6e4))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,heads,d,dv,page", [(1, 1, 64, 64, 16), (50, 5, 80, 80, 7), (300, 3, 34, 128, 1),
                                               (2500, 2, 128, 128, 64), (77, 9, 2, 6, 3)])
def test_gather(n, heads, d, dv, page, layout, dtype):
    rng = np.random.default_rng([n, d])
    pages = 40 // page + 2
    whole, kc, vc = make_cache(rng, layout, pages, page, heads, d, dv, DT[dtype])
    ids = rng.integers(-2, pages * page + 2, n)         # repeats, and slots beside the cache
    if n > 4:
        ids[:3] = [2 ** 31 - 1, -2 ** 31, pages * page - 1]
    slots = torch.from_numpy(ids).to(torch.int32 if n % 2 else torch.int64).cuda()
    # into column blocks of one matrix
    out = torch.full((n, heads, d + dv + 8), 7.0, dtype=DT[dtype], device="cuda")
    ko, vo = out[..., :d], out[..., d + 8:]
    got = rn.kv_gather(kc, vc, slots, k_out=ko, v_out=vo)
    assert got[0] is ko and got[1] is vo
    assert np.array_equal(f64(ko), oh.gather(f64(kc), ids)) and np.array_equal(f64(vo), oh.gather(f64(vc), ids))
    assert bool((out[..., d:d + 8] == 7).all())
    k, v = rn.kv_gather(kc, vc, slots)
    assert torch.equal(_bits(k), _bits(ko)) and torch.equal(_bits(v), _bits(vo))


def test_a_long_cache():
    """Slots whose offsets pass 2^32 bytes and 2^31 elements."""
    pages, page, heads, d = 300000, 16, 8, 64           # 4.9 GB of keys at 16 bits
    kc = torch.zeros(pages, page, heads, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(pages, heads, page, 2, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    rng = np.random.default_rng(0)
    n = 50
    k, v = rounded(rng, (n, heads, d), "bf16"), rounded(rng, (n, heads, 2), "bf16")
    ids = torch.from_numpy(rng.permutation(pages * page - 1)[:n]).cuda()
    ids[0] = pages * page - 1
    assert int(ids[0]) * heads * d > 2 ** 31
    rn.kv_append(k, v, ids, kc, vc)
    assert torch.equal(kc[ids // page, ids % page], k) and torch.equal(vc[ids // page, ids % page], v)
    gk, gv = rn.kv_gather(kc, vc, ids)
    assert torch.equal(gk, k) and torch.equal(gv, v)
    kc[ids // page, ids % page] = 0
    assert not bool(kc.any())


def test_refusals_of_the_binding():
    c = Case(16, 4, 2, 64, 64, "bf16")
    v = c.k.contiguous()
    slots = torch.arange(16, device="cuda")
    kc = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    e = torch.zeros(4, 8, 2, 64, device="cuda").to(E4M3)
    for bad, kind in [
        (lambda: rn.kv_append(c.k, v, slots[1:], kc, vc), ValueError),
        (lambda: rn.kv_append(c.k, v, slots.int(), kc, vc, c.pos, c.table), TypeError),
        (lambda: rn.kv_append(c.k, v[:, :1], slots, kc, vc), ValueError),
        (lambda: rn.kv_append(c.k, v.float(), slots, kc, vc), TypeError),
        (lambda: rn.kv_append(c.k, v, slots, kc.float(), vc.float()), TypeError),
        (lambda: rn.kv_append(c.k, v, slots, kc, e), TypeError),
        (lambda: rn.kv_append(c.k, v, slots, kc[:2], vc), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc[..., :32], vc), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc.transpose(2, 3), vc), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc[0], vc[0]), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc, kc), rn.RowNormError),
        (lambda: rn.kv_append(c.k, v, slots, kc, vc, k_scale=2.0), rn.RowNormError),
        (lambda: rn.kv_append(c.k, v, slots, e, e.clone(), v_scale=0.0), rn.RowNormError),
        (lambda: rn.kv_append(c.k, v, slots, kc, vc, q_out=v), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc, vc, wq=c.wq), ValueError),
        (lambda: rn.kv_append(c.k, v, slots, kc[:1].expand(4, 8, 2, 64), vc), rn.RowNormError),
        (lambda: rn.kv_gather(kc, vc, slots, dtype=torch.float16), TypeError),
        (lambda: rn.kv_gather(kc, e, slots), TypeError),
        (lambda: rn.kv_gather(kc, vc, slots, k_out=v[1:]), ValueError),
        (lambda: rn.kv_gather(kc, vc, slots.float()), TypeError),
        (lambda: rn.kv_gather(kc, vc, slots, k_out=kc.view(-1, 2, 64)[:16]), rn.RowNormError),
        (lambda: rn.kv_gather(kc, vc, slots, v_scale=2.0), rn.RowNormError),
    ]:
        with pytest.raises(kind):
            bad()
    assert not bool(kc.any()) and not bool(vc.any())
    # nothing to do
    none = slots[:0]
    assert rn.kv_append(c.k[:0], v[:0], none, kc, vc) is None
    assert rn.kv_gather(kc, vc, none)[0].shape == (0, 2, 64)
    empty = kc[:0]
    rn.kv_append(c.k, v, slots, empty, empty)
    assert not bool(rn.kv_gather(empty, empty, slots)[0].any())


# ---- together --------------------------------------------------------------
def _attend(q, k, v, first):
    """Causal attention of grouped heads in plain products: query i sees keys 0 .. first + i."""
    g = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(g, 1).double(), v.repeat_interleave(g, 1).double()
    s = torch.einsum("qhd,khd->hqk", q.double(), k) / q.shape[2] ** 0.5
    i = torch.arange(q.shape[0], device="cuda")[:, None] + first
    s = s.masked_fill(torch.arange(k.shape[0], device="cuda")[None] > i, -np.inf)
    return torch.einsum("hqk,khd->qhd", s.softmax(-1), v)


@pytest.mark.parametrize("graph", [False, True])
def test_a_served_layer_gives_what_whole_sequences_give(graph):
    """Prompts in two chunks, then tokens one at a time, of sequences of different lengths, with
    page tables, a padded batch and another stream: at every step the cache's rows are the
    whole sequence's keys, bit for bit, and attention over them is the same."""
    rng = np.random.default_rng(9)
    hq, hk, d, page, width = 8, 2, 64, 8, 12
    lens, steps = [31, 1, 17, 50, 8], 3
    seqs = len(lens)
    total = [n + steps for n in lens]
    x = [rounded(rng, (n, hq + 2 * hk, d), "bf16") for n in total]
    wq, wk = rounded(rng, (d,), "bf16"), rounded(rng, (d,), "bf16")
    table = table_of(rng, 200, d)
    page_table = torch.from_numpy(rng.permutation(seqs * width).reshape(seqs, width)).cuda()
    kc = torch.zeros(seqs * width, page, hk, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ref = [rn.qk_rope_fwd(t[:, :hq], t[:, hq:hq + hk], torch.arange(len(t), device="cuda"), table, wq, wk,
                          EPS) for t in x]
    done = [0] * seqs
    pad = 2
    state = {}

    def step(new):
        n = sum(new)
        offsets = torch.tensor([0] + list(np.cumsum(new)), device="cuda")
        starts = torch.tensor(done, device="cuda")
        rows = torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(seqs)] +
                         [torch.full((pad, hq + 2 * hk, d), 9.0, dtype=torch.bfloat16, device="cuda")])

        def run(rows, starts, offsets):
            slots, pos = rn.kv_slots(page_table, starts, offsets, n + pad, page)
            q = rn.kv_append(rows[:, hq:hq + hk], rows[:, hq + hk:], slots, kc, vc, pos, table, wk, EPS,
                             q=rows[:, :hq], wq=wq)
            return q, slots

        if graph and max(new) == 1:
            if "graph" not in state:
                state["in"] = rows.clone(), starts.clone(), offsets.clone()
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    run(*state["in"])
                torch.cuda.current_stream().wait_stream(side)
                state["graph"] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(state["graph"]):
                    state["out"] = run(*state["in"])
            for a, b in zip(state["in"], (rows, starts, offsets)):
                a.copy_(b)
            state["graph"].replay()
            q, slots = state["out"]
        else:
            q, slots = run(rows, starts, offsets)
        assert bool((slots[n:] == -1).all())
        at = 0
        for b in range(seqs):
            seen = done[b] + new[b]
            ends = torch.tensor([0, seen], device="cuda")
            whole, _ = rn.kv_slots(page_table[b:b + 1], torch.zeros(1, dtype=torch.int64, device="cuda"), ends,
                                   seen, page)
            k, v = rn.kv_gather(kc, vc, whole)
            assert torch.equal(k, ref[b][1][:seen]) and torch.equal(v, x[b][:seen, hq + hk:])
            if new[b]:
                qb = q[at:at + new[b]]
                assert torch.equal(qb, ref[b][0][done[b]:seen])
                a = _attend(qb, k, v, done[b])
                w = _attend(ref[b][0][:seen], ref[b][1][:seen], x[b][:seen, hq + hk:], 0)[done[b]:]
                assert torch.allclose(a, w, rtol=0, atol=1e-12)
            at += new[b]
            done[b] = seen

    step([n // 2 for n in lens])
    step([n - n // 2 for n in lens])
    for _ in range(steps):
        step([1] * seqs)
    # slots of nobody were never written
    used = torch.zeros(seqs * width * page, dtype=torch.bool, device="cuda")
    for b in range(seqs):
        s, _ = rn.kv_slots(page_table[b:b + 1], torch.zeros(1, dtype=torch.int64, device="cuda"),
                           torch.tensor([0, total[b]], device="cuda"), total[b], page)
        used[s] = True
    assert not bool(kc.view(-1, hk, d)[~used].any()) and not bool(vc.view(-1, hk, d)[~used].any())


def test_a_trained_layer_has_the_gradient_of_its_formula():
    """Embedding rows, a norm, a projection, queries and keys normed and turned, attention, logits
    and log probabilities, and the way back through this library's gradients: against automatic
    differentiation in 64 bits of the same inputs."""
    rng = np.random.default_rng(4)
    n, vocab, width, hq, hk, d = 40, 90, 48, 4, 2, 16
    new = lambda *s, std=1.0: rounded(rng, s, "f32", std)  # noqa: E731
    emb, gamma, proj = new(vocab, width), new(width), new(width, (hq + 2 * hk) * d, std=0.2)
    wq, wk, head = new(d), new(d), new(hq * d, vocab, std=0.2)
    table = table_of(rng, n, d)
    pos = torch.arange(n, device="cuda")
    tok = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
    tgt = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
    params = [t.double().requires_grad_() for t in (emb, gamma, proj, wq, wk, head)]

    def rms64(x, w):
        return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w

    def turn64(x):
        c, s = table.double()[pos][:, None, :d // 2], table.double()[pos][:, None, d // 2:]
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    e, g, p, a, b, h = params
    x = (rms64(e[tok], g) @ p).view(n, hq + 2 * hk, d)
    q, k = turn64(rms64(x[:, :hq], a)), turn64(rms64(x[:, hq:hq + hk], b))
    o = _attend(q, k, x[:, hq + hk:], 0).reshape(n, hq * d)
    loss = -(o @ h).log_softmax(-1)[pos, tgt].mean()
    want = torch.autograd.grad(loss, params)

    # the same through the library, products and attention in plain FP32
    r = rn.embed_fwd(tok, emb)
    y = rn.rms_fwd(r, gamma, EPS)
    x = (y @ proj).view(n, hq + 2 * hk, d)
    q, k = rn.qk_rope_fwd(x[:, :hq], x[:, hq:hq + hk], pos, table, wq, wk, EPS)
    leaves = [t.detach().double().requires_grad_() for t in (q, k, x[:, hq + hk:])]
    o = _attend(*leaves, 0).reshape(n, hq * d)
    logits = (o.detach().float() @ head)
    logp, _, lse, _, _ = rn.logprob_fwd(logits, tgt)
    assert abs(float(-logp.mean()) - float(loss.detach())) < 1e-5
    dlogits = rn.logprob_bwd(torch.full_like(logp, -1 / n), logits, tgt, lse)
    dhead = o.detach().float().t() @ dlogits
    dq, dk, dv = torch.autograd.grad(o, leaves, (dlogits @ head.t()).double())
    dx = torch.empty_like(x)                  # one gradient of the packed projection
    dx[:, hq + hk:] = dv.float()
    _, _, dwq, dwk = rn.qk_rope_bwd(dq.float(), dk.float(), x[:, :hq], x[:, hq:hq + hk], pos, table, wq, wk,
                                    EPS, dq=dx[:, :hq], dk=dx[:, hq:hq + hk])
    dx = dx.view(n, -1)
    dr, dgamma = rn.rms_bwd(dx @ proj.t(), r, gamma, EPS)
    demb = rn.embed_bwd(dr, tok, vocab)
    for name, got, w in zip(("emb", "gamma", "proj", "wq", "wk", "head"),
                            (demb, dgamma, y.t() @ dx, dwq, dwk, dhead), want):
        # products of up to 90 FP32 terms a step through five of them: some hundred roundings
        off = float((got.double() - w).norm() / w.norm())
        assert off < 500 * 2.0 ** -24, (name, off)


def test_calls_of_several_threads():
    cases = [Case(50 + i, 4, 2, 64, 64, "bf16") for i in range(4)]
    want, wrong = [], []
    for c in cases:
        g = c.q.contiguous(), c.k.contiguous()
        want.append((g, rn.qk_rope_fwd(c.q, c.k, *c.args()) + rn.qk_rope_bwd(*g, c.q, c.k, *c.args())))
    torch.cuda.synchronize()

    def work(i):
        c, (g, w) = cases[i], want[i]
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(30):
                got = rn.qk_rope_fwd(c.q, c.k, *c.args()) + rn.qk_rope_bwd(*g, c.q, c.k, *c.args())
                st.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, w)):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("d,rot", [(128, 128), (80, 40), (132, 132), (34, 34)])
def test_calls_back_to_back_wait_for_one_another(d, rot):
    """Each call reads what the one ahead of it wrote, without a pause: append, gather, rotate back
    and append elsewhere, over and over, against the same chain with a synchronisation after every
    call."""
    c = Case(600, 8, 8, d, rot, "bf16", outside=False)
    n = c.n
    slots = [torch.from_numpy(c.rng.permutation(700)[:n]).cuda() for _ in range(2)]

    def chain(wait):
        caches = [torch.zeros(100, 7, 8, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        k, v = c.q.contiguous(), c.k.contiguous()
        for i in range(40):
            q = rn.kv_append(k, v, slots[i % 2], *caches, c.pos, c.table, q=v)
            if wait:
                torch.cuda.synchronize()
            rn.kv_gather(*caches, slots[i % 2], k_out=k, v_out=v)
            if wait:
                torch.cuda.synchronize()
            rn.qk_rope_bwd(k, q, None, None, c.pos, c.table, dq=k, dk=v)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return k, v, *caches

    want = chain(True)
    for _ in range(20):
        for a, b in zip(chain(False), want):
            assert torch.equal(_bits(a), _bits(b))
