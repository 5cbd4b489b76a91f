"""Embedding rows and their gradient against the float64 definitions."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
import token_checks
from oracle import tokens as ot
from row_wise_normalization_gb300 import capi
from token_util import CODE, DT, Framed, f64, rounded

pytestmark = pytest.mark.gpu
IT = {"i32": torch.int32, "i64": torch.int64}


def _bits_equal(got, want):
    return torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,vocab,d,itype,scale", [
    (1, 1, 1, "i64", 1.0), (1, 50, 4096, "i32", 2.5), (7, 50, 33, "i32", -1.5),
    (300, 1000, 128, "i64", 27.75), (33, 100, 771, "i64", 1.0), (65, 64, 2050, "i32", 0.125),
    (5, 9, 16384, "i64", 1.0), (2049, 300, 12, "i32", 1.0),
])
def test_rows(dtype, n, vocab, d, itype, scale):
    rng = np.random.default_rng([n, d])
    table = rounded(rng, (vocab, d), dtype)
    tok = torch.from_numpy(rng.integers(0, vocab, n)).to(IT[itype]).cuda()
    if n > 4:
        tok[1], tok[3] = -1, vocab
    out = Framed(n, d, DT[dtype])
    rn.embed_fwd(tok, table, scale, out=out.view)
    out.check()
    there = (tok >= 0) & (tok < vocab)
    # one FP32 product and one rounding: the same bits
    want = (table[tok.long().clamp(0, vocab - 1)].float() * scale).to(DT[dtype])
    want[~there] = 0
    assert _bits_equal(out.view, want)
    ref = ot.embed(tok.cpu().numpy(), f64(table), scale)
    assert np.all(np.abs(out.f64() - ref) <= (token_checks.UT[dtype] + 2 * token_checks.U)
                  * np.abs(ref) + token_checks.TINY[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,ldt,ldo,off_t,off_o", [
    (64, 64, 64, 0, 0), (64, 72, 80, 8, 16), (64, 66, 64, 2, 0), (63, 64, 65, 1, 3),
    (96, 100, 96, 4, 4),
])
def test_strides_and_phases(dtype, d, ldt, ldo, off_t, off_o):
    rng = np.random.default_rng(d + ldt)
    vocab, n = 37, 50
    table = Framed(vocab, d, DT[dtype], ldt, off_t, fill=rounded(rng, (vocab, d), dtype))
    out = Framed(n, d, DT[dtype], ldo, off_o)
    tok = torch.from_numpy(rng.integers(-3, vocab + 3, n)).cuda()
    # straight through the C ABI: phases that a torch view need not have
    st = capi.embed_fwd(CODE[dtype], 1, tok.data_ptr(), table.view.data_ptr(), ldt,
                        out.view.data_ptr(), ldo, n, vocab, d, 0.5,
                        torch.cuda.current_stream().cuda_stream)
    capi.check(st)
    torch.cuda.synchronize()
    out.check("out")
    table.check("table")
    there = (tok >= 0) & (tok < vocab)
    want = (table.view[tok.clamp(0, vocab - 1)].float() * 0.5).to(DT[dtype])
    want[~there] = 0
    assert _bits_equal(out.view, want)


def test_rows_far_into_a_table():
    """Row offsets past 2^32 bytes (and, with the stride, past 2^31 elements)."""
    ld, vocab, d = 1 << 22, 600, 64
    flat = torch.empty(((vocab - 1) * ld + d,), dtype=torch.bfloat16, device="cuda")
    table = flat.as_strided((vocab, d), (ld, 1))
    table.copy_(torch.randn(vocab, d, device="cuda"))
    tok = torch.tensor([599, 0, 512, 511, 600], device="cuda")
    out = rn.embed_fwd(tok, table, 2.0)
    want = table[tok.clamp(max=599)] * 2
    want[4] = 0
    assert torch.equal(out, want)
    dout = torch.randn(5, d, device="cuda").bfloat16()
    flat.zero_()
    rn.embed_bwd(dout, tok, vocab, 1.0, dtable=table, accumulate=True)
    assert torch.equal(table[599], dout[0]) and torch.equal(table[511], dout[3])
    assert not bool(table[510].any())


def _tokens(rng, kind, n, vocab):
    if kind == "uniform":
        return rng.integers(0, vocab, n)
    if kind == "one":
        return np.full(n, vocab // 2)
    if kind == "outside":
        return np.where(rng.random(n) < 0.5, -1, vocab + 7)
    if kind == "heavy":     # half of the batch one id, the ends of the vocabulary in it
        t = rng.integers(-1, vocab + 1, n)
        t[rng.random(n) < 0.5] = vocab - 1
        t[rng.random(n) < 0.2] = 0
        return t
    return np.sort(rng.integers(0, vocab, n))[::-1].copy()


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                        ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("n,vocab,d,kind", [
    (1, 1, 1, "uniform"), (1, 700, 64, "uniform"), (31, 5, 8, "heavy"), (32, 40, 33, "one"),
    (33, 40, 257, "one"), (129, 100, 1030, "heavy"), (1000, 2000, 771, "uniform"),
    (4097, 600, 48, "heavy"), (5000, 3, 20, "heavy"), (700, 70000, 16, "descending"),
    (9000, 300, 4, "one"), (300, 90, 64, "outside"), (13000, 270000, 2, "uniform"),
    (1024, 37, 9, "heavy"), (1025, 37, 9, "heavy"), (1024, 2000, 300, "one"),
    (64, 9, 8192, "heavy"),
    (65, 9, 8200, "heavy"), (257, 5000, 520, "descending"), (992, 1500, 100, "uniform"),
])
def test_gradient(dtype, grad, n, vocab, d, kind):
    rng = np.random.default_rng([n, vocab, d])
    tok = _tokens(rng, kind, n, vocab)
    dout = rounded(rng, (n, d), dtype)
    g = Framed(vocab, d, DT[grad])
    t = torch.from_numpy(tok).to(torch.int32 if n % 2 else torch.int64).cuda()
    rn.embed_bwd(dout, t, vocab, 1.5, dtable=g.view)
    g.check()
    want, absum, terms = ot.embed_backward(f64(dout), tok, vocab, 1.5)
    token_checks.check_embed_bwd(g.f64(), want, absum, terms, grad)
    assert not np.any(g.f64()[terms == 0])
    # the same bits again, from a workspace that holds other values
    ws = torch.full((capi.embed_bwd_workspace_size(n, vocab, d),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    assert _bits_equal(rn.embed_bwd(dout, t, vocab, 1.5, dtype=DT[grad], workspace=ws), g.view)


@pytest.mark.parametrize("n,vocab,d,kind", [
    (2048, 400, 8, "heavy"), (2049, 400, 8, "heavy"), (30000, 131072, 3, "uniform"),
    (33000, 511, 2, "uniform"), (33000, 512, 2, "heavy"), (100000, 50001, 4, "heavy"),
    (163840, 1000, 2, "uniform"), (163841, 1000, 2, "uniform"), (200000, 300000, 1, "heavy"),
    (300001, 200, 2, "one"), (170000, 1 << 20, 8, "descending"),
])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_many_ids(n, vocab, d, kind, accumulate):
    """Every size of the sort: one CTA, clusters, global memory; one digit to three."""
    rng = np.random.default_rng([n, vocab])
    tok = _tokens(rng, kind, n, vocab)
    # small whole numbers: sums are exact, so the order of terms does not matter
    vals = rng.integers(-8, 9, (n, d)).astype(np.float32)
    dout = torch.from_numpy(vals).cuda()
    old = torch.full((vocab, d), 3.0, device="cuda")
    g = Framed(vocab, d, torch.float32, fill=old)
    rn.embed_bwd(dout, torch.from_numpy(tok).cuda(), vocab, dtable=g.view, accumulate=accumulate)
    g.check()
    want = np.zeros((vocab, d))
    ok = (tok >= 0) & (tok < vocab)
    np.add.at(want, tok[ok], vals[ok])
    assert np.array_equal(g.f64(), want + (3.0 if accumulate else 0.0))


@pytest.mark.parametrize("dtype,grad", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("n,vocab,d", [(65, 200, 24), (700, 90, 129)])
def test_gradient_accumulates(dtype, grad, n, vocab, d):
    rng = np.random.default_rng([n, d])
    tok = _tokens(rng, "heavy", n, vocab)
    dout = rounded(rng, (n, d), dtype)
    old = rounded(rng, (vocab, d), grad)
    g = Framed(vocab, d, DT[grad], ld=d + 3, offset=1, fill=old)
    rn.embed_bwd(dout, torch.from_numpy(tok).cuda(), vocab, -0.5, dtable=g.view, accumulate=True)
    g.check()
    want, absum, terms = ot.embed_backward(f64(dout), tok, vocab, -0.5)
    token_checks.check_embed_bwd(g.f64(), want, absum, terms, grad, old=f64(old))
    absent = terms == 0
    assert np.array_equal(g.f64()[absent], f64(old)[absent])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,ldd,ldg,off_d,off_g", [(64, 72, 80, 0, 0), (64, 64, 66, 2, 0),
                                                   (61, 64, 61, 1, 3)])
def test_gradient_strides_and_phases(dtype, d, ldd, ldg, off_d, off_g):
    rng = np.random.default_rng(ldd + ldg)
    n, vocab = 200, 50
    tok = _tokens(rng, "heavy", n, vocab)
    t = torch.from_numpy(tok).cuda()
    dout = Framed(n, d, DT[dtype], ldd, off_d, fill=rounded(rng, (n, d), dtype))
    g = Framed(vocab, d, DT[dtype], ldg, off_g)
    ws = torch.empty(capi.embed_bwd_workspace_size(n, vocab, d), dtype=torch.uint8, device="cuda")
    capi.check(capi.embed_bwd(CODE[dtype], CODE[dtype], 1, dout.view.data_ptr(), ldd, t.data_ptr(),
                              g.view.data_ptr(), ldg, n, vocab, d, 1.0, 0, ws.data_ptr(),
                              ws.numel(), torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    g.check("dtable")
    dout.check("dout")
    want, absum, terms = ot.embed_backward(dout.f64(), tok, vocab, 1.0)
    token_checks.check_embed_bwd(g.f64(), want, absum, terms, dtype)


def test_gradient_of_nothing():
    g = Framed(20, 8, torch.float32, ld=11, offset=1)
    dout = torch.empty(0, 8, device="cuda")
    tok = torch.empty(0, dtype=torch.int64, device="cuda")
    rn.embed_bwd(dout, tok, 20, dtable=g.view, accumulate=True)
    assert torch.equal(g.bits, g.before)
    rn.embed_bwd(dout, tok, 20, dtable=g.view)
    g.check()
    assert not bool(g.view.any())
    assert rn.embed_fwd(tok, torch.ones(3, 8, device="cuda")).shape == (0, 8)


def test_gradient_against_differences():
    """<E(w + s v) - E(w - s v), dout> / 2s against <gradient, v>, the forward
    rows taken from the GPU."""
    rng = np.random.default_rng(5)
    vocab, d, n = 40, 24, 90
    tok = torch.from_numpy(rng.integers(-1, vocab + 1, n)).cuda()
    w, v = rounded(rng, (vocab, d), "f32"), rounded(rng, (vocab, d), "f32")
    dout = rounded(rng, (n, d), "f32")
    s = 0.5   # the map is linear: any step will do, a power of two adds no rounding
    up, dn = rn.embed_fwd(tok, w + s * v, 1.25), rn.embed_fwd(tok, w - s * v, 1.25)
    diff = float(((up.double() - dn.double()) * dout.double()).sum()) / (2 * s)
    g = rn.embed_bwd(dout, tok, vocab, 1.25)
    got = float((g.double() * v.double()).sum())
    # up, dn, g: a few roundings each of values of order |w| + |v|, per product
    bound = 16 * token_checks.U * 1.25 * float(
        ((w.abs() + v.abs()).double().max() * dout.double().abs()).sum()) * 4
    assert abs(diff - got) <= bound


def test_non_finite_rows_stay_in_their_rows():
    dout = torch.ones(70, 16, device="cuda")
    tok = torch.arange(70, device="cuda") % 7
    dout[3, 5] = float("nan")
    dout[64, 1] = float("inf")
    g = rn.embed_bwd(dout, tok, 9)
    bad = torch.zeros(9, 16, dtype=torch.bool, device="cuda")
    bad[3, 5] = True
    assert torch.equal(torch.isnan(g), bad)
    assert torch.isinf(g[1, 1]) and bool((g[7:] == 0).all())
    # a row that no id may read
    dout[5] = float("nan")
    t2 = torch.where(torch.arange(70, device="cuda") % 5 == 0, -1, tok)
    dout[3, 5] = 1.0
    assert not bool(torch.isnan(rn.embed_bwd(dout, t2, 9)).any())


def test_two_dimensional_ids_and_refusals():
    table = torch.randn(11, 6, device="cuda")
    tok = torch.randint(0, 11, (3, 5), device="cuda")
    y = rn.embed_fwd(tok, table)
    assert y.shape == (3, 5, 6) and torch.equal(y, table[tok])
    g = rn.embed_bwd(y, tok, 11)
    assert g.shape == (11, 6)
    with pytest.raises(ValueError):
        rn.embed_bwd(y, tok, 11, accumulate=True)
    with pytest.raises(ValueError):
        rn.embed_bwd(y[:2], tok, 11)
    with pytest.raises(TypeError):
        rn.embed_bwd(y, tok, 11, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rn.embed_bwd(y, tok, 11, dtable=torch.empty(10, 6, device="cuda"))
    with pytest.raises(capi.RowNormError):
        rn.embed_bwd(y, tok, 11, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(capi.RowNormError):
        rn.embed_fwd(tok, table, float("inf"))
    with pytest.raises(ValueError):
        rn.embed_fwd(tok, table, out=torch.empty(14, 6, device="cuda"))
    host_ws = torch.empty(capi.embed_bwd_workspace_size(15, 11, 6), dtype=torch.uint8,
                          pin_memory=True)
    st = capi.embed_bwd(0, 0, 1, y.data_ptr(), 6, tok.data_ptr(), g.data_ptr(), 6, 15, 11, 6, 1.0,
                        0, host_ws.data_ptr(), host_ws.numel(), 0)
    assert st == capi.RN_ERR_HOSTMEM


def test_pinned_host_table():
    """Rows read over the host link, as the library's other calls do."""
    table = torch.randn(100, 64).pin_memory()
    tok = torch.randint(0, 100, (37,), device="cuda")
    y = rn.embed_fwd(tok, table, 3.0)
    assert y.is_cuda and torch.equal(y.cpu(), table[tok.cpu()] * 3)


@pytest.mark.parametrize("n,vocab", [(50, 21_000_000), (1500, 5_000_000), (1500, 17_000_001)])
def test_zeros_of_a_vast_vocabulary(n, vocab):
    # more ids than the marks of all clearing CTAs hold at a time
    rng = np.random.default_rng(n + vocab)
    tok = torch.from_numpy(rng.permutation(vocab)[:n]).cuda()
    tok[0], tok[1] = 0, vocab - 1
    tok = torch.unique(tok)
    dout = rounded(rng, (tok.numel(), 1), "bf16")
    want = torch.zeros(vocab, 1, dtype=torch.bfloat16, device="cuda")
    want[tok] = dout
    got = torch.full_like(want, float("nan"))
    assert _bits_equal(rn.embed_bwd(dout, tok, vocab, dtable=got), want)


@pytest.mark.parametrize("gtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [40, 1100])
@pytest.mark.parametrize("d,ldg,off", [
    (256, 256, 0), (256, 264, 8), (1031, 1031, 3), (2048, 2050, 1), (5000, 5000, 0), (2052, 2056, 4),
])
def test_zeros_of_long_rows(gtype, n, d, ldg, off):
    # one sum an id: its bits; all else zeros, and what lies between the rows as it was
    rng = np.random.default_rng([n, d])
    vocab = 1500
    tok = torch.from_numpy(rng.permutation(vocab)[:n]).cuda()
    dout = rounded(rng, (n, d), gtype)
    grad = Framed(vocab, d, DT[gtype], ldg, off)
    rn.embed_bwd(dout, tok, vocab, dtable=grad.view)
    grad.check()
    want = torch.zeros(vocab, d, dtype=DT[gtype], device="cuda")
    want[tok] = dout
    assert _bits_equal(grad.view, want)


@pytest.mark.parametrize("n", [40, 3000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_in_pinned_host_memory(n, accumulate):
    """Rows read and written over the host link, long ones too."""
    rng = np.random.default_rng(n)
    vocab, d = 300, 640
    tok = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
    dout = torch.from_numpy(rng.integers(-3, 4, (n, d)).astype(np.float32))
    grad = torch.from_numpy(rng.integers(-3, 4, (vocab, d)).astype(np.float32)).pin_memory()
    want = grad.clone() if accumulate else torch.zeros(vocab, d)
    want.index_add_(0, tok.cpu(), dout)
    got = rn.embed_bwd(dout.pin_memory(), tok, vocab, dtable=grad, accumulate=accumulate)
    torch.cuda.synchronize()
    assert got is grad and torch.equal(grad, want)
