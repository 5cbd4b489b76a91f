"""Log probabilities, entropies, alternatives and their gradient against the
float64 definitions."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
import token_checks
from oracle import tokens as ot
from row_wise_normalization_gb300 import capi
from token_util import CODE, DT, Framed, f64, rounded

pytestmark = pytest.mark.gpu


def _run(x, t, scale=1.0, top=0, entropy=True):
    logp, ent, lse, ids, tl = rn.logprob_fwd(x, t, scale, top=top, want_entropy=entropy)
    out = {"logp": logp, "entropy": ent, "lse": lse, "top_ids": ids, "top_logp": tl}
    return {k: None if v is None else
            (v.cpu().numpy() if k == "top_ids" else f64(v)) for k, v in out.items()}


def _check(x, t, scale=1.0, top=0, entropy=True, what=""):
    got = _run(x, t, scale, top, entropy)
    want = ot.logprob(f64(x), None if t is None else t.cpu().numpy(), scale, top)
    token_checks.check_logprob(got, want, f64(x), scale, what)
    return got, want


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,top,scale", [
    (1, 1, 1, 1.0), (3, 2, 2, 1.0), (5, 31, 0, 0.5), (4, 32, 32, 1.0), (7, 33, 5, 2.0),
    (6, 1000, 20, 1.0), (9, 1001, 32, 1.25), (2, 16384, 1, 1.0), (3, 16391, 7, 1.0),
    (1, 50001, 20, 0.8125), (2, 128000, 32, 1.0), (300, 257, 3, 1.0), (1, 300007, 5, 1.0),
    (160, 4099, 0, 1.0), (700, 2048, 8, 1.0),
])
def test_forward(dtype, rows, vocab, top, scale):
    rng = np.random.default_rng([rows, vocab])
    x = rounded(rng, (rows, vocab), dtype, 3.0)
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    if rows > 4:
        t[1], t[3] = -100, vocab
    _check(x, t, scale, top)
    _check(x, t.int(), scale, top, entropy=False)


def test_outputs_agree_whatever_else_is_asked():
    rng = np.random.default_rng(3)
    x = rounded(rng, (20, 5003), "bf16", 3.0)
    t = torch.from_numpy(rng.integers(0, 5003, 20)).cuda()
    a = rn.logprob_fwd(x, t, top=9)
    b = rn.logprob_fwd(x, t, want_entropy=False)
    assert b[1] is None and b[3] is None and b[4] is None
    c = rn.logprob_fwd(x, None, top=9)
    assert c[0] is None and torch.equal(c[3], a[3])
    # alternatives hold the target's log probability where they name it
    hit = a[3] == t[:, None]
    assert torch.equal(a[4][hit], a[0][hit.any(1)])


def _pattern(kind, rng, rows, vocab):
    if kind == "ascending":
        return np.tile(np.arange(vocab) * 0.01, (rows, 1))
    if kind == "descending":
        return np.tile(-np.arange(vocab) * 0.01, (rows, 1))
    if kind == "equal":
        return np.full((rows, vocab), 1.25)
    if kind == "two values":
        return rng.integers(0, 2, (rows, vocab)) * 4.0
    if kind == "signed zeros":
        return np.where(rng.random((rows, vocab)) < 0.5, 0.0, -0.0)
    if kind == "far":       # large offsets: only differences count
        return rng.standard_normal((rows, vocab)) * 2 + 3000.0
    if kind == "peaked":
        x = rng.standard_normal((rows, vocab))
        x[np.arange(rows), rng.integers(0, vocab, rows)] += 60
        return x
    if kind == "crowded":   # the largest all in one thread's columns
        x = rng.standard_normal((rows, vocab)) - 30
        x[:, 8:40] = 10 + rng.standard_normal((rows, min(32, vocab - 8)))
        return x
    if kind == "masked":
        x = rng.standard_normal((rows, vocab)) * 3
        x[rng.random((rows, vocab)) < 0.9] = -np.inf
        x[0] = -np.inf                                # nothing left
        x[1] = -np.inf
        x[1, vocab // 3] = 2.0                        # one column left
        x[2, : vocab // 2] = -np.inf
        return x
    if kind == "lowest":    # masks of the type's lowest value
        x = rng.standard_normal((rows, vocab)) * 3
        x[rng.random((rows, vocab)) < 0.5] = np.nan   # replaced by the caller
        x[1] = np.nan
        return x
    raise ValueError(kind)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["ascending", "descending", "equal", "two values",
                                  "signed zeros", "far", "peaked", "crowded", "masked", "lowest"])
@pytest.mark.parametrize("vocab,top", [(40, 32), (5003, 32), (40000, 5)])
def test_patterns(dtype, kind, vocab, top):
    rng = np.random.default_rng([vocab, top])
    a = torch.from_numpy(_pattern(kind, rng, 4, vocab).astype(np.float32))
    x = a.to(DT[dtype])
    if kind == "lowest":
        x = torch.where(torch.isnan(a), torch.finfo(DT[dtype]).min, x)
        x[3] = torch.where(torch.isnan(a[3]), float("-inf"), torch.finfo(DT[dtype]).min)
    x = x.cuda()
    t = torch.tensor([0, vocab // 3, vocab - 1, -1], device="cuda")
    got, want = _check(x, t, 1.0, top, what=f"{kind} ")
    if kind == "masked":
        assert got["entropy"][0] == 0 and got["lse"][0] == -np.inf and got["logp"][0] == -np.inf


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 2.0 ** -13, 64.0, 2.0 ** 40])
def test_extreme_scales_with_masks(dtype, scale):
    rng = np.random.default_rng(21)
    x = rounded(rng, (5, 2100), dtype, 3.0)
    x[:, ::3] = float("-inf")
    x[1] = torch.where(torch.isinf(x[1]), x[1], torch.finfo(DT[dtype]).min)
    x[2, 1] = torch.finfo(DT[dtype]).max
    x[3, 7:900] = torch.finfo(DT[dtype]).min
    t = torch.tensor([1, 2, 4, 8, 3], device="cuda")
    _check(x, t, scale, 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_nan_and_infinity_poison_their_row_alone(dtype):
    rng = np.random.default_rng(8)
    x = rounded(rng, (6, 3001), dtype, 2.0)
    x[1, 7] = float("nan")
    x[3, 2999] = float("inf")
    x[4, 5] = float("nan")
    x[4, 3000] = float("nan")
    t = torch.tensor([5, 5, 2, -1, 0, 1], device="cuda")
    got, want = _check(x, t, 1.0, 4)
    # (a padded target has no value to spoil)
    assert np.isnan(got["lse"][[1, 3, 4]]).all() and got["logp"][3] == 0
    assert got["top_ids"][4, :2].tolist() == [5, 3000]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab,ld,off", [(1000, 1024, 0), (1000, 1001, 1), (1003, 1005, 3),
                                          (17, 18, 5), (9, 40, 7)])
def test_strides_and_phases(dtype, vocab, ld, off):
    rng = np.random.default_rng(ld)
    rows = 5
    x = Framed(rows, vocab, DT[dtype], ld, off, fill=rounded(rng, (rows, vocab), dtype, 2.0))
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    outs = [Framed(1, rows, torch.float32, offset=1) for _ in range(3)]
    ids, tl = Framed(rows, 4, torch.int64), Framed(rows, 4, torch.float32, offset=3)
    capi.check(capi.logprob_fwd(CODE[dtype], 1, x.view.data_ptr(), ld, t.data_ptr(),
                                *[o.view.data_ptr() for o in outs], ids.view.data_ptr(),
                                tl.view.data_ptr(), rows, vocab, 4, 1.0,
                                torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    for o in outs + [ids, tl, x]:
        o.check()
    want = ot.logprob(x.f64(), t.cpu().numpy(), 1.0, 4)
    got = {"logp": outs[0].f64()[0], "entropy": outs[1].f64()[0], "lse": outs[2].f64()[0],
           "top_ids": ids.view.cpu().numpy(), "top_logp": tl.f64()}
    token_checks.check_logprob(got, want, x.f64(), 1.0)


def _bwd_case(rng, rows, vocab, dtype, masked):
    x = rounded(rng, (rows, vocab), dtype, 3.0)
    if masked and vocab > 3:
        x[:, torch.from_numpy(rng.random(vocab) < 0.3).cuda()] = float("-inf")
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    g = torch.from_numpy(rng.standard_normal(rows).astype(np.float32)).cuda()
    h = torch.from_numpy(rng.standard_normal(rows).astype(np.float32)).cuda()
    if rows > 4:
        t[0], t[3] = -100, vocab + 5
        g[1], h[1] = 0.0, 0.0
        h[3] = 0.0
        x[2] = float("-inf")
    return x, t, g, h


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("which", ["logp", "entropy", "both"])
@pytest.mark.parametrize("rows,vocab,scale,masked", [
    (1, 1, 1.0, False), (5, 7, 1.0, True), (6, 1000, 0.8125, False), (9, 8193, 1.25, True),
    (2, 50001, 1.0, True), (40, 256, 1.0, False), (1, 128000, 1.0, False),
])
def test_gradient(dtype, which, rows, vocab, scale, masked):
    rng = np.random.default_rng([rows, vocab])
    x, t, g, h = _bwd_case(rng, rows, vocab, dtype, masked)
    _, ent, lse, _, _ = rn.logprob_fwd(x, t, scale)
    g = g if which != "entropy" else None
    h = h if which != "logp" else None
    d = Framed(rows, vocab, DT[dtype])
    rn.logprob_bwd(g, x, t if g is not None else None, lse, scale, dentropy=h,
                   entropy=ent if h is not None else None, dlogits=d.view)
    d.check()
    want, mag, factor = ot.logprob_backward(
        None if g is None else f64(g), None if h is None else f64(h), f64(x), t.cpu().numpy(),
        f64(lse), f64(ent), scale)
    token_checks.check_logprob_bwd(d.f64(), want, mag, factor, dtype)
    # the gradient in the logits' place: the same bits
    y = x.clone()
    rn.logprob_bwd(g, y, t if g is not None else None, lse, scale, dentropy=h,
                   entropy=ent if h is not None else None, dlogits=y)
    assert torch.equal(y.view(torch.uint8), d.view.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,ldl,ldd,off_l,off_d", [(1000, 1008, 1016, 0, 8),
                                                       (1000, 1001, 1001, 1, 1),
                                                       (1001, 1003, 1002, 0, 1),
                                                       (13, 16, 16, 5, 5)])
def test_gradient_strides_and_phases(dtype, vocab, ldl, ldd, off_l, off_d):
    rng = np.random.default_rng(ldl + ldd)
    rows = 6
    a, t, g, h = _bwd_case(rng, rows, vocab, dtype, False)
    x = Framed(rows, vocab, DT[dtype], ldl, off_l, fill=a)
    _, ent, lse, _, _ = rn.logprob_fwd(a, t)
    d = Framed(rows, vocab, DT[dtype], ldd, off_d)
    capi.check(capi.logprob_bwd(CODE[dtype], 1, g.data_ptr(), h.data_ptr(), x.view.data_ptr(), ldl,
                                t.data_ptr(), lse.data_ptr(), ent.data_ptr(), d.view.data_ptr(),
                                ldd, rows, vocab, 1.0, torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    d.check("dlogits")
    x.check("logits")
    want, mag, factor = ot.logprob_backward(f64(g), f64(h), f64(a), t.cpu().numpy(), f64(lse),
                                            f64(ent), 1.0)
    token_checks.check_logprob_bwd(d.f64(), want, mag, factor, dtype)


def test_gradient_against_differences():
    """Central differences of the float64 definition at the GPU's inputs."""
    rng = np.random.default_rng(4)
    x = rounded(rng, (3, 50), "f32", 2.0)
    t = torch.tensor([4, 49, -1], device="cuda")
    g, h = rounded(rng, (3,), "f32"), rounded(rng, (3,), "f32")
    scale, step = 0.75, 1e-4
    _, ent, lse, _, _ = rn.logprob_fwd(x, t, scale)
    d = f64(rn.logprob_bwd(g, x, t, lse, scale, dentropy=h, entropy=ent))
    a = f64(x)
    for i in range(3):
        for j in range(50):
            f = []
            for s in (step, -step):
                y = a.copy()
                y[i, j] += s
                q = ot.logprob(y, t.cpu().numpy(), scale)
                f.append((f64(g) * q["logp"]).sum() + (f64(h) * q["entropy"]).sum())
            # truncation ~ step^2 / 6 of a third derivative of order 10; FP32 terms of order 10
            assert abs((f[0] - f[1]) / (2 * step) - d[i, j]) < 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradient_where_lse_is_too_large_to_hold(dtype):
    """Rows of the type's lowest value, alone or with -inf, and rows far from
    zero: against the definition from the logits themselves."""
    rng = np.random.default_rng(12)
    low = torch.finfo(DT[dtype]).min
    vocab = 3001
    x = rounded(rng, (6, vocab), dtype, 2.0)
    x[0] = low
    x[1] = low
    x[1, ::2] = float("-inf")
    x[2, 5:] = low                                    # an ordinary masked row
    x[3] = x[3] + 20000
    x[4] = x[4] - 30000
    t = torch.tensor([4, 7, 2, 10, -1, 3000], device="cuda")
    g, h = rounded(rng, (6,), "f32"), rounded(rng, (6,), "f32")
    _, ent, lse, _, _ = rn.logprob_fwd(x, t)
    want, mag, factor = ot.logprob_backward(f64(g), f64(h), f64(x), t.cpu().numpy(), None,
                                            f64(ent), 1.0)
    # log S from a sum of vocab / 256 terms a thread (and 13 more), the ordinary
    # rows' lse from the forward pass
    u = token_checks.U
    more = mag * u * (vocab / 256 + 13 + token_checks.depth(vocab) + 16)
    d = rn.logprob_bwd(g, x, t, lse, dentropy=h, entropy=ent)
    for got in (d, rn.logprob_bwd(g, x, t, lse, dentropy=h, entropy=ent, dlogits=x)):
        err = np.abs(f64(got) - want)
        tol = (8 * u * mag + more + token_checks.UT[dtype] * (np.abs(want) + more)
               + token_checks.TINY[dtype] + 2.0 ** -126 * factor * 2)
        assert np.all(err <= tol), np.argwhere(~(err <= tol))[:3]


def test_rows_far_into_the_logits():
    """Row offsets past 2^31 elements."""
    vocab, ld = 300, 1 << 22
    flat = torch.zeros((599 * ld + vocab,), dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((600, vocab), (ld, 1))
    x.copy_(torch.randn(600, vocab, device="cuda"))
    t = torch.randint(0, vocab, (600,), device="cuda")
    got, _ = _check(x, t, 1.0, 3)
    lse = torch.from_numpy(got["lse"]).float().cuda()
    g = torch.ones(600, device="cuda")
    want = rn.logprob_bwd(g, x.contiguous(), t, lse)
    rn.logprob_bwd(g, x, t, lse, dlogits=x)
    assert torch.equal(x, want)


def test_shapes_and_refusals():
    x = torch.randn(2, 3, 40, device="cuda")
    t = torch.randint(0, 40, (2, 3), device="cuda")
    logp, ent, lse, ids, tl = rn.logprob_fwd(x, t, top=5)
    assert logp.shape == ent.shape == lse.shape == (2, 3) and ids.shape == tl.shape == (2, 3, 5)
    assert rn.logprob_bwd(torch.ones_like(lse), x, t, lse).shape == x.shape
    e = torch.empty(0, 40, device="cuda")
    assert rn.logprob_fwd(e, t[:0, 0], top=2)[3].shape == (0, 2)
    for bad in (lambda: rn.logprob_fwd(x, t, top=33), lambda: rn.logprob_fwd(x, t, 0.0),
                lambda: rn.logprob_fwd(x, t, top=-1),
                lambda: rn.logprob_bwd(None, x, None, lse),
                lambda: rn.logprob_bwd(lse, x, None, lse),
                lambda: rn.logprob_bwd(lse, x, t, lse, dentropy=ent)):
        with pytest.raises(capi.RowNormError):
            bad()
    with pytest.raises(ValueError):
        rn.logprob_fwd(x, t[:, :2])
    with pytest.raises(ValueError):
        rn.logprob_bwd(logp[:1], x, t, lse)
    with pytest.raises(TypeError):
        rn.logprob_bwd(logp.double(), x, t, lse)
    with pytest.raises(TypeError):
        rn.logprob_bwd(logp, x, t, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(3, 40001), (700, 2999)])
def test_logits_in_pinned_host_memory(dtype, rows, vocab):
    """Rows read over the host link: the same bits as from device memory."""
    rng = np.random.default_rng([rows, vocab])
    x = rounded(rng, (rows, vocab), dtype)
    t = torch.from_numpy(rng.integers(0, vocab, rows)).cuda()
    host = x.cpu().pin_memory()
    for kw in ({"want_entropy": False}, {}, {"top": 7}, {"top": 32, "want_entropy": False}):
        a, b = rn.logprob_fwd(x, t, 0.7, **kw), rn.logprob_fwd(host, t, 0.7, **kw)
        torch.cuda.synchronize()
        for p, q in zip(a, b):
            assert (p is None and q is None) or torch.equal(p.cpu(), q.cpu())
