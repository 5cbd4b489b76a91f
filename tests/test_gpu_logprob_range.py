"""Log probabilities at the ends of their ranges: the largest and smallest scales,
logits as far apart as the type allows, rows far from zero."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
import token_checks
from oracle import tokens as ot
from token_util import DT, f64, rounded

pytestmark = pytest.mark.gpu
F32_MAX = float(np.finfo(np.float32).max)


def _check(x, t, scale, top):
    logp, ent, lse, ids, tl = rn.logprob_fwd(x, t, scale, top=top)
    plain = rn.logprob_fwd(x, t, scale, want_entropy=False)
    want = ot.logprob(f64(x), t.cpu().numpy(), scale, top)
    token_checks.check_logprob({"logp": f64(logp), "entropy": f64(ent), "lse": f64(lse),
                                "top_ids": ids.cpu().numpy(), "top_logp": f64(tl)}, want, f64(x),
                               scale)
    token_checks.check_logprob({"logp": f64(plain[0]), "lse": f64(plain[2])}, want, f64(x), scale)
    return ent, lse


def _check_gradient(x, t, scale, lse, ent, dtype, std, off_by):
    """Against the definition from the logits themselves; off_by: what lse (or the
    kernel's own log S) may be off by, which makes a probability off by as much."""
    rng = np.random.default_rng(77)
    g, h = (rounded(rng, (x.shape[0],), "f32", std) for _ in range(2))
    d = rn.logprob_bwd(g, x, t, lse, scale, dentropy=h, entropy=ent)
    want, mag, factor = ot.logprob_backward(f64(g), f64(h), f64(x), t.cpu().numpy(), None, f64(ent),
                                            scale)
    u = token_checks.U
    more = 8 * u * mag + mag * np.reshape(off_by, (-1, 1))
    # Below 2^-126 each rounding is off by up to s = 2^-150, whatever the value. With gs = g scale,
    # b = -h scale (s each) and a = b H - gs (s |H| + s + s), the element e^z (a + b z) + gs is
    # off by p (s |z| + s (|H| + 2) + s) + s + s, and p |z| < 1, p <= 1: s (|H| + 6).
    more = more + 2.0 ** -150 * (np.abs(f64(ent)[:, None]) + 6)
    tol = (more + token_checks.UT[dtype] * (np.abs(want) + more) + token_checks.TINY[dtype]
           + 2.0 ** -126 * factor * 2)
    err = np.abs(f64(d) - want)
    assert np.all(err <= tol), (np.argwhere(~(err <= tol))[:3], err.max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** 127, float(np.float32(3e38)), F32_MAX])
@pytest.mark.parametrize("vocab", [3, 700, 20011])
def test_the_largest_scales(dtype, scale, vocab):
    """Differences of a logit are beyond the exponential's range: p is 0, or 1 over the
    columns that share the maximum."""
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(-rng.integers(1, 90, (6, vocab)).astype(np.float32))
    x[0, 0] = 0.0
    x[1, 2] = 0.0
    x[1, 0] = float("-inf")
    x[2, ::2] = 0.0                       # entropy: log of their number
    x[3] = 1.0                            # lse = scale + log vocab
    x[4, 1] = 4.0                         # lse: beyond FP32
    x[5] = torch.finfo(DT[dtype]).min     # a mask's lowest value, and one column
    x[5, 1] = 0.0
    x = x.to(DT[dtype]).cuda()
    t = torch.tensor([0, 0, 1, 2, 1, 1], device="cuda")
    ent, lse = _check(x, t, scale, 3)
    if dtype != "f16":                    # (whose range ends at 65504)
        u = token_checks.U
        off = u * (vocab / 256 + 13 + token_checks.depth(vocab) + 16)
        _check_gradient(x, t, scale, lse, ent, dtype, 2.0 ** -20, np.full(6, off))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -70, 1.0, 2.0 ** 40, float(np.float32(3e38))])
@pytest.mark.parametrize("vocab", [6, 2100])
def test_nan_rows_with_masks(dtype, scale, vocab):
    """A NaN spoils every value of its row, those of masked columns too."""
    x = torch.full((4, vocab), float("-inf"))
    x[:, 2] = 0.5
    x[1, 4] = float("nan")
    x[2, 2] = float("nan")                # nothing but NaN and -inf
    x[3, 1] = -1.5
    x = x.to(DT[dtype]).cuda()
    t = torch.tensor([0, 0, 0, -1], device="cuda")
    _check(x, t, scale, 4)
    _check(x, torch.full_like(t, 2), scale, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -130, 2.0 ** -127, 2.0 ** -126, 2.0 ** -120,
                                   2.0 ** -60])
@pytest.mark.parametrize("vocab", [5, 2100])
def test_logits_as_far_apart_as_the_type_allows(dtype, scale, vocab):
    """Differences of logits beyond FP32's range, whose products with the scale are ordinary."""
    rng = np.random.default_rng(vocab)
    top = torch.finfo(DT[dtype]).max
    a = rng.uniform(-1.0, 1.0, (4, vocab))
    a[1] = np.where(rng.random(vocab) < 0.5, 1.0, -1.0)
    a[2, ::2] = -np.inf
    a[0, :2], a[1, :2], a[2, 1] = (1.0, -1.0), (-1.0, 1.0), 1.0
    x = torch.from_numpy(a * top).to(DT[dtype]).cuda()
    t = torch.tensor([1, 0, 3, 2], device="cuda")
    ent, lse = _check(x, t, scale, 4)
    u = token_checks.U
    off = 4 * u * (np.abs(f64(lse)) + np.log(vocab)) + u * (token_checks.depth(vocab) + 32)
    if dtype != "f16":                    # (all of whose logits are alike at such scales)
        _check_gradient(x, t, scale, lse, ent, dtype, 1.0, off)


@pytest.mark.parametrize("offset", [300.0, 1000.0, 3900.0, -3000.0])
@pytest.mark.parametrize("scale", [0.7, 0.8125, 1.0, 1.0333])
@pytest.mark.parametrize("vocab", [64, 5003])
def test_lse_far_from_zero(offset, scale, vocab):
    """lse is what log S adds to the largest product, rounded once: half a step of its own, and
    S's and the logarithm's errors. A gradient from it is off by as much."""
    rng = np.random.default_rng([vocab, int(abs(offset))])
    scale = float(np.float32(scale))
    x = (rounded(rng, (40, vocab), "f32", 2.0) + offset).contiguous()
    t = torch.from_numpy(rng.integers(0, vocab, 40)).cuda()
    ent, lse = _check(x, t, scale, 2)
    a = scale * f64(x)
    m = a.max(1)
    z = np.abs(a - m[:, None])
    p = np.exp(-z) / np.exp(-z).sum(1, keepdims=True)
    want = m + np.log(np.exp(-z).sum(1))
    u = token_checks.U
    # S along its chain and its elements' exponents (token_checks), the logarithm, and the two
    # sums of small numbers that precede the rounding
    off = (u * np.abs(want) + u * (token_checks.depth(vocab) + 4 + 4 * (p * z).sum(1))
           + 6 * u * np.log(vocab) + 4 * u)
    err = np.abs(f64(lse) - want)
    assert np.all(err <= off), (err.max(), off.min())
    _check_gradient(x, t, scale, lse, ent, "f32", 1.0, off)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [1.0, 1.25, 64.0, 2.0 ** 30])
@pytest.mark.parametrize("vocab,pad", [(7, 0), (700, 0), (5003, 5)])
def test_rows_of_masks_alone(dtype, scale, vocab, pad):
    """Nothing but a mask's lowest value: its columns share the row, although lse may be beyond
    FP32. Nothing but -inf: no gradient."""
    low = torch.finfo(DT[dtype]).min
    x = torch.full((4, vocab + pad), low, dtype=DT[dtype], device="cuda")[:, :vocab]
    x[1, ::2] = float("-inf")
    x[2] = float("-inf")
    x[3, 3:] = 0.25
    t = torch.tensor([1, 3, 0, 2], device="cuda")
    ent, lse = _check(x, t, scale, 3)
    assert ent[2] == 0 and lse[2] == -np.inf
    u = token_checks.U
    off = u * (vocab / 256 + 13 + token_checks.depth(vocab) + 16 + np.abs(0.25 * scale)
               * (0.25 * scale < 4096))
    if dtype != "f16" or scale < 100:
        _check_gradient(x, t, scale, lse, ent, dtype, 2.0 ** -8, np.full(4, off))
        d = rn.logprob_bwd(torch.ones(4, device="cuda"), x, t, lse, scale, dlogits=x.clone())
        assert not bool(d[2].any()) and bool(d[0].any())
