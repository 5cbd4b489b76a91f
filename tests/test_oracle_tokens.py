"""The token operators' oracle: closed forms, differences and planted mistakes."""
import numpy as np
import pytest

import token_checks
from oracle import tokens as ot


def test_uniform_row():
    r = ot.logprob(np.zeros((1, 8)), [3], 1.0, top=3)
    assert np.allclose(r["lse"], np.log(8)) and np.allclose(r["entropy"], np.log(8))
    assert np.allclose(r["logp"], -np.log(8))
    assert r["top_ids"].tolist() == [[0, 1, 2]]


def test_masked_and_empty_rows():
    inf = np.inf
    x = np.array([[0.0, -inf, 0.0], [-inf, -inf, -inf], [1.0, np.nan, 2.0], [inf, 0.0, 1.0]])
    r = ot.logprob(x, [1, 0, 0, 5], 1.0, top=2)
    assert np.allclose(r["lse"][0], np.log(2)) and r["lse"][1] == -inf
    assert np.isnan(r["lse"][2:]).all() and r["entropy"][1] == 0
    assert r["logp"][0] == -inf and r["logp"][1] == -inf and r["logp"][3] == 0
    assert r["top_ids"].tolist() == [[0, 2], [0, 1], [1, 2], [0, 2]]


def test_ties_take_the_lowest_column():
    x = np.array([[0.0, 2.0, -0.0, 2.0, 0.0]])
    assert ot.logprob(x, None, 1.0, top=5)["top_ids"].tolist() == [[1, 3, 0, 2, 4]]


@pytest.mark.parametrize("scale", [1.0, 0.75])
def test_logprob_gradient_against_differences(scale):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 7)) * 2
    x[1, 2] = -np.inf
    t = np.array([4, 0, -100])
    g, h = rng.normal(size=3), rng.normal(size=3)
    r = ot.logprob(x, t, scale)
    d, _, _ = ot.logprob_backward(g, h, x, t, r["lse"], r["entropy"], scale)
    step = 1e-5
    for i in range(3):
        for j in range(7):
            if not np.isfinite(x[i, j]):
                assert d[i, j] == 0
                continue
            f = []
            for s in (step, -step):
                y = x.copy()
                y[i, j] += s
                q = ot.logprob(y, t, scale)
                f.append((g * q["logp"]).sum() + (h * q["entropy"]).sum())
            assert abs((f[0] - f[1]) / (2 * step) - d[i, j]) < 1e-8


def test_embedding_gradient_is_the_transpose():
    rng = np.random.default_rng(1)
    tok = np.array([3, 0, 3, -1, 9, 2])
    w, dy = rng.normal(size=(5, 4)), rng.normal(size=(6, 4))
    g, _, m = ot.embed_backward(dy, tok, 5, 1.5)
    # <E(w), dy> = <w, E^T(dy)>
    assert np.isclose((ot.embed(tok, w, 1.5) * dy).sum(), (w * g).sum())
    assert m.tolist() == [1, 0, 1, 2, 0]


def test_checks_catch_planted_mistakes():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(2, 50))
    t = np.array([7, 11])
    want = ot.logprob(x, t, 1.0, top=4)
    token_checks.check_logprob(dict(want), want, x, 1.0)
    for key in ("lse", "entropy", "logp", "top_logp"):
        bad = {k: np.array(v) for k, v in want.items()}
        bad[key].reshape(-1)[0] *= 1 + 1e-4
        with pytest.raises(AssertionError):
            token_checks.check_logprob(bad, want, x, 1.0)
    bad = {k: np.array(v) for k, v in want.items()}
    bad["top_ids"][0, :2] = bad["top_ids"][0, 1::-1]
    with pytest.raises(AssertionError):
        token_checks.check_logprob(bad, want, x, 1.0)
    dy = rng.normal(size=(6, 4))
    g, a, m = ot.embed_backward(dy, [1, 1, 0, 2, 1, 1], 3, 1.0)
    token_checks.check_embed_bwd(g, g, a, m, "f32")
    with pytest.raises(AssertionError):
        token_checks.check_embed_bwd(g + 1e-5 * a, g, a, m, "f32")
