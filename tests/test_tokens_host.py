"""The token operators on the host: argument checks before any CUDA call, and
the binding's own refusals (no GPU needed)."""
import math

import pytest
import torch

import row_wise_normalization_gb300 as rn
from row_wise_normalization_gb300 import capi

A = 1 << 32          # fake, aligned addresses; never dereferenced
STEP = 1 << 32


def _ef(**kw):
    a = dict(dtype=0, itype=1, tokens=A, table=A + STEP, ldt=8, out=A + 2 * STEP, ldo=8, n=4,
             vocab=10, d=8, scale=1.0)
    a.update(kw)
    return capi.embed_fwd(**a)


def _eb(**kw):
    a = dict(dtype=1, gtype=0, itype=1, dout=A, lddo=8, tokens=A + STEP, dtable=A + 2 * STEP, ldg=8,
             n=4, vocab=10, d=8, scale=1.0, accumulate=0, workspace=A + 3 * STEP,
             workspace_bytes=1 << 20)
    a.update(kw)
    return capi.embed_bwd(**a)


def _lf(**kw):
    a = dict(dtype=0, itype=1, logits=A, ldl=100, targets=A + STEP, logp=A + 2 * STEP,
             entropy=A + 3 * STEP, lse=A + 4 * STEP, top_ids=A + 5 * STEP, top_logp=A + 6 * STEP,
             rows=4, vocab=100, top=3, scale=1.0)
    a.update(kw)
    return capi.logprob_fwd(**a)


def _lb(**kw):
    a = dict(dtype=0, itype=1, dlogp=A, dentropy=A + STEP, logits=A + 2 * STEP, ldl=100,
             targets=A + 3 * STEP, lse=A + 4 * STEP, entropy=A + 5 * STEP, dlogits=A + 6 * STEP,
             ldd=100, rows=4, vocab=100, scale=1.0)
    a.update(kw)
    return capi.logprob_bwd(**a)


SIZE, NULL, ALIGN = capi.RN_ERR_SIZE, capi.RN_ERR_NULL, capi.RN_ERR_ALIGN
ALIAS, DTYPE, SCALE = capi.RN_ERR_ALIAS, capi.RN_ERR_DTYPE, capi.RN_ERR_SCALE


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(itype=2), DTYPE), (dict(n=-1), SIZE), (dict(vocab=0), SIZE),
    (dict(vocab=(1 << 30) + 1), SIZE), (dict(d=0), SIZE), (dict(ldt=7), SIZE), (dict(ldo=7), SIZE),
    (dict(n=1 << 60), SIZE), (dict(n=1 << 41), SIZE), (dict(scale=math.nan), SCALE),
    (dict(scale=math.inf), SCALE), (dict(tokens=0), NULL), (dict(table=0), NULL),
    (dict(out=0), NULL), (dict(tokens=A + 4), ALIGN), (dict(table=A + STEP + 2), ALIGN),
    (dict(out=A + 2 * STEP + 1), ALIGN), (dict(out=A + STEP + 32), ALIAS), (dict(out=A), ALIAS),
    (dict(n=0, tokens=0, table=0, out=0), capi.RN_OK),
])
def test_embed_fwd_checks(kw, want):
    if kw.get("n") == 1 << 41:
        kw = dict(kw, tokens=1 << 60, out=1 << 61)
    assert _ef(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(gtype=2), DTYPE), (dict(dtype=0, gtype=1), DTYPE),
    (dict(itype=-1), DTYPE), (dict(n=-1), SIZE), (dict(n=1 << 31), SIZE), (dict(vocab=0), SIZE),
    (dict(d=0), SIZE), (dict(lddo=7), SIZE), (dict(ldg=7), SIZE), (dict(scale=math.inf), SCALE),
    (dict(n=1 << 30, d=1 << 20, lddo=1 << 20, ldg=1 << 20), SIZE),
    (dict(dout=0), NULL), (dict(tokens=0), NULL), (dict(dtable=0), NULL),
    (dict(workspace=0), NULL), (dict(workspace=A + 3 * STEP + 8), ALIGN),
    (dict(dout=A + 1), ALIGN), (dict(dtable=A + 2 * STEP + 2), ALIGN),
    (dict(workspace_bytes=64), SIZE), (dict(dtable=A + 16), ALIAS),
    (dict(workspace=A + 2 * STEP), ALIAS), (dict(workspace=A + STEP), ALIAS),
    (dict(n=0, accumulate=1, dout=0, tokens=0, dtable=0, workspace=0), capi.RN_OK),
    (dict(n=0, dtable=0), NULL),
])
def test_embed_bwd_checks(kw, want):
    assert _eb(**kw) == want


def test_embed_bwd_workspace():
    assert capi.embed_bwd_workspace_size(0, 100, 8) == 0
    small = capi.embed_bwd_workspace_size(100, 1000, 64)
    assert 0 < small <= capi.embed_bwd_workspace_size(101, 1000, 64)
    for bad in ((-1, 10, 8), (4, 0, 8), (4, 10, 0), (1 << 31, 10, 8)):
        with pytest.raises(capi.RowNormError):
            capi.embed_bwd_workspace_size(*bad)


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), DTYPE), (dict(itype=5), DTYPE), (dict(rows=-1), SIZE), (dict(vocab=0), SIZE),
    (dict(ldl=99), SIZE), (dict(top=-1), SIZE), (dict(top=33), SIZE),
    (dict(vocab=2, top=3), SIZE), (dict(rows=1 << 60), SIZE),
    (dict(vocab=(1 << 30) + 1, ldl=1 << 31), SIZE),
    (dict(scale=0.0), SCALE), (dict(scale=-1.0), SCALE), (dict(scale=math.nan), SCALE),
    (dict(logits=0), NULL), (dict(targets=0), NULL), (dict(top_ids=0, top_logp=0), NULL),
    (dict(logp=0, entropy=0, lse=0, top=0), NULL),
    (dict(logits=A + 2), ALIGN), (dict(targets=A + STEP + 4), ALIGN),
    (dict(lse=A + 4 * STEP + 2), ALIGN), (dict(top_ids=A + 5 * STEP + 4), ALIGN),
    (dict(lse=A + 16), ALIAS), (dict(lse=A + 2 * STEP + 4), ALIAS),
    (dict(top_logp=A + 5 * STEP + 8), ALIAS), (dict(logp=A + STEP), ALIAS),
    (dict(rows=0, logits=0), capi.RN_OK),
])
def test_logprob_fwd_checks(kw, want):
    assert _lf(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=-1), DTYPE), (dict(itype=2), DTYPE), (dict(rows=-1), SIZE), (dict(vocab=0), SIZE),
    (dict(ldl=99), SIZE), (dict(ldd=99), SIZE), (dict(scale=0.0), SCALE),
    (dict(dlogp=0, dentropy=0), NULL), (dict(targets=0), NULL), (dict(entropy=0), NULL),
    (dict(lse=0), NULL), (dict(logits=0), NULL), (dict(dlogits=0), NULL),
    (dict(dlogp=A + 2), ALIGN), (dict(dlogits=A + 6 * STEP + 2), ALIGN),
    (dict(dlogits=A + 2 * STEP + 4), ALIAS), (dict(dlogits=A + 2 * STEP, ldd=101), ALIAS),
    (dict(dlogits=A + 4 * STEP), ALIAS), (dict(rows=0, logits=0), capi.RN_OK),
])
def test_logprob_bwd_checks(kw, want):
    assert _lb(**kw) == want


def test_scale_status_has_a_text():
    assert "scale" in capi.status_str(SCALE)


def test_binding_refusals():
    f, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        rn.embed_fwd(i, f.double())
    with pytest.raises(TypeError):
        rn.embed_fwd(i.to(torch.int16), f)
    with pytest.raises(TypeError):
        rn.embed_fwd([0, 1], f)
    with pytest.raises(ValueError):
        rn.embed_fwd(i, f.reshape(-1))
    with pytest.raises(TypeError):
        rn.logprob_fwd(f.to(torch.int32), i)
    with pytest.raises(TypeError):
        rn.logprob_bwd(f[:, 0], f.double(), i, f[:, 0])
    if not torch.cuda.is_available():
        # pageable host memory without a GPU that reads it
        with pytest.raises(ValueError):
            rn.embed_fwd(i, f)
        with pytest.raises(ValueError):
            rn.logprob_fwd(f, i)
