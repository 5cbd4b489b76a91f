"""Seeded random calls of the token operators against the float64 definitions:
sizes, types, strides, phases, masks and id distributions drawn together."""
import math
import threading

import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
import token_checks
from oracle import tokens as ot
from row_wise_normalization_gb300 import capi
from token_util import CODE, DT, Framed, f64, rounded

pytestmark = pytest.mark.gpu


def _spread(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _stride(rng, d):
    return d + int(rng.choice([0, 0, 1, 3, 8, 16]))


def _ids(rng, n, vocab):
    kind = rng.integers(0, 4)
    t = rng.integers(-2, vocab + 2, n)
    if kind == 1:
        t[rng.random(n) < 0.7] = rng.integers(0, vocab)
    elif kind == 2:
        t = np.minimum(np.exp(rng.random(n) * math.log(vocab + 1)).astype(np.int64), vocab) - 1
    elif kind == 3:
        t = np.sort(t)
    return t


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("seed", range(40))
def test_embedding(seed):
    rng = np.random.default_rng([1, seed])
    dtype = str(rng.choice(["f32", "bf16", "f16"]))
    grad = str(rng.choice([dtype, "f32"]))
    n, d = _spread(rng, 1, 6000), _spread(rng, 1, 3000)
    while n * d > 2_000_000:
        n = max(1, n // 2)
    vocab = _spread(rng, 1, max(1, min(40000, 4_000_000 // d)))
    tok = _ids(rng, n, vocab)
    it = int(rng.integers(0, 2))
    t = torch.from_numpy(tok).to([torch.int32, torch.int64][it]).cuda()
    # ids at any multiple of their size
    t = torch.cat([t.new_zeros(3), t])[int(rng.integers(0, 4)):]
    t = t[t.numel() - n:]
    scale = float(np.float32(rng.choice([1.0, -0.5, math.sqrt(d)])))
    table = Framed(vocab, d, DT[dtype], _stride(rng, d), int(rng.integers(0, 9)),
                   fill=rounded(rng, (vocab, d), dtype))
    out = Framed(n, d, DT[dtype], _stride(rng, d), int(rng.integers(0, 9)))
    capi.check(capi.embed_fwd(CODE[dtype], it, t.data_ptr(), table.view.data_ptr(), table.ld,
                              out.view.data_ptr(), out.ld, n, vocab, d, scale, _stream()))
    dout = Framed(n, d, DT[dtype], _stride(rng, d), int(rng.integers(0, 9)),
                  fill=rounded(rng, (n, d), dtype))
    old = rounded(rng, (vocab, d), grad)
    acc = int(rng.integers(0, 2))
    g = Framed(vocab, d, DT[grad], _stride(rng, d), int(rng.integers(0, 9)), fill=old)
    ws = torch.full((capi.embed_bwd_workspace_size(n, vocab, d),), 0xC3, dtype=torch.uint8,
                    device="cuda")
    capi.check(capi.embed_bwd(CODE[dtype], CODE[grad], it, dout.view.data_ptr(), dout.ld,
                              t.data_ptr(), g.view.data_ptr(), g.ld, n, vocab, d, scale, acc,
                              ws.data_ptr(), ws.numel(), _stream()))
    torch.cuda.synchronize()
    for f in (table, out, dout, g):
        f.check()
    there = torch.from_numpy((tok >= 0) & (tok < vocab)).cuda()
    at = torch.from_numpy(tok).cuda().clamp(0, vocab - 1)
    want = (table.view[at].float() * scale).to(DT[dtype])
    want[~there] = 0
    assert torch.equal(out.view, want)
    want, absum, terms = ot.embed_backward(dout.f64(), tok, vocab, scale)
    token_checks.check_embed_bwd(g.f64(), want, absum, terms, grad, old=f64(old) if acc else None)


@pytest.mark.parametrize("seed", range(60))
def test_log_probabilities(seed):
    rng = np.random.default_rng([2, seed])
    dtype = str(rng.choice(["f32", "bf16", "f16"]))
    vocab = _spread(rng, 1, 200000)
    rows = min(_spread(rng, 1, 800), max(1, 1_500_000 // vocab))
    top = int(min(vocab, rng.choice([0, 1, 2, 7, 16, 17, 31, 32])))
    scale = float(np.float32(rng.choice([1.0, 0.3, 1.7, 10.0])))
    std = float(rng.choice([0.1, 1.0, 4.0, 30.0]))
    x = Framed(rows, vocab, DT[dtype], _stride(rng, vocab), int(rng.integers(0, 9)),
               fill=rounded(rng, (rows, vocab), dtype, std))
    mask = rng.choice([0.0, 0.0, 0.5, 0.999])
    if mask:
        low = float("-inf") if rng.random() < 0.5 else torch.finfo(DT[dtype]).min
        x.view[torch.from_numpy(rng.random((rows, vocab)) < mask).cuda()] = low
        x.before.copy_(x.bits)
    it = int(rng.integers(0, 2))
    tgt = _ids(rng, rows, vocab)
    t = torch.from_numpy(tgt).to([torch.int32, torch.int64][it]).cuda()
    ent = bool(rng.integers(0, 2))
    outs = [Framed(1, rows, torch.float32) for _ in range(3)]
    ids = Framed(rows, max(top, 1), t.dtype)
    tl = Framed(rows, max(top, 1), torch.float32)
    capi.check(capi.logprob_fwd(CODE[dtype], it, x.view.data_ptr(), x.ld, t.data_ptr(),
                                outs[0].view.data_ptr(), outs[1].view.data_ptr() if ent else 0,
                                outs[2].view.data_ptr(), ids.view.data_ptr(), tl.view.data_ptr(),
                                rows, vocab, top, scale, _stream()))
    torch.cuda.synchronize()
    for f in outs + [x, ids, tl]:
        f.check()
    want = ot.logprob(x.f64(), tgt, scale, top)
    got = {"logp": outs[0].f64()[0], "entropy": outs[1].f64()[0] if ent else None,
           "lse": outs[2].f64()[0]}
    if top:
        got.update(top_ids=ids.view.cpu().numpy(), top_logp=tl.f64())
    token_checks.check_logprob(got, want, x.f64(), scale)

    # the gradient, where an FP32 lse holds log p
    lse = outs[2].view[0].contiguous()
    if bool((lse.abs() >= 4096).any()):
        return
    h = None if rng.random() < 0.4 else rounded(rng, (rows,), "f32")
    g = rounded(rng, (rows,), "f32")
    H = torch.from_numpy(want["entropy"]).float().cuda()
    d = Framed(rows, vocab, DT[dtype], _stride(rng, vocab), int(rng.integers(0, 9)))
    capi.check(capi.logprob_bwd(CODE[dtype], it, g.data_ptr(), 0 if h is None else h.data_ptr(),
                                x.view.data_ptr(), x.ld, t.data_ptr(), lse.data_ptr(),
                                H.data_ptr(), d.view.data_ptr(), d.ld, rows, vocab, scale,
                                _stream()))
    torch.cuda.synchronize()
    d.check()
    ref, mag, factor = ot.logprob_backward(f64(g), None if h is None else f64(h), x.f64(), tgt,
                                           f64(lse), f64(H), scale)
    token_checks.check_logprob_bwd(d.f64(), ref, mag, factor, dtype)


def test_calls_from_several_threads():
    """Every thread on a stream of its own, shapes of every launch path."""
    errors = []

    def work(k):
        try:
            rng = np.random.default_rng([3, k])
            with torch.cuda.stream(torch.cuda.Stream()):
                for n, vocab, d in ((100, 300, 64), (5000, 900, 33), (40000, 5000, 16)):
                    tok = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
                    x = torch.from_numpy(rng.integers(-4, 5, (n, d)).astype(np.float32)).cuda()
                    want = torch.zeros(vocab, d, device="cuda").index_add_(0, tok, x)
                    for _ in range(5):
                        if not torch.equal(rn.embed_bwd(x, tok, vocab), want):
                            raise AssertionError("gradient")
                        if not torch.equal(rn.embed_fwd(tok, want), want[tok]):
                            raise AssertionError("rows")
                for rows, v in ((1, 40000), (30, 9000), (700, 500)):
                    x = torch.from_numpy(rng.standard_normal((rows, v)).astype(np.float32)).cuda()
                    first = rn.logprob_fwd(x, top=9)
                    for _ in range(5):
                        again = rn.logprob_fwd(x, top=9)
                        if not all(a is b or torch.equal(a, b) for a, b in zip(first, again)):
                            raise AssertionError("log probabilities")
                    if not torch.equal(first[3], torch.sort(x, dim=1, descending=True,
                                                            stable=True).indices[:, :9]):
                        raise AssertionError("alternatives")
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_pinned_host_logits():
    """Logits, gradients and outputs in pinned host memory, as the norms take them."""
    x = (torch.randn(6, 3001) * 3).pin_memory()
    t = torch.randint(0, 3001, (6,)).pin_memory()
    logp, ent, lse, ids, top = rn.logprob_fwd(x, t, top=4)
    torch.cuda.synchronize()
    assert not logp.is_cuda and not ids.is_cuda
    want = ot.logprob(x.double().numpy(), t.numpy(), 1.0, 4)
    token_checks.check_logprob({"logp": f64(logp), "entropy": f64(ent), "lse": f64(lse),
                                "top_ids": ids.numpy(), "top_logp": f64(top)}, want,
                               x.double().numpy(), 1.0)
    g = torch.ones(6).pin_memory()
    d = rn.logprob_bwd(g, x, t, lse)
    torch.cuda.synchronize()
    ref, mag, factor = ot.logprob_backward(f64(g), None, x.double().numpy(), t.numpy(), f64(lse),
                                           None, 1.0)
    token_checks.check_logprob_bwd(f64(d), ref, mag, factor, "f32")
