"""The token operators as they are used: with the norms between them, on other
streams, captured and replayed, back to back."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
import token_checks
from row_wise_normalization_gb300 import capi

pytestmark = pytest.mark.gpu


def _model(vocab, d, n, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=gen) * std  # noqa: E731
    return {"table": r(vocab, d, std=0.1), "gamma": 1 + 0.1 * r(d), "beta": 0.1 * r(d),
            "head": r(vocab, d, std=d ** -0.5),
            "tokens": torch.randint(0, vocab, (n,), device="cuda", generator=gen),
            "targets": torch.randint(-1, vocab, (n,), device="cuda", generator=gen)}


def _step(m, scale=4.0, coef=0.01):
    """A bigram model's training step: embedding row, LayerNorm, tied-size head,
    log probability and entropy, and the gradients of -sum logp - coef sum H."""
    x = rn.embed_fwd(m["tokens"], m["table"], scale)
    y, mean, rstd = rn.ln_fwd(x, m["gamma"], m["beta"])
    logits = y @ m["head"].t()
    logp, ent, lse, ids, top = rn.logprob_fwd(logits, m["targets"], top=3)
    dlogp = torch.full_like(logp, -1.0)
    dent = torch.full_like(ent, -coef)
    dlogits = rn.logprob_bwd(dlogp, logits, m["targets"], lse, dentropy=dent, entropy=ent)
    dy = dlogits @ m["head"]
    dhead = dlogits.t() @ y
    dx, dgamma, dbeta = rn.ln_bwd(dy, x, m["gamma"], mean, rstd)
    dtable = rn.embed_bwd(dx, m["tokens"], m["table"].shape[0], scale)
    return [logp, ent, ids, top, dhead, dgamma, dbeta, dtable]


def _reference(m, scale=4.0, coef=0.01):
    """The same step by automatic differentiation in 64 bits."""
    p = {k: m[k].double().requires_grad_(True) for k in ("table", "gamma", "beta", "head")}
    x = scale * p["table"][m["tokens"]]
    y = torch.nn.functional.layer_norm(x, x.shape[-1:], p["gamma"], p["beta"], 1e-5)
    lq = torch.log_softmax(y @ p["head"].t(), 1)
    there = m["targets"] >= 0
    logp = torch.where(there, lq.gather(1, m["targets"].clamp(min=0)[:, None])[:, 0], 0.0)
    ent = -(lq.exp() * lq).sum(1)
    (-logp.sum() - coef * ent.sum()).backward()
    return logp, ent, lq, {k: v.grad for k, v in p.items()}


def test_training_step(monkeypatch):
    # FP32 products: the library's own matrix products are not under test
    monkeypatch.setattr(torch.backends.cuda.matmul, "allow_tf32", False)
    m = _model(777, 96, 400)
    logp, ent, ids, top, dhead, dgamma, dbeta, dtable = _step(m)
    rlogp, rent, lq, grads = _reference(m)
    # FP32 chains of a few hundred terms, of order one: relative to the norm
    near = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert near(logp, rlogp) < 1e-5 and near(ent, rent) < 1e-5
    assert near(dhead, grads["head"]) < 2e-5 and near(dtable, grads["table"]) < 2e-5
    assert near(dgamma, grads["gamma"]) < 2e-5 and near(dbeta, grads["beta"]) < 2e-5
    want = lq.topk(3, dim=1)
    gap = (want.values[:, :2] - want.values[:, 1:]).min(1).values > 1e-4
    assert bool((ids[gap] == want.indices[gap]).all())


def test_on_another_stream():
    m = _model(500, 64, 300)
    want = _step(m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = rn.embed_fwd(m["tokens"], m["table"], 4.0, stream=s)
    g = rn.embed_bwd(x, m["tokens"], 500, stream=s)
    lp = rn.logprob_fwd(x, m["tokens"] % 64, top=2, stream=s)
    d = rn.logprob_bwd(lp[0], x, m["tokens"] % 64, lp[2], stream=s.cuda_stream)
    # memory of the calls' own is theirs until the stream is done with it
    junk = [torch.full_like(g, 7.0) for _ in range(8)]
    s.synchronize()
    x2 = rn.embed_fwd(m["tokens"], m["table"], 4.0)
    g2 = rn.embed_bwd(x2, m["tokens"], 500)
    lp2 = rn.logprob_fwd(x2, m["tokens"] % 64, top=2)
    d2 = rn.logprob_bwd(lp2[0], x2, m["tokens"] % 64, lp2[2])
    del junk
    assert torch.equal(x, x2) and torch.equal(g, g2) and torch.equal(d, d2)
    assert all(torch.equal(a, b) for a, b in zip(lp, lp2))
    with torch.cuda.stream(s):
        again = _step(m)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, again))


@pytest.mark.parametrize("vocab,d,n", [(900, 128, 500), (2500, 96, 7000)])
def test_captured_and_replayed(vocab, d, n):
    """The gradient in one launch, and by the sort and its companions."""
    m = _model(vocab, d, n)
    _step(m)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(m)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(m)
    for seed in (1, 2):
        other = _model(vocab, d, n, seed)
        for k in m:
            m[k].copy_(other[k])
        want = [t.clone() for t in _step(other)]
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("vocab,d,n", [(300, 256, 2000), (300, 256, 200), (3000, 200, 20000)])
def test_back_to_back_calls_see_each_other(vocab, d, n):
    """Chains in which each call reads what the one before wrote, against the
    same chain with a synchronization after every call."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    w0 = torch.randn(vocab, d, device="cuda", generator=gen)
    tok = torch.randint(0, vocab, (n,), device="cuda", generator=gen)
    tgt = torch.randint(0, d, (n,), device="cuda", generator=gen)
    ws = torch.empty(capi.embed_bwd_workspace_size(n, vocab, d), dtype=torch.uint8, device="cuda")

    def chain(sync):
        w = w0.clone()
        x = torch.empty(n, d, device="cuda")
        dx = torch.empty(n, d, device="cuda")
        for _ in range(6):
            rn.embed_fwd(tok, w, out=x)
            if sync:
                torch.cuda.synchronize()
            lp, ent, lse, _, _ = rn.logprob_fwd(x, tgt)
            if sync:
                torch.cuda.synchronize()
            rn.logprob_bwd(lp, x, tgt, lse, dentropy=ent, entropy=ent, dlogits=dx)
            if sync:
                torch.cuda.synchronize()
            rn.embed_bwd(dx, tok, vocab, 0.01, dtable=w, accumulate=True, workspace=ws)
            if sync:
                torch.cuda.synchronize()
            rn.embed_bwd(dx, tok, vocab, 0.5, dtable=w, workspace=ws)
            if sync:
                torch.cuda.synchronize()
        return w

    want = chain(True)
    for _ in range(40):
        assert torch.equal(chain(False), want)


def test_two_streams_with_workspaces_of_their_own():
    rng = np.random.default_rng(0)
    jobs = []
    for k in range(2):
        s = torch.cuda.Stream()
        tok = torch.from_numpy(rng.integers(0, 3000, 20000)).cuda()
        dout = torch.randn(20000, 64, device="cuda")
        jobs.append((s, tok, dout, rn.embed_bwd(dout, tok, 3000)))
    torch.cuda.synchronize()
    for _ in range(10):
        got = [rn.embed_bwd(dout, tok, 3000, stream=s) for s, tok, dout, _ in jobs]
        torch.cuda.synchronize()
        for g, (_, _, _, want) in zip(got, jobs):
            assert torch.equal(g, want)


def test_stream_and_device_refusals():
    t = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        rn.embed_fwd(t.float(), torch.ones(4, 4, device="cuda"))
    with pytest.raises(ValueError):
        rn.embed_fwd(t, torch.ones(4, 8, device="cuda")[:, ::2])
    assert token_checks.depth(128000) < 200


def test_large_and_small_gradients_in_turn():
    """Calls of every launch path behind each other on one stream, one workspace, one
    gradient: rows cleared by one call are read by the next."""
    rng = np.random.default_rng(1)
    vocab, d = 4000, 64
    jobs = []
    for n in (5, 40000, 300, 1500, 1, 200000, 1024, 9000):
        tok = torch.from_numpy(rng.integers(0, vocab, n)).cuda()
        x = torch.from_numpy(rng.integers(-3, 4, (n, d)).astype(np.float32)).cuda()
        jobs.append((tok, x, torch.zeros(vocab, d, device="cuda").index_add_(0, tok, x)))
    ws = torch.empty(max(capi.embed_bwd_workspace_size(t.numel(), vocab, d) for t, _, _ in jobs),
                     dtype=torch.uint8, device="cuda")
    g = torch.empty(vocab, d, device="cuda")
    for _ in range(5):
        sums = []
        for tok, x, _ in jobs:
            rn.embed_bwd(x, tok, vocab, dtable=g, workspace=ws)
            sums.append(rn.embed_fwd(torch.arange(vocab, device="cuda"), g))
            rn.embed_bwd(x, tok, vocab, dtable=g, accumulate=True, workspace=ws)
            sums.append(g * 0.5)
        for k, (_, _, want) in enumerate(jobs):
            assert torch.equal(sums[2 * k], want) and torch.equal(sums[2 * k + 1], want)


@pytest.mark.parametrize("n", [200, 1500, 9000])
def test_ids_written_by_the_kernel_ahead(n):
    """The most probable columns as the ids of the next call, in the same memory every time."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    vocab, d = 700, 96
    x = torch.randint(-3, 4, (n, d), device="cuda", generator=gen).float()
    ws = torch.empty(capi.embed_bwd_workspace_size(n, vocab, d), dtype=torch.uint8, device="cuda")
    logits = [torch.randn(n, vocab, device="cuda", generator=gen) for _ in range(8)]
    want = [torch.zeros(vocab, d, device="cuda").index_add_(0, t.argmax(1), x) for t in logits]
    g = torch.empty(vocab, d, device="cuda")
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for t in logits:
            ids = rn.logprob_fwd(t, want_entropy=False, top=1)[3]
            rn.embed_bwd(x, ids, vocab, dtable=g, workspace=ws)
            got.append(rn.embed_fwd(torch.arange(vocab, device="cuda"), g))
            del ids
        assert all(torch.equal(a, b) for a, b in zip(got, want))
