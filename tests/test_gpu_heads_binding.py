"""The head operators' two ways from Python into the library, the native one for plain calls and
the general one: the same bits, the same refusals."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
from row_wise_normalization_gb300 import tokens
from test_gpu_heads import EPS, TYPES, Case, _bits
from token_util import rounded

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def _both(monkeypatch, fn, native=True):
    """fn() by the native way and in Python; native: whether the first takes the call."""
    rn.qk_rope_fwd(torch.zeros(1, 1, 2, device="cuda"), None)        # (the way is looked for once)
    found = tokens._B
    if isinstance(found, tokens._InPython):
        pytest.skip("the native binding is not built here")
    took = []

    class Watch:
        def __getattr__(self, name):
            def call(*args):
                out = getattr(found, name)(*args)
                took.append(out is not None)
                return out
            return call

    with monkeypatch.context() as m:
        m.setattr(tokens, "_B", Watch())
        a = fn()
    with monkeypatch.context() as m:
        m.setattr(tokens, "_B", tokens._InPython())
        b = fn()
    assert took and all(t is native for t in took)
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert (x is None) == (y is None)
        if x is not None:
            assert x.dtype is y.dtype and x.shape == y.shape and x.stride() == y.stride()
            assert not x.requires_grad and torch.equal(_bits(x), _bits(y))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,hq,hk,d,rot,norm,interleaved,itype", [
    (5, 4, 2, 64, 64, True, False, "i64"), (33, 6, 3, 80, 40, True, True, "i32"),
    (7, 3, 0, 34, 34, False, False, "i32"), (9, 2, 2, 128, 0, True, False, "i64"), (0, 2, 1, 64, 64, True, False, "i64"),
])
def test_rotation(monkeypatch, n, hq, hk, d, rot, norm, interleaved, itype, dtype):
    c = Case(n, hq, hk, d, rot, dtype, norm, interleaved, itype, outside=n > 0)
    _both(monkeypatch, lambda: rn.qk_rope_fwd(c.q, c.k, *c.args(), **c.kw))
    g = rounded(c.rng, (n, hq, d), dtype), rounded(c.rng, (n, hk, d), dtype) if hk else None
    for params in (True, False):
        _both(monkeypatch, lambda: rn.qk_rope_bwd(*g, c.q, c.k, *c.args(), param_grads=params, **c.kw))
    if not norm:
        _both(monkeypatch, lambda: rn.qk_rope_bwd(*g, None, None, c.pos, c.table, **c.kw))
    _both(monkeypatch, lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, norm=True))


def test_batches_and_orders(monkeypatch):
    c = Case(24, 4, 2, 64, 64, "bf16")
    q = c.q.contiguous().view(2, 12, 4, 64)
    k = c.k.contiguous().view(2, 12, 2, 64).transpose(1, 2).contiguous().transpose(1, 2)
    _both(monkeypatch, lambda: rn.qk_rope_fwd(q, k, c.pos.view(2, 12), c.table, c.wq, c.wk))
    _both(monkeypatch, lambda: rn.qk_rope_bwd(q, k, q, k, c.pos, c.table, c.wq, c.wk))
    _both(monkeypatch, lambda: rn.qk_rope_fwd(q.expand(2, 12, 4, 64), None, c.pos, c.table))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eight", [False, True])
def test_cache(monkeypatch, dtype, eight):
    c = Case(21, 4, 2, 64, 64, dtype)
    v = rounded(c.rng, (21, 2, 32), dtype)
    ks, vs = (0.5, 0.25) if eight else (1.0, 1.0)
    t = E4M3 if eight else c.q.dtype
    slots = torch.from_numpy(c.rng.permutation(32)[:21]).cuda()
    slots[3] = -1

    def run(q):
        kc, vc = torch.zeros(4, 8, 2, 64, device="cuda").to(t), torch.zeros(4, 2, 8, 32, device="cuda").to(t)
        vc = vc.transpose(1, 2)
        out = rn.kv_append(c.k, v, slots, kc, vc, c.pos, c.table, c.wk, EPS, q=c.q if q else None,
                           wq=c.wq if q else None, k_scale=ks, v_scale=vs)
        return (out, kc, vc) + rn.kv_gather(kc, vc, slots, k_scale=ks, v_scale=vs)

    _both(monkeypatch, lambda: run(True))
    _both(monkeypatch, lambda: run(False))
    if eight:
        kc = torch.zeros(4, 8, 2, 64, device="cuda").to(E4M3)
        for out in (None, torch.float32, torch.float16):
            _both(monkeypatch, lambda: rn.kv_gather(kc, kc, slots, dtype=out))


def test_slots(monkeypatch):
    for t in (torch.int32, torch.int64):
        table = torch.randperm(60, device="cuda").view(5, 12).to(t)
        starts = torch.tensor([3, 0, 7, 1, 40], device="cuda").to(t)
        offsets = torch.tensor([0, 4, 4, 30, 31, 50], device="cuda").to(t)
        _both(monkeypatch, lambda: rn.kv_slots(table, starts, offsets, 53, 4))
        _both(monkeypatch, lambda: rn.kv_slots(table[:, 2:7], starts, offsets, 53, 4))


def test_what_is_not_plain_goes_the_general_way(monkeypatch):
    c = Case(8, 2, 1, 64, 64, "f32")
    pinned = c.q.cpu().pin_memory()
    for fn in (lambda: rn.qk_rope_fwd(pinned, None, c.pos, c.table),
               lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table[:, :0]),
               lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, norm=1)):
        _both(monkeypatch, fn, native=False)
    # a wrong call says so in either case, and has written nothing
    for way in (tokens._B, tokens._InPython()):
        with monkeypatch.context() as m:
            m.setattr(tokens, "_B", way)
            for bad, kind in [
                (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos[1:], c.table), ValueError),
                (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table[:, :63]), rn.RowNormError),
                (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, c.wq, eps=float("nan")), rn.RowNormError),
                (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos.float(), c.table), TypeError),
                (lambda: rn.qk_rope_fwd(c.q, c.k.half(), c.pos, c.table), TypeError),
                (lambda: rn.qk_rope_fwd(c.q, 3, c.pos, c.table), TypeError),
                (lambda: rn.qk_rope_bwd(c.q, c.k, c.q[1:], c.k, c.pos, c.table, c.wq), ValueError),
                (lambda: rn.kv_gather(c.q, c.q, c.pos), ValueError),
                (lambda: rn.kv_slots(c.pos.view(2, 4), c.pos[:2], c.pos[:2], 4, 16), ValueError),
                (lambda: rn.kv_slots(c.pos.view(2, 4), c.pos[:2], c.pos[:3], 4, 0), rn.RowNormError),
            ]:
                with pytest.raises(kind):
                    bad()


def test_leaves_that_need_gradients_and_many_calls():
    """Calls on leaves of autograd, and no memory held behind the results."""
    c = Case(50, 4, 2, 64, 64, "bf16")
    w = c.wq.clone().requires_grad_()
    q, k = rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, w, c.wk)
    assert torch.equal(q, rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, c.wq, c.wk)[0])
    torch.cuda.synchronize()
    del q, k
    before = torch.cuda.memory_allocated()
    for _ in range(200):
        rn.qk_rope_bwd(*rn.qk_rope_fwd(c.q, c.k, *c.args()), c.q, c.k, *c.args())
    assert torch.cuda.memory_allocated() == before
