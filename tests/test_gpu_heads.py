"""Norms of queries and keys with the position rotation, and their gradient, against the
float64 definitions."""
import numpy as np
import pytest
import torch

import head_checks
import row_wise_normalization_gb300 as rn
from oracle import heads as oh
from row_wise_normalization_gb300 import capi
from token_util import DT, f64, rounded

pytestmark = pytest.mark.gpu
IT = {"i32": torch.int32, "i64": torch.int64}
TYPES = ["f32", "bf16", "f16"]
EPS = float(np.float32(1e-5))


def _bits(t):
    return t.contiguous().view(torch.uint8)


def table_of(rng, rows, rot):
    a = rng.uniform(-3.2, 3.2, (rows, rot // 2))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


class Case:
    """Inputs of a call, on the GPU; queries and keys from one packed matrix."""

    def __init__(self, n, hq, hk, d, rot, dtype, norm=True, interleaved=False, itype="i64",
                 outside=True, rows=50):
        rng = np.random.default_rng([n, hq, hk, d, rot])
        self.rng, self.n, self.hq, self.hk, self.d, self.dtype = rng, n, hq, hk, d, dtype
        packed = rounded(rng, (n, hq + hk, d), dtype, 1.7)
        self.q = packed[:, :hq]
        self.k = packed[:, hq:] if hk else None
        self.wq = rounded(rng, (d,), dtype) if norm else None
        self.wk = rounded(rng, (d,), dtype) if norm and hk else None
        pos = rng.integers(0, rows, n)
        if outside and n > 3:
            pos[1], pos[n - 1] = -1, rows
        self.pos = torch.from_numpy(pos).to(IT[itype]).cuda()
        self.table = table_of(rng, rows, rot) if rot else None
        self.norm, self.kw = norm, dict(interleaved=interleaved)

    def args(self):
        return (self.pos, self.table, self.wq, self.wk, EPS)

    def want(self, which):
        x, w = (self.q, self.wq) if which == "q" else (self.k, self.wk)
        return oh.rope(f64(x), None if w is None else f64(w), self.pos.cpu().numpy(),
                       None if self.table is None else f64(self.table), EPS, self.norm,
                       self.kw["interleaved"])

    def want_bwd(self, which, dy):
        x, w = (self.q, self.wq) if which == "q" else (self.k, self.wk)
        return oh.rope_backward(f64(dy), f64(x), None if w is None else f64(w),
                                self.pos.cpu().numpy(),
                                None if self.table is None else f64(self.table), EPS, self.norm,
                                self.kw["interleaved"])


# every lane count and access width: vectors of 16 bytes, pairs, single values
SHAPES = [
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (5, 4, 4, 32, 32), (3, 2, 1, 2, 2), (4, 3, 0, 6, 2),
    (33, 12, 3, 96, 32), (17, 5, 2, 80, 80), (9, 7, 3, 80, 20), (6, 3, 1, 34, 34), (5, 2, 2, 256, 64),
    (4, 3, 1, 512, 512), (3, 2, 1, 510, 510), (4, 2, 1, 510, 250), (7, 70, 9, 16, 8),
    (300, 8, 1, 128, 0), (40, 9, 5, 112, 56), (8, 6, 2, 192, 128), (5, 3, 2, 130, 66), (6, 2, 1, 508, 4),
    (5, 3, 2, 132, 128), (2, 65, 17, 64, 32), (7, 2, 2, 10, 6),
    (11, 7, 4, 40, 40), (12, 13, 2, 48, 24), (10, 7, 3, 80, 40), (6, 5, 2, 72, 8), (7, 3, 2, 100, 100),
    (5, 5, 1, 140, 140), (9, 9, 3, 78, 78), (4, 3, 2, 222, 222), (6, 9, 5, 24, 24), (3, 2, 2, 384, 256),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("norm,interleaved,itype", [(True, False, "i64"), (True, True, "i32"),
                                                    (False, False, "i32"), (False, True, "i64")])
@pytest.mark.parametrize("n,hq,hk,d,rot", SHAPES)
def test_forward(n, hq, hk, d, rot, norm, interleaved, itype, dtype):
    c = Case(n, hq, hk, d, rot, dtype, norm, interleaved, itype)
    q, k = rn.qk_rope_fwd(c.q, c.k, *c.args(), **c.kw)
    head_checks.check_rope(f64(q), *c.want("q"), norm, dtype, "q")
    if hk:
        head_checks.check_rope(f64(k), *c.want("k"), norm, dtype, "k")
    else:
        assert k is None
    if not norm and not rot:
        assert torch.equal(_bits(q), _bits(c.q))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("param_grads", [True, False])
@pytest.mark.parametrize("norm,interleaved,itype", [(True, False, "i64"), (True, True, "i32"),
                                                    (False, True, "i32")])
@pytest.mark.parametrize("n,hq,hk,d,rot", SHAPES + [(3000, 3, 1, 32, 16), (700, 20, 4, 64, 64)])
def test_backward(n, hq, hk, d, rot, norm, interleaved, itype, param_grads, dtype):
    c = Case(n, hq, hk, d, rot, dtype, norm, interleaved, itype)
    gq = rounded(c.rng, (n, hq, d), dtype, 0.7)
    gk = rounded(c.rng, (n, hk, d), dtype, 0.7) if hk else None
    ws = torch.full((capi.qk_rope_bwd_workspace_size(d),), 0xA5, dtype=torch.uint8, device="cuda")
    dq, dk, dwq, dwk = rn.qk_rope_bwd(gq, gk, c.q, c.k, *c.args(), **c.kw, param_grads=param_grads,
                                      workspace=ws if param_grads else None)
    again = rn.qk_rope_bwd(gq, gk, c.q, c.k, *c.args(), **c.kw, param_grads=param_grads)
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert (a is None and b is None) or torch.equal(_bits(a), _bits(b))
    for which, g, dx, dw, heads in (("q", gq, dq, dwq, hq), ("k", gk, dk, dwk, hk)):
        if not heads:
            assert dx is None and dw is None
            continue
        want = c.want_bwd(which, g)
        head_checks.check_rope_bwd(f64(dx), want, norm, dtype, "d" + which)
        if norm and param_grads:
            head_checks.check_dw(f64(dw), want, n, hq + hk, dtype, "dw" + which)
        else:
            assert dw is None


def _guarded(shape, dtype):
    """A tensor of one bit pattern, to see what is written of it."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    _fill(t)
    return t


def _fill(t):
    t.view(torch.uint8).fill_(0x5A)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["packed", "head_major", "batched", "batched_head_major", "shifted1",
                                    "shifted2", "wide"])
@pytest.mark.parametrize("d,rot", [(64, 64), (80, 32), (20, 10)])
def test_layouts(layout, d, rot, dtype):
    """Outputs as blocks of one matrix, or in other orders than the inputs', both directions; the
    memory between rows keeps its bits."""
    b, s, hq, hk = 3, 11, 6, 2
    n, t = b * s, DT[dtype]
    c = Case(n, hq, hk, d, rot, dtype, rows=60)
    gq, gk = rounded(c.rng, (n, hq, d), dtype), rounded(c.rng, (n, hk, d), dtype)

    def place(total):
        """(whole, views) of tensors for heads hq and hk inside one allocation."""
        if layout in ("packed", "wide"):
            whole = _guarded((n, total + (3 if layout == "wide" else 0), d), t)
            return whole, lambda a, h: whole[:, a:a + h]
        if layout.startswith("shifted"):
            off = int(layout[-1])
            whole = _guarded((n * total * d + 8,), t)
            inner = whole[off:off + n * total * d].view(n, total, d)
            return whole, lambda a, h: inner[:, a:a + h]
        if layout == "head_major":
            whole = _guarded((total, n, d), t)
            return whole, lambda a, h: whole[a:a + h].transpose(0, 1)
        if layout == "batched":
            whole = _guarded((b, s, total, d), t)
            return whole, lambda a, h: whole[:, :, a:a + h]
        whole = _guarded((b, total, s, d), t)
        return whole, lambda a, h: whole[:, a:a + h].transpose(1, 2)

    def shaped(x, like):
        return x.view(b, s, x.shape[1], d) if like.dim() == 4 else x

    total = hq + hk + 1                       # a head between them stays as it is
    src, at = place(total)
    q, k = at(0, hq), at(hq + 1, hk)
    q.copy_(shaped(c.q, q))
    k.copy_(shaped(c.k, k))
    whole, at2 = place(total)
    qo, ko = at2(0, hq), at2(hq + 1, hk)
    got = rn.qk_rope_fwd(q, k, *c.args(), q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    ref = rn.qk_rope_fwd(c.q.contiguous(), c.k.contiguous(), *c.args())
    head_checks.check_rope(f64(qo.reshape(n, hq, d)), *c.want("q"), True, dtype, "q")
    head_checks.check_rope(f64(ko.reshape(n, hk, d)), *c.want("k"), True, dtype, "k")
    if not layout.startswith("shifted"):
        assert torch.equal(qo.reshape(n, hq, d), ref[0]) and torch.equal(ko.reshape(n, hk, d), ref[1])

    def untouched(whole, views):
        back = whole.clone()
        for v in views:
            v.view(torch.int32 if v.element_size() == 4 else torch.int16).fill_(
                0x5A5A5A5A if v.element_size() == 4 else 0x5A5A)
        assert bool((whole.view(torch.uint8) == 0x5A).all())
        whole.copy_(back)

    untouched(whole, (qo, ko))
    # the gradient: of and into the same kind of memory, then in the place of what reaches it
    gwhole, at3 = place(total)
    go_q, go_k = at3(0, hq), at3(hq + 1, hk)
    go_q.copy_(shaped(gq, go_q))
    go_k.copy_(shaped(gk, go_k))
    want_q, want_k = c.want_bwd("q", gq), c.want_bwd("k", gk)
    _fill(whole)
    dq, dk, dwq, dwk = rn.qk_rope_bwd(go_q, go_k, q, k, *c.args(), dq=qo, dk=ko)
    head_checks.check_rope_bwd(f64(dq.reshape(n, hq, d)), want_q, True, dtype)
    head_checks.check_rope_bwd(f64(dk.reshape(n, hk, d)), want_k, True, dtype)
    head_checks.check_dw(f64(dwq), want_q, n, hq + hk, dtype)
    head_checks.check_dw(f64(dwk), want_k, n, hq + hk, dtype)
    inplace = rn.qk_rope_bwd(go_q, go_k, q, k, *c.args(), dq=go_q, dk=go_k)
    assert torch.equal(go_q, dq) and torch.equal(go_k, dk)
    assert torch.equal(inplace[2], dwq) and torch.equal(inplace[3], dwk)
    untouched(whole, (qo, ko))
    untouched(gwhole, (go_q, go_k))
    # the forward pass in its inputs' place
    rn.qk_rope_fwd(q, k, *c.args(), q_out=q, k_out=k)
    head_checks.check_rope(f64(q.reshape(n, hq, d)), *c.want("q"), True, dtype, "q in place")
    untouched(src, (q, k))


@pytest.mark.parametrize("dtype", TYPES)
def test_repeated_rows_as_inputs(dtype):
    """Inputs of stride 0: one head for all, one token for all."""
    c = Case(9, 4, 1, 64, 64, dtype)
    one = c.k.expand(9, 4, 64)
    got, _ = rn.qk_rope_fwd(one, None, c.pos, c.table, c.wk, None, EPS)
    want = rn.qk_rope_fwd(one.contiguous(), None, c.pos, c.table, c.wk, None, EPS)[0]
    assert torch.equal(got, want)
    g = rounded(c.rng, (1, 4, 64), dtype).expand(9, 4, 64)
    a = rn.qk_rope_bwd(g, None, one, None, c.pos, c.table, c.wk, None, EPS)
    b = rn.qk_rope_bwd(g.contiguous(), None, one.contiguous(), None, c.pos, c.table, c.wk, None, EPS)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    with pytest.raises(rn.RowNormError, match="overlap"):
        rn.qk_rope_fwd(one, None, c.pos, c.table, c.wk, None, EPS, q_out=one)


def test_strided_and_shifted_table():
    c = Case(20, 3, 1, 64, 48, "bf16")
    want = rn.qk_rope_fwd(c.q, c.k, *c.args())
    for ld, off in ((64, 0), (50, 0), (49, 1), (48, 3), (52, 2)):
        flat = torch.full((50 * ld + off,), float("nan"), device="cuda")
        table = flat[off:].as_strided((50, 48), (ld, 1))
        table.copy_(c.table)
        got = rn.qk_rope_fwd(c.q, c.k, c.pos, table, c.wq, c.wk, EPS)
        head_checks.check_rope(f64(got[0]), *c.want("q"), True, "bf16", f"q {ld} {off}")
        head_checks.check_rope(f64(got[1]), *c.want("k"), True, "bf16", f"k {ld} {off}")
    assert torch.equal(_bits(want[0]), _bits(rn.qk_rope_fwd(c.q, c.k, *c.args())[0]))


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_without_weights_and_one_weight(dtype):
    c = Case(12, 4, 2, 48, 48, dtype)
    c.wq = c.wk = None
    q, k = rn.qk_rope_fwd(c.q, c.k, *c.args(), norm=True)
    head_checks.check_rope(f64(q), *c.want("q"), True, dtype)
    g = rounded(c.rng, (12, 4, 48), dtype), rounded(c.rng, (12, 2, 48), dtype)
    dq, dk, dwq, dwk = rn.qk_rope_bwd(*g, c.q, c.k, *c.args(), norm=True)
    assert dwq is None and dwk is None
    head_checks.check_rope_bwd(f64(dk), c.want_bwd("k", g[1]), True, dtype)
    c.wk = rounded(c.rng, (48,), dtype)
    q2, k2 = rn.qk_rope_fwd(c.q, c.k, *c.args())
    assert torch.equal(q, q2)
    head_checks.check_rope(f64(k2), *c.want("k"), True, dtype)
    dq2, dk2, dwq, dwk = rn.qk_rope_bwd(*g, c.q, c.k, *c.args())
    assert dwq is None and torch.equal(dq, dq2)
    head_checks.check_dw(f64(dwk), c.want_bwd("k", g[1]), 12, 6, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 34])
def test_special_values_stay_in_their_rows(dtype, d):
    c = Case(8, 3, 1, d, d, dtype, outside=False)
    q = c.q.contiguous()
    clean = rn.qk_rope_fwd(q, None, c.pos, c.table, c.wq, None, EPS)[0]
    q[2, 1] = 0
    q[3, 0, 5] = float("inf")
    q[4, 2, 0] = float("nan")
    got = rn.qk_rope_fwd(q, None, c.pos, c.table, c.wq, None, EPS)[0]
    same = torch.ones(8, 3, dtype=torch.bool, device="cuda")
    same[2, 1] = same[3, 0] = same[4, 2] = False
    assert torch.equal(got[same], clean[same])
    assert not bool(got[2, 1].any()) and bool(got[4, 2].isnan().all())
    assert bool(got[3, 0].isnan().any())
    # rows of padding count for nothing, whatever they hold
    g = rounded(c.rng, (8, 3, d), dtype)
    c.pos[3], c.pos[4] = -1, 50
    g[3, 0], g[4, 2] = float("nan"), float("inf")
    dq, _, dwq, _ = rn.qk_rope_bwd(g, None, q, None, c.pos, c.table, c.wq, None, EPS)
    assert not bool(dq[3:5].any()) and bool(dwq.isfinite().all()) and bool(dq.isfinite().all())
    got = rn.qk_rope_fwd(q, None, c.pos, c.table, c.wq, None, EPS)[0]
    assert not bool(got[3:5].any())


@pytest.mark.parametrize("dtype", TYPES)
def test_empty_batches(dtype):
    q = torch.empty(0, 4, 64, dtype=DT[dtype], device="cuda")
    w = torch.ones(64, dtype=DT[dtype], device="cuda")
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    table = torch.ones(3, 64, device="cuda")
    qo, ko = rn.qk_rope_fwd(q, q[:, :2], pos, table, w, w)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    dw = torch.full((64,), 3.0, dtype=DT[dtype], device="cuda")
    _, _, a, b = rn.qk_rope_bwd(q, q[:, :2], q, q[:, :2], pos, table, w, w, dwq=dw)
    assert a is dw and not bool(a.any()) and not bool(b.any())


def test_rows_far_apart():
    """Token offsets past 2^32 bytes and 2^31 elements."""
    ld, n, d = 1 << 27, 20, 64
    flat = torch.empty(((n - 1) * ld + d,), dtype=torch.bfloat16, device="cuda")
    q = flat.as_strided((n, 1, d), (ld, d, 1))
    c = Case(n, 1, 1, d, d, "bf16")
    q.copy_(c.q)
    want = rn.qk_rope_fwd(c.q, None, c.pos, c.table, c.wq, None, EPS)[0]
    assert torch.equal(rn.qk_rope_fwd(q, None, c.pos, c.table, c.wq, None, EPS)[0], want)
    rn.qk_rope_fwd(q, None, c.pos, c.table, c.wq, None, EPS, q_out=q)
    assert torch.equal(q, want)


def test_many_tokens_gradient_of_weights():
    """Sums over every CTA, a token count that leaves the last units ragged."""
    n, hq, hk, d = 9001, 6, 2, 128
    rng = np.random.default_rng(5)
    x = rounded(rng, (n, hq + hk, d), "bf16")
    g = rounded(rng, (n, hq + hk, d), "bf16")
    w = rounded(rng, (d,), "bf16")
    pos = torch.arange(n, device="cuda") % 40
    table = table_of(rng, 40, d)
    dq, dk, dwq, dwk = rn.qk_rope_bwd(g[:, :hq], g[:, hq:], x[:, :hq], x[:, hq:], pos, table, w, w, EPS)
    # the definition in 64 bits, on the GPU
    half = d // 2
    cs, sn = table[pos].double()[:, None, :half], table[pos].double()[:, None, half:]
    gd, xd = g.double(), x.double()
    t = torch.cat([gd[..., :half] * cs + gd[..., half:] * sn, gd[..., half:] * cs - gd[..., :half] * sn], -1)
    mag = torch.cat([gd[..., :half].abs() * cs.abs() + gd[..., half:].abs() * sn.abs(),
                     gd[..., half:].abs() * cs.abs() + gd[..., :half].abs() * sn.abs()], -1)
    r = (xd.square().mean(-1, keepdim=True) + EPS).rsqrt()
    for sl, dw in ((slice(0, hq), dwq), (slice(hq, None), dwk)):
        want = {"dw": (t * xd * r)[:, sl].sum((0, 1)).cpu().numpy(),
                "dw_abs": (mag * xd.abs() * r)[:, sl].sum((0, 1)).cpu().numpy()}
        head_checks.check_dw(f64(dw), want, n, hq + hk, "bf16")


def test_graph_replays_follow_their_inputs():
    """Forward and gradient captured together, with two workspaces' graphs on two streams."""
    cases = [Case(70, 8, 2, 128, 128, "bf16"), Case(33, 4, 4, 80, 40, "bf16")]
    graphs = []
    for c in cases:
        g = rounded(c.rng, (c.n, c.hq, c.d), "bf16"), rounded(c.rng, (c.n, c.hk, c.d), "bf16")
        x = c.q.clone(), c.k.clone()
        ws = torch.empty(capi.qk_rope_bwd_workspace_size(c.d), dtype=torch.uint8, device="cuda")
        run = lambda c=c, g=g, x=x, ws=ws: (rn.qk_rope_fwd(*x, *c.args()),  # noqa: E731
                                            rn.qk_rope_bwd(*g, *x, *c.args(), workspace=ws))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out, x, run, side))
    for k in range(3):
        for graph, out, x, run, side in graphs:
            for t in x:
                t.normal_(generator=torch.Generator(device="cuda").manual_seed(k))
        torch.cuda.synchronize()
        for graph, out, x, run, side in graphs:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for graph, out, x, run, side in graphs:
            for a, b in zip(out[0] + out[1], sum(run(), ())):
                assert torch.equal(a, b)


def test_streams_and_refusals_of_the_binding():
    c = Case(64, 8, 2, 64, 64, "f16")
    want = rn.qk_rope_fwd(c.q, c.k, *c.args())
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = rn.qk_rope_fwd(c.q, c.k, *c.args(), stream=st)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad, kind in [
        (lambda: rn.qk_rope_fwd(c.q, c.k[:-1], *c.args()), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k[..., :32], *c.args()), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k.float(), *c.args()), TypeError),
        (lambda: rn.qk_rope_fwd(c.q.transpose(1, 2), None), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos[:-1], c.table), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, None, c.table), TypeError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table[0]), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table.t()), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, c.pos, c.table[:, :63]), rn.RowNormError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, *c.args()[:2], c.wq[:-1]), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, *c.args()[:2], c.wq.float()), TypeError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, *c.args()[:4], -1.0), rn.RowNormError),
        (lambda: rn.qk_rope_fwd(c.q, None, k_out=want[1]), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, q_out=want[0][1:]), ValueError),
        (lambda: rn.qk_rope_fwd(c.q, c.k, q_out=c.q[:, :, :].flip(0)[:64].contiguous().float()), TypeError),
        (lambda: rn.qk_rope_bwd(c.q, c.k, None, None, wq=c.wq), TypeError),
        (lambda: rn.qk_rope_bwd(c.q, c.k, None, None, dwq=c.wq), ValueError),
        (lambda: rn.qk_rope_bwd(c.q, None, None, None, dk=c.k), ValueError),
        (lambda: rn.qk_rope_bwd(want[0], want[1], c.q, c.k, *c.args(),
                                workspace=torch.empty(16, device="cuda")), rn.RowNormError),
        (lambda: rn.qk_rope_bwd(want[0], want[1], c.q, c.k, *c.args(), workspace=torch.empty(16)),
         ValueError),
    ]:
        with pytest.raises(kind):
            bad()


def test_host_rows():
    """Pinned host tensors, read and written in place."""
    c = Case(37, 4, 2, 64, 32, "f32")
    q, k = c.q.cpu().pin_memory(), c.k.cpu().pin_memory()
    want = rn.qk_rope_fwd(c.q, c.k, *c.args())
    got = rn.qk_rope_fwd(q, k, *c.args(), q_out=torch.empty_like(q).pin_memory(),
                         k_out=torch.empty_like(k).pin_memory())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0].cpu()) and torch.equal(got[1], want[1].cpu())


@pytest.mark.parametrize("dtype", TYPES)
def test_keys_alone_through_the_c_abi(dtype):
    """No queries: every unit and every partial sum belongs to the keys."""
    c = Case(37, 1, 3, 64, 64, dtype)
    code = {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    n, hk, d = 37, 3, 64
    k, none = c.k.contiguous(), capi.heads(0, 0, 0, 0, 0)
    rows = lambda t: (t.data_ptr(), hk, 0, hk * d, d)  # noqa: E731
    g = rounded(c.rng, (n, hk, d), dtype)
    out, dk = torch.empty_like(k), torch.empty_like(k)
    dw = torch.empty(d, dtype=DT[dtype], device="cuda")
    ws = torch.empty(capi.qk_rope_bwd_workspace_size(d), dtype=torch.uint8, device="cuda")
    qk = capi.qk(0, 0, 0, 0, 0, *rows(k), 0, c.wk.data_ptr(), c.pos.data_ptr(), c.table.data_ptr(), 50, 64,
                 64, 1, n, d, code, 1, 1, 0, EPS, 0)
    st = torch.cuda.current_stream().cuda_stream
    capi.check(capi.qk_rope_fwd(qk, none, capi.heads(*rows(out)), st))
    capi.check(capi.qk_rope_bwd(qk, none, capi.heads(*rows(g)), none, capi.heads(*rows(dk)), 0,
                                dw.data_ptr(), ws.data_ptr(), ws.numel(), st))
    head_checks.check_rope(f64(out), *c.want("k"), True, dtype)
    want = c.want_bwd("k", g)
    head_checks.check_rope_bwd(f64(dk), want, True, dtype)
    head_checks.check_dw(f64(dw), want, n, hk, dtype)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    """Shapes, strides, alignments, types and modes at random."""
    rng = np.random.default_rng([77, seed])
    dtype = TYPES[rng.integers(3)]
    d = 2 * int(rng.integers(1, 100)) if rng.random() < 0.6 else int(rng.choice([64, 80, 96, 112, 128, 192, 256, 384]))
    rot = int(rng.choice([d, d // 4 * 2, 2 * rng.integers(0, d // 2 + 1)]))
    n, hq, hk = int(rng.integers(1, 90)), int(rng.integers(1, 14)), int(rng.integers(0, 6))
    norm = bool(rng.random() < 0.7)
    c = Case(n, hq, hk, d, rot, dtype, norm, bool(rng.random() < 0.5), "i32" if seed % 2 else "i64")

    def place(x):
        """The values of x in memory with gaps between tokens and heads, at some element offset."""
        if x is None:
            return None
        gap, head, off = int(rng.integers(0, 9)), int(rng.integers(0, 5)), int(rng.integers(0, 9))
        if rng.random() < 0.4:
            gap, head, off = 0, 0, 0
        hs = d + head
        ts = x.shape[1] * hs + gap
        t = _guarded((off + n * ts,), x.dtype)[off:].as_strided(x.shape, (ts, hs, 1))
        t.copy_(x)
        return t

    q, k = place(c.q), place(c.k)
    qo, ko = place(torch.zeros_like(q)), place(torch.zeros_like(k)) if hk else None
    rn.qk_rope_fwd(q, k, *c.args(), norm=norm, q_out=qo, k_out=ko, **c.kw)
    head_checks.check_rope(f64(qo), *c.want("q"), norm, dtype, "q")
    gq, gk = place(rounded(rng, (n, hq, d), dtype)), place(rounded(rng, (n, hk, d), dtype)) if hk else None
    dq, dk, dwq, dwk = rn.qk_rope_bwd(gq, gk, q, k, *c.args(), norm=norm, dq=qo, dk=ko, **c.kw)
    want = c.want_bwd("q", gq)
    head_checks.check_rope_bwd(f64(dq), want, norm, dtype, "dq")
    if norm:
        head_checks.check_dw(f64(dwq), want, n, hq + hk, dtype, "dwq")
    if hk:
        rn.qk_rope_fwd(q, k, *c.args(), norm=norm, k_out=ko, **c.kw)
        head_checks.check_rope(f64(ko), *c.want("k"), norm, dtype, "k")
        want = c.want_bwd("k", gk)
        rn.qk_rope_bwd(gq, gk, q, k, *c.args(), norm=norm, dk=gk, **c.kw)
        head_checks.check_rope_bwd(f64(gk), want, norm, dtype, "dk in place")
