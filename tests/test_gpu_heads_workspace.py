"""What the gradient's sums and the append's queries are made of: nothing that the workspace held
before, and the bits that the other entry point gives."""
import pytest
import torch

import head_checks
import row_wise_normalization_gb300 as rn
from row_wise_normalization_gb300 import capi
from test_gpu_heads import EPS, TYPES, Case, _bits
from test_gpu_kv_cache import E4M3, make_cache
from token_util import DT, f64, rounded

pytestmark = pytest.mark.gpu

# one CTA's work and thousands', both directions' heads alone, every access width and number of lanes
# (5, 6 and 10 among them), several tokens to a warp
SIZES = [(1, 1, 1, 64, 64), (5, 4, 4, 32, 32), (4, 3, 0, 6, 2), (700, 20, 4, 64, 64), (3000, 3, 1, 32, 16),
         (9000, 2, 1, 32, 32), (300, 8, 1, 128, 0), (11, 7, 4, 40, 40), (12, 13, 2, 48, 24),
         (10, 7, 3, 80, 40), (9, 7, 3, 80, 20), (9, 9, 3, 78, 78), (4, 3, 1, 512, 512), (3, 2, 1, 510, 510),
         (5, 3, 2, 130, 66), (2, 65, 17, 64, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot", SIZES)
def test_sums_hold_nothing_of_the_workspace(n, hq, hk, d, rot, interleaved, dtype):
    """A workspace of NaN (all bits set) and one of zeros: the same bits, right to the definition;
    what lies behind the workspace's bytes is left alone."""
    c = Case(n, hq, hk, d, rot, dtype, True, interleaved)
    gq = rounded(c.rng, (n, hq, d), dtype, 0.7)
    gk = rounded(c.rng, (n, hk, d), dtype, 0.7) if hk else None
    need, got = capi.qk_rope_bwd_workspace_size(d), []
    for fill in (0xFF, 0):
        ws = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        got.append(rn.qk_rope_bwd(gq, gk, c.q, c.k, *c.args(), **c.kw, workspace=ws[:need]))
        assert bool((ws[need:] == fill).all())
    for a, b in zip(*got):
        assert (a is None and b is None) or torch.equal(_bits(a), _bits(b))
    for which, g, dw, heads in (("q", gq, got[0][2], hq), ("k", gk, got[0][3], hk)):
        if heads:
            head_checks.check_dw(f64(dw), c.want_bwd(which, g), n, hq + hk, dtype, "dw" + which)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "e4m3"),
                                         ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("layout", ["by_token", "by_head", "halves"])
@pytest.mark.parametrize("n,hq,hk,d,rot,norm", [(1, 4, 1, 64, 64, True), (37, 8, 2, 128, 128, True),
                                                (20, 5, 3, 80, 40, False), (33, 6, 3, 34, 34, True),
                                                (14, 5, 1, 256, 256, True), (9, 3, 1, 512, 64, True)])
def test_appends_queries_and_keys_are_the_forwards(n, hq, hk, d, rot, norm, layout, dtype, cache):
    """Rows of one width, which both entry points read by the same accesses: the same bits of the
    queries, and of the keys where the cache is of the rows' type."""
    c = Case(n, hq, hk, d, rot, dtype, norm, n % 2 == 0)
    v = rounded(c.rng, (n, hk, d), dtype)
    eight = cache == "e4m3"
    _, kc, vc = make_cache(c.rng, layout, n // 16 + 1, 16, hk, d, d, E4M3 if eight else DT[dtype])
    slots = torch.arange(n, device="cuda")
    got = rn.kv_append(c.k, v, slots, kc, vc, c.pos, c.table, c.wk, EPS, q=c.q, wq=c.wq, norm=norm,
                       **c.kw)
    q, k = rn.qk_rope_fwd(c.q, c.k, c.pos, c.table, c.wq, c.wk, EPS, norm=norm, **c.kw)
    assert torch.equal(_bits(got), _bits(q))
    if not eight:
        held = kc[slots // 16, slots % 16].contiguous()
        assert torch.equal(_bits(held), _bits(k.contiguous()))
