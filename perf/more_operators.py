"""What is measured of the head operators: norms of queries and keys with the
position rotation, their gradient, and the paged cache that keys and values
are appended to and gathered from.

``own`` says which side ``run`` takes: False computes the operators in their
plain form (elementary torch operations in 32 bits, rounded once at the end),
True makes the calls of this package. Both take what ``prepare`` made.

Queries, keys and values are column blocks of one projection's output, as a
network's fused projection leaves them. Positions run through packed sequences
of different lengths; the rotation's table holds cosines and sines in FP32.
Pages of a sequence lie anywhere in the cache.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
       "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
_IT = {"i32": torch.int32, "i64": torch.int64}
_EPS = float(np.float32(1e-5))
_E4M3_MAX = 448.0


def _qk(op, name, n, hq, hk, d, rot, dtype, itype, interleaved=False, norm=True):
    return {"name": name, "op": op, "n": n, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "dtype": dtype, "itype": itype, "interleaved": interleaved, "norm": norm}


def _slots(name, seqs, new, context, page, itype, pad=0):
    """seqs sequences of about `new` tokens each, after contexts of up to
    `context`; pad: tokens of the batch behind the last sequence."""
    return {"name": name, "op": "kv_slots", "seqs": seqs, "new": new, "context": context,
            "page": page, "itype": itype, "pad": pad}


def _append(name, n, hq, hk, d, rot, dtype, cache, itype, page, by_head=False,
            interleaved=False, norm=True, pad=0):
    """hq: query heads rotated in the same call (0: keys and values alone); by_head:
    a page holds its tokens head by head; pad: tokens without a slot."""
    return {"name": name, "op": "kv_append", "n": n, "hq": hq, "hk": hk, "d": d, "rot": rot,
            "dtype": dtype, "cache": cache, "itype": itype, "page": page, "by_head": by_head,
            "interleaved": interleaved, "norm": norm, "pad": pad}


def _gather(name, n, hk, d, dtype, cache, itype, page, by_head=False, pad=0):
    return {"name": name, "op": "kv_gather", "n": n, "hk": hk, "d": d, "dtype": dtype,
            "cache": cache, "itype": itype, "page": page, "by_head": by_head, "pad": pad}


def listed():
    fwd, bwd = "qk_rope_fwd", "qk_rope_bwd"
    return [
        # one decoding step of 16 sequences whose cache is the caller's: latency counts
        _qk(fwd, "qk_rope_fwd_step", 16, 32, 8, 128, 128, "bf16", "i64"),
        # an odd batch of narrow heads, a part of each rotated, neighbours paired
        _qk(fwd, "qk_rope_fwd_odd", 4097, 12, 3, 96, 32, "f16", "i32", interleaved=True),
        # a training batch, or the prompts of a batch, with grouped heads
        _qk(fwd, "qk_rope_fwd_train", 32768, 64, 8, 128, 128, "bf16", "i64"),
        # one short sequence in full precision
        _qk(bwd, "qk_rope_bwd_small", 511, 12, 12, 64, 64, "f32", "i64"),
        # an odd batch at a head width that is no power of two
        _qk(bwd, "qk_rope_bwd_odd", 4097, 20, 5, 80, 80, "f16", "i32", interleaved=True),
        # the training batch's gradient
        _qk(bwd, "qk_rope_bwd_train", 32768, 64, 8, 128, 128, "bf16", "i64"),
        # a decoding step: one token a sequence, the batch padded to a captured size
        _slots("kv_slots_step", 61, 1, 4096, 16, "i32", pad=3),
        # whole prompts of a batch, or the slots of everything a batch has cached
        _slots("kv_slots_prompt", 255, 512, 0, 64, "i64"),
        # a decoding step of 64 sequences: queries, keys and values in one call
        _append("kv_append_step", 64, 32, 8, 128, 128, "bf16", "bf16", "i64", 16),
        # a batch of prompts into an 8-bit cache that holds its pages head by head
        _append("kv_append_prompt", 16384, 64, 8, 128, 128, "bf16", "e4m3", "i64", 64,
                by_head=True),
        # a short prefix at an odd head width, from pages of a few tokens
        _gather("kv_gather_odd", 1021, 5, 80, "f16", "f16", "i32", 7, pad=3),
        # the cached prefixes of a batch, from 8 bits
        _gather("kv_gather_prefix", 131072, 8, 128, "bf16", "e4m3", "i64", 64),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_rope_fwd", "qk_rope_bwd", "kv_slots", "kv_append", "kv_gather"])
    itype = rng.choice(["i32", "i64"])
    if op == "kv_slots":
        case = _slots("", _spread(rng, 1, 255), _spread(rng, 1, 512),
                      rng.choice([0, 100, 4096]), rng.choice([1, 7, 16, 64, 128]), itype,
                      rng.choice([0, 0, 1, 17]))
        del case["name"]
        return case
    dtype = rng.choice(["f32", "bf16", "f16"])
    d = rng.choice([32, 64, 80, 96, 112, 128, 128, 192, 256, 2 * rng.randint(8, 128)])
    rot = rng.choice([d, d, 2 * (d // 4), 2 * rng.randint(0, d // 2)])
    hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hq = hk * rng.choice([1, 1, 4, 5, 8])
    n = _spread(rng, 1, max(1, min(16384, (1 << 27) // ((hq + 2 * hk) * d))))
    interleaved = rng.random() < 0.4
    norm = rng.random() < 0.8
    if op.startswith("qk"):
        case = _qk(op, "", n, hq, hk, d, rot, dtype, itype, interleaved, norm)
    else:
        cache = rng.choice([dtype, dtype, "e4m3"])
        page = rng.choice([1, 7, 16, 64, 128])
        by_head = rng.random() < 0.4
        pad = rng.choice([0, 0, min(3, n - 1)])
        if op == "kv_append":
            case = _append("", n, rng.choice([0, hq, hq]), hk, d, rot, dtype, cache, itype, page,
                           by_head, interleaved, norm, pad)
        else:
            case = _gather("", n, hk, d, dtype, cache, itype, page, by_head, pad)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(shape, dtype, gen, std=1.0, mean=0.0):
    x = torch.empty(shape, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype,
                    device="cuda")
    return x.normal_(mean, std, generator=gen).to(dtype)


def _table(rot, count=32768):
    """[count, rot] in FP32: the cosines of rot / 2 angles a position, then the sines."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(count, device="cuda", dtype=torch.float64)[:, None] * \
        torch.exp(i * (-2.0 / max(rot, 1) * math.log(500000.0)))
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _positions(n, gen, itype):
    """Positions of n tokens of packed sequences, which begin at about every 700th."""
    at = torch.arange(n, device="cuda")
    begins = torch.rand(n, device="cuda", generator=gen) < 1 / 700
    first = torch.cummax(torch.where(begins, at, torch.zeros_like(at)), 0).values
    return (at - first + torch.randint(0, 4000, (1,), device="cuda", generator=gen)).to(itype)


def _heads(case, st, gen):
    """Queries, keys and values as column blocks of one matrix, and the norms' weights."""
    n, hq, hk, d = case["n"], case["hq"], case["hk"], case["d"]
    t = _DT[case["dtype"]]
    x = _normal((n, hq + 2 * hk, d), t, gen, 1.5)
    st["q"], st["k"], st["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    st["wq"] = _normal((d,), t, gen, 0.2, 1.0) if case["norm"] else None
    st["wk"] = _normal((d,), t, gen, 0.2, 1.0) if case["norm"] else None
    st["positions"] = _positions(n, gen, _IT[case["itype"]])
    st["table"] = _table(case["rot"])


def _cache(case, st, gen):
    """A cache of about twice the tokens' pages, full of other tokens, and the slots of
    the call's tokens: sequences' pages anywhere, each filled in order."""
    n, hk, d, page = case["n"], case["hk"], case["d"], case["page"]
    pages = 2 * (-(-n // page)) + 1
    for name in ("k_cache", "v_cache"):
        if case["by_head"]:
            st[name] = _normal((pages, hk, page, d), _DT[case["cache"]], gen).transpose(1, 2)
        else:
            st[name] = _normal((pages, page, hk, d), _DT[case["cache"]], gen)
    at = torch.arange(n, device="cuda")
    slots = torch.randperm(pages, device="cuda", generator=gen)[at // page] * page + at % page
    if case["pad"]:
        slots[n - case["pad"]:] = -1
    st["slots"] = slots.to(_IT[case["itype"]])
    eight = case["cache"] == "e4m3"
    st["k_scale"] = 0.03125 if eight else 1.0
    st["v_scale"] = float(np.float32(0.021)) if eight else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "kv_slots":
        seqs, page, it = case["seqs"], case["page"], _IT[case["itype"]]
        new = torch.randint(0, 2 * case["new"], (seqs,), device="cuda", generator=gen) \
            if case["new"] > 1 else torch.ones(seqs, dtype=torch.int64, device="cuda")
        ends = new.cumsum(0)
        n = seqs * case["new"]                 # what the batch holds: longer ones are cut
        ends = ends.clamp(max=n)
        st["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(it)
        starts = torch.randint(0, case["context"] + 1, (seqs,), device="cuda", generator=gen)
        st["starts"] = starts.to(it)
        width = -(-(case["context"] + 2 * case["new"]) // page)
        st["page_table"] = torch.randperm(seqs * width, device="cuda",
                                          generator=gen).view(seqs, width).to(it)
        st["n"] = n + case["pad"]
    elif op == "kv_gather":
        _cache(case, st, gen)
    else:
        _heads(case, st, gen)
        if op == "kv_append":
            _cache(case, st, gen)
        elif op == "qk_rope_bwd":
            t = _DT[case["dtype"]]
            st["dq_out"] = _normal((case["n"], case["hq"], case["d"]), t, gen, 0.02)
            st["dk_out"] = _normal((case["n"], case["hk"], case["d"]), t, gen, 0.02)
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _rotate(y, st, back=False):
    """The rotation of FP32 rows [n, heads, d], or its transpose."""
    rot = st["rot"]
    if rot == 0:
        return y
    row = st["table"][st["positions"].long()][:, None]
    c, s = row[..., :rot // 2], row[..., rot // 2:]
    if back:
        s = -s
    out = y.clone()
    if st["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2] = a * c - b * s
        out[..., 1:rot:2] = b * c + a * s
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2] = a * c - b * s
        out[..., rot // 2:rot] = b * c + a * s
    return out


def _norm_rotate(x, w, st):
    x = x.float()
    if st["norm"]:
        r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS)
        x = x * r * w.float()
    return _rotate(x, st)


def _plain_fwd(st):
    t = _DT[st["dtype"]]
    return {"q": _norm_rotate(st["q"], st["wq"], st).to(t),
            "k": _norm_rotate(st["k"], st["wk"], st).to(t)}


def _plain_bwd(st):
    t = _DT[st["dtype"]]
    out = {}
    for h in ("q", "k"):
        g = _rotate(st["d" + h + "_out"].float(), st, back=True)
        if st["norm"]:
            x, w = st[h].float(), st["w" + h].float()
            r = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS)
            x = x * r
            out["dw" + h] = (g * x).sum(dim=(0, 1)).to(t)
            g = g * w
            g = r * (g - x * (g * x).mean(dim=-1, keepdim=True))
        out["d" + h] = g.to(t)
    return out


def _plain_slots(st):
    n, page, it = st["n"], st["page"], _IT[st["itype"]]
    off, table = st["offsets"].long(), st["page_table"].long()
    at = torch.arange(n, device="cuda")
    b = (at[:, None] >= off[None, 1:]).sum(dim=1)      # ends at or before the token
    there = b < st["seqs"]
    b = b.clamp(max=st["seqs"] - 1)
    pos = st["starts"].long()[b] + at - off[b]
    col = torch.div(pos, page, rounding_mode="floor").clamp(max=table.shape[1] - 1)
    slot = table[b, col] * page + pos % page
    none = torch.full_like(pos, -1)
    return {"slots": torch.where(there, slot, none).to(it),
            "positions": torch.where(there, pos, none).to(it)}


def _stored(y, scale, cache):
    if cache == "e4m3":
        return (y / scale).clamp(-_E4M3_MAX, _E4M3_MAX).to(_DT[cache]).view(torch.uint8)
    return y.to(_DT[cache])


def _plain_append(st):
    n, page, cache = st["n"], st["page"], st["cache"]
    slots = st["slots"].long()
    # a token without a slot writes what the first token writes, once more
    src = torch.where(slots < 0, torch.zeros_like(slots), torch.arange(n, device="cuda"))
    slots = slots[src]
    at = (torch.div(slots, page, rounding_mode="floor"), slots % page)
    k = _stored(_norm_rotate(st["k"], st["wk"], st), st["k_scale"], cache)[src]
    v = _stored(st["v"].float(), st["v_scale"], cache)[src]
    st["k_cache"].view(k.dtype)[at] = k
    st["v_cache"].view(v.dtype)[at] = v
    out = {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if st["hq"]:
        out["q"] = _norm_rotate(st["q"], st["wq"], st).to(_DT[st["dtype"]])
    return out


def _plain_gather(st):
    page, t = st["page"], _DT[st["dtype"]]
    slots = st["slots"].long()
    there = (slots >= 0)[:, None, None]
    slots = slots.clamp(min=0)
    at = (torch.div(slots, page, rounding_mode="floor"), slots % page)
    out = {}
    for h in ("k", "v"):
        y = st[h + "_cache"]
        if st["cache"] == "e4m3":
            y = y.view(torch.uint8)[at].view(_DT["e4m3"]).float() * st[h + "_scale"]
        else:
            y = y[at].float()
        out[h] = torch.where(there, y, torch.zeros_like(y)).to(t)
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(st):
    import row_wise_normalization_gb300 as rn

    op = st["op"]
    if op == "qk_rope_fwd":
        q, k = rn.qk_rope_fwd(st["q"], st["k"], st["positions"], st["table"], st["wq"], st["wk"],
                              _EPS, interleaved=st["interleaved"])
        return {"q": q, "k": k}
    if op == "qk_rope_bwd":
        dq, dk, dwq, dwk = rn.qk_rope_bwd(st["dq_out"], st["dk_out"], st["q"], st["k"],
                                          st["positions"], st["table"], st["wq"], st["wk"], _EPS,
                                          interleaved=st["interleaved"])
        out = {"dq": dq, "dk": dk}
        if st["norm"]:
            out["dwq"], out["dwk"] = dwq, dwk
        return out
    if op == "kv_slots":
        slots, positions = rn.kv_slots(st["page_table"], st["starts"], st["offsets"], st["n"],
                                       st["page"])
        return {"slots": slots, "positions": positions}
    if op == "kv_append":
        q = rn.kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"],
                         st["positions"], st["table"], st["wk"], _EPS,
                         q=st["q"] if st["hq"] else None, wq=st["wq"] if st["hq"] else None,
                         interleaved=st["interleaved"], k_scale=st["k_scale"],
                         v_scale=st["v_scale"])
        out = {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        if st["hq"]:
            out["q"] = q
        return out
    k, v = rn.kv_gather(st["k_cache"], st["v_cache"], st["slots"], dtype=_DT[st["dtype"]],
                        k_scale=st["k_scale"], v_scale=st["v_scale"])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"qk_rope_fwd": _plain_fwd, "qk_rope_bwd": _plain_bwd, "kv_slots": _plain_slots,
            "kv_append": _plain_append, "kv_gather": _plain_gather}[state["op"]](state)


# ---------------------------------------------------------------------------
# bytes and operations no implementation can do without
# ---------------------------------------------------------------------------
def work(case):
    isz = 4 if case["itype"] == "i32" else 8
    op = case["op"]
    if op == "kv_slots":
        n, seqs = case["seqs"] * case["new"] + case["pad"], case["seqs"]
        pages = n // case["page"] + seqs            # entries of the page table in use
        return {"bytes": isz * (2 * n + 2 * seqs + 1 + pages), "flops": 6 * n}
    n, d, hk = case["n"], case["d"], case["hk"]
    es = _SIZE[case["dtype"]]
    if op == "kv_gather":
        return {"bytes": 2 * n * hk * d * (es + _SIZE[case["cache"]]) + n * isz,
                "flops": 2 * n * hk * d}
    hq, rot = case["hq"], case["rot"]
    # the table's rows of the positions that occur: packed sequences share them
    side = n * isz + min(n, 8000) * rot * 4
    row = (4 if case["norm"] else 0) * d + 3 * rot
    if op == "qk_rope_fwd":
        return {"bytes": 2 * n * (hq + hk) * d * es + side, "flops": n * (hq + hk) * row}
    if op == "qk_rope_bwd":
        passes = 3 if case["norm"] else 2
        return {"bytes": passes * n * (hq + hk) * d * es + side,
                "flops": n * (hq + hk) * ((11 if case["norm"] else 0) * d + 3 * rot)}
    cs = _SIZE[case["cache"]]
    return {"bytes": n * d * (2 * hq * es + 2 * hk * (es + cs)) + side + n * isz,
            "flops": n * ((hq + hk) * row + 2 * hk * d)}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _turn(st, a, b):
    """For tokens a .. b: (partner column of each column, cosines, signed sines) so that the
    rotation of y is y * c + y[partner] * s."""
    d, rot = st["d"], st["rot"]
    j = torch.arange(d, device="cuda")
    if st["interleaved"]:
        partner, pair, low = j ^ 1, j // 2, j % 2 == 0
    else:
        half = max(rot // 2, 1)
        low = j < half
        partner, pair = torch.where(low, j + half, j - half), j % half
    turned = j < rot
    partner = torch.where(turned, partner, j)
    c = torch.ones((b - a, d), dtype=torch.float64, device="cuda")
    s = torch.zeros((b - a, d), dtype=torch.float64, device="cuda")
    if rot:
        rows = st["table"][st["positions"][a:b].long()].double()
        c[:, :rot] = rows[:, pair[:rot]]
        s[:, :rot] = rows[:, rot // 2 + pair[:rot]]
        s = torch.where(low & turned, -s, s)
    return partner, c[:, None], s[:, None]


def _exact_rows(st, x, w, a, b):
    x = x[a:b].double()
    if st["norm"]:
        x = x / (x.square().mean(-1, keepdim=True) + _EPS).sqrt() * w.double()
    partner, c, s = _turn(st, a, b)
    return x * c + x[..., partner] * s


def _in_parts(st, fn):
    step = max(1, (1 << 25) // (max(st["hq"], st["hk"]) * st["d"]))
    return torch.cat([fn(a, min(st["n"], a + step)) for a in range(0, st["n"], step)])


def _exact_bwd(st, h):
    dw = torch.zeros(st["d"], dtype=torch.float64, device="cuda")

    def part(a, b):
        dy = st["d" + h + "_out"][a:b].double()
        partner, c, s = _turn(st, a, b)
        # y_j = n_j c_j + n_partner s_j: n_j is reached from y_j and from its partner's y
        g = dy * c + (dy * s)[..., partner]
        if not st["norm"]:
            return g
        x, w = st[h][a:b].double(), st["w" + h].double()
        ms = x.square().mean(-1, keepdim=True) + _EPS
        dw.add_((g * x / ms.sqrt()).sum((0, 1)))
        gw = g * w
        return gw / ms.sqrt() - x * (gw * x).sum(-1, keepdim=True) / (st["d"] * ms * ms.sqrt())

    return _in_parts(st, part), dw


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "kv_slots":
        off, starts = st["offsets"].tolist(), st["starts"].tolist()
        table, page = st["page_table"].cpu().numpy(), case["page"]
        slots = np.full(st["n"], -1, dtype=np.int64)
        pos = np.full(st["n"], -1, dtype=np.int64)
        for b in range(case["seqs"]):
            p = np.arange(off[b + 1] - off[b]) + starts[b]
            pos[off[b]:off[b + 1]] = p
            slots[off[b]:off[b + 1]] = table[b, p // page].astype(np.int64) * page + p % page
        it = _IT[case["itype"]]
        return {"slots": torch.from_numpy(slots).cuda().to(it),
                "positions": torch.from_numpy(pos).cuda().to(it)}
    if op == "qk_rope_fwd":
        return {h: _in_parts(st, lambda a, b: _exact_rows(st, st[h], st["w" + h], a, b))
                for h in ("q", "k")}
    if op == "qk_rope_bwd":
        out = {}
        for h in ("q", "k"):
            out["d" + h], dw = _exact_bwd(st, h)
            if case["norm"]:
                out["dw" + h] = dw
        return out
    slots, page = st["slots"].long(), case["page"]
    keep = slots >= 0
    # the cache as rows in the order of their slots
    rows = {h: st[h + "_cache"].double().reshape(-1, case["hk"], case["d"]) for h in ("k", "v")}
    if op == "kv_gather":
        out = {}
        for h in ("k", "v"):
            y = torch.zeros((case["n"], case["hk"], case["d"]), dtype=torch.float64,
                            device="cuda")
            y[keep] = rows[h][slots[keep]] * st[h + "_scale"]
            out[h] = y
        return out
    new = {"k": _in_parts(st, lambda a, b: _exact_rows(st, st["k"], st["wk"], a, b)),
           "v": st["v"].double()}
    out = {}
    for h in ("k", "v"):
        y = new[h][keep] / st[h + "_scale"]
        if case["cache"] == "e4m3":
            y = y.clamp(-_E4M3_MAX, _E4M3_MAX)
        rows[h][slots[keep]] = y
        out[h + "_cache"] = rows[h].view(-1, page, case["hk"], case["d"])
    if case["hq"]:
        out["q"] = _in_parts(st, lambda a, b: _exact_rows(st, st["q"], st["wq"], a, b))
    return out
