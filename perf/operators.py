"""What is measured of the token operators: embedding rows and their
gradient, and token log probabilities and their gradient.

``own`` says which side ``run`` takes: False computes the operators in their
plain form (elementary torch operations in 32 bits, rounded once at the end),
True makes the calls of this package. Both take what ``prepare`` made.

Ids follow a log-uniform law over a shuffled vocabulary (a few ids take much
of a batch, most occur once or never), which is what text does to an
embedding gradient. Logits are normal with a few units of spread.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_IT = {"i32": torch.int32, "i64": torch.int64}


def _f32(v):
    """The FP32 value nearest to v (a scale both sides read alike)."""
    return float(np.float32(v))


def _embed_fwd(name, n, vocab, d, dtype, itype, scale, pad=0.0):
    return {"name": name, "op": "embed_fwd", "n": n, "vocab": vocab, "d": d, "dtype": dtype,
            "itype": itype, "scale": _f32(scale), "pad": pad}


def _embed_bwd(name, n, vocab, d, dtype, grad, itype, scale, pad=0.0):
    """pad: the share of the batch that holds one and the same id."""
    return {"name": name, "op": "embed_bwd", "n": n, "vocab": vocab, "d": d, "dtype": dtype,
            "grad": grad, "itype": itype, "scale": _f32(scale), "pad": pad}


def _logprob_fwd(name, rows, vocab, dtype, itype, top, scale, entropy=True, masked=0.0, pad=0.0):
    """masked: the share of the vocabulary at -inf; pad: rows without a target."""
    return {"name": name, "op": "logprob_fwd", "rows": rows, "vocab": vocab, "dtype": dtype,
            "itype": itype, "top": top, "scale": _f32(scale), "entropy": entropy,
            "masked": masked, "pad": pad}


def _logprob_bwd(name, rows, vocab, dtype, itype, scale, entropy, masked=0.0, pad=0.0):
    return {"name": name, "op": "logprob_bwd", "rows": rows, "vocab": vocab, "dtype": dtype,
            "itype": itype, "scale": _f32(scale), "entropy": entropy, "masked": masked,
            "pad": pad}


def listed():
    return [
        # one decoding step of 16 sequences: latency is all that counts
        _embed_fwd("embed_fwd_step", 16, 32000, 4096, "bf16", "i64", 1.0),
        # an odd width: rows start at every 2-byte phase
        _embed_fwd("embed_fwd_odd", 4097, 50001, 771, "f16", "i32", math.sqrt(771)),
        # the prompts of a batch, or a training batch, at the widest rows
        _embed_fwd("embed_fwd_prompt", 32768, 128000, 8192, "bf16", "i64", math.sqrt(8192)),
        # one short sequence: the gradient's rows are nearly all zeros
        _embed_bwd("embed_bwd_small", 512, 32000, 768, "f32", "f32", "i64", 1.0),
        # a padded batch (a third of it one id) at an odd width, FP32 gradient of FP16 rows
        _embed_bwd("embed_bwd_batch", 16383, 50001, 771, "f16", "f32", "i32", math.sqrt(771),
                   pad=0.35),
        # a training batch over a large vocabulary
        _embed_bwd("embed_bwd_large", 65536, 128000, 4096, "bf16", "bf16", "i64", 1.0),
        # one token of one sequence, with its alternatives
        _logprob_fwd("logprob_fwd_step", 1, 128000, "f32", "i64", 5, 1.0),
        # a decoding step of 64 sequences over an odd vocabulary, a fifth of it masked off
        _logprob_fwd("logprob_fwd_serve", 64, 50001, "bf16", "i64", 20, 1.25, masked=0.2),
        # scoring of prompts, with alternatives for every token
        _logprob_fwd("logprob_fwd_score", 2048, 128000, "bf16", "i32", 8, 1.0, entropy=False),
        # a training batch: log probability and entropy, no alternatives
        _logprob_fwd("logprob_fwd_train", 8192, 128000, "bf16", "i64", 0, 1.0, pad=0.1),
        # a small padded batch over an odd vocabulary, log probability alone
        _logprob_bwd("logprob_bwd_small", 255, 50001, "f32", "i32", 0.8125, False, pad=0.25),
        # the training batch's gradient, of the log probability and the entropy
        _logprob_bwd("logprob_bwd_train", 8192, 128000, "bf16", "i64", 1.0, True, pad=0.1),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "logprob_fwd", "logprob_bwd"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    itype = rng.choice(["i32", "i64"])
    vocab = _spread(rng, 1000, 128000)
    if rng.random() < 0.5:
        vocab = max(1000, vocab // 64 * 64)
    if op.startswith("embed"):
        d = _spread(rng, 64, 8192 if op == "embed_fwd" else 4096)
        if rng.random() < 0.6:
            d = max(64, d // 16 * 16)
        n = _spread(rng, 1, 16384)
        scale = rng.choice([1.0, math.sqrt(d)])
        pad = rng.choice([0.0, 0.2, 0.6])
        if op == "embed_fwd":
            case = _embed_fwd("", n, vocab, d, dtype, itype, scale, pad)
        else:
            grad = rng.choice([dtype, "f32"])
            case = _embed_bwd("", n, vocab, d, dtype, grad, itype, scale, pad)
    else:
        rows = _spread(rng, 1, 2048)
        scale = rng.choice([1.0, 0.8125, 1.25])
        masked = rng.choice([0.0, 0.0, 0.3])
        pad = rng.choice([0.0, 0.1, 0.5])
        entropy = rng.random() < 0.5
        if op == "logprob_fwd":
            top = rng.choice([0, 1, 5, 20, 32])
            case = _logprob_fwd("", rows, vocab, dtype, itype, top, scale, entropy, masked, pad)
        else:
            case = _logprob_bwd("", rows, vocab, dtype, itype, scale, entropy, masked, pad)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ids(case, n, gen, pad, pad_id):
    """n ids of a log-uniform law over a shuffled vocabulary, a share `pad` of
    them replaced by pad_id."""
    vocab = case["vocab"]
    u = torch.rand(n, device="cuda", generator=gen, dtype=torch.float64)
    t = torch.exp(u * math.log(vocab + 1.0)).long().sub_(1).clamp_(0, vocab - 1)
    t = torch.randperm(vocab, device="cuda", generator=gen)[t]
    if pad > 0:
        t[torch.rand(n, device="cuda", generator=gen) < pad] = pad_id
    return t.to(_IT[case["itype"]])


def _normal(shape, dtype, gen, std):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    return x.normal_(0.0, std, generator=gen)


def _logits(case, gen):
    rows, vocab = case["rows"], case["vocab"]
    x = _normal((rows, vocab), _DT[case["dtype"]], gen, 2.5)
    if case["masked"] > 0:
        off = torch.rand(vocab, device="cuda", generator=gen) < case["masked"]
        x[:, off] = float("-inf")
    t = _ids(case, rows, gen, case["pad"], -100)
    return x, t


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op == "embed_fwd":
        st["tokens"] = _ids(case, case["n"], gen, case["pad"], 0)
        st["table"] = _normal((case["vocab"], case["d"]), _DT[case["dtype"]], gen, 0.02)
    elif op == "embed_bwd":
        st["tokens"] = _ids(case, case["n"], gen, case["pad"], 0)
        st["dout"] = _normal((case["n"], case["d"]), _DT[case["dtype"]], gen, 0.02)
    elif op == "logprob_fwd":
        st["logits"], st["targets"] = _logits(case, gen)
    else:
        st["logits"], st["targets"] = _logits(case, gen)
        # what the forward pass left, and the gradients that reach it
        lse, ent = [], []
        for x in st["logits"].split(512):
            x = x.float() * case["scale"]
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            lse.append(z)
            ent.append(torch.where(p > 0, p * (z[:, None] - x), torch.zeros_like(p)).sum(1))
        st["lse"] = torch.cat(lse)
        st["ent"] = torch.cat(ent)
        rows = case["rows"]
        st["dlogp"] = _normal((rows,), torch.float32, gen, 1.0)
        st["dentropy"] = _normal((rows,), torch.float32, gen, 0.1) if case["entropy"] else None
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_embed_fwd(st):
    t = st["tokens"].long()
    there = (t >= 0) & (t < st["vocab"])
    y = st["table"][t.clamp(0, st["vocab"] - 1)].float() * st["scale"]
    y = torch.where(there[:, None], y, torch.zeros_like(y))
    return y.to(_DT[st["dtype"]])


def _plain_embed_bwd(st):
    t = st["tokens"].long()
    there = (t >= 0) & (t < st["vocab"])
    g = torch.where(there[:, None], st["dout"].float(), torch.zeros((), device="cuda"))
    acc = torch.zeros((st["vocab"], st["d"]), dtype=torch.float32, device="cuda")
    acc.index_add_(0, t.clamp(0, st["vocab"] - 1), g)
    return (acc * st["scale"]).to(_DT[st["grad"]])


def _plain_logprob_fwd(st):
    raw = st["logits"].float()
    x = raw * st["scale"]
    m = x.max(dim=1, keepdim=True).values
    empty = m == float("-inf")
    z = x - torch.where(empty, torch.zeros_like(m), m)
    e = torch.exp(z)
    s = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(s)
    t = st["targets"].long()
    there = (t >= 0) & (t < st["vocab"])
    xt = x.gather(1, t.clamp(0, st["vocab"] - 1)[:, None])
    lp = torch.where(empty, m, xt - lse)[:, 0]
    out = {"logp": torch.where(there, lp, torch.zeros_like(lp)), "lse": lse[:, 0]}
    if st["entropy"]:
        w = torch.where(e > 0, e * z, torch.zeros_like(e)).sum(dim=1, keepdim=True)
        h = torch.log(s) - w / s
        out["entropy"] = torch.where(empty, torch.zeros_like(h), h)[:, 0]
    if st["top"]:
        # one whole number that orders values first and, among equal ones, the
        # lowest index first (adding zero makes -0.0 equal to 0.0)
        bits = (raw + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        last = st["vocab"] - 1
        key = (order << 32) + (last - torch.arange(st["vocab"], device="cuda"))
        ids = last - (torch.topk(key, st["top"], dim=1).values & 0xFFFFFFFF)
        out["top_ids"] = ids.to(_IT[st["itype"]])
        out["top_logp"] = torch.where(empty, m, x.gather(1, ids) - lse)
    return out


def _plain_logprob_bwd(st):
    x = st["logits"].float() * st["scale"]
    t = st["targets"].long()
    there = (t >= 0) & (t < st["vocab"])
    lse = st["lse"][:, None]
    g = torch.where(there, st["dlogp"], torch.zeros_like(st["dlogp"]))[:, None]
    z = x - lse
    p = torch.exp(z)
    d = -g * p
    if st["dentropy"] is not None:
        u = torch.where(p > 0, p * (z + st["ent"][:, None]), torch.zeros_like(p))
        d = d - st["dentropy"][:, None] * u
    d.scatter_add_(1, t.clamp(0, st["vocab"] - 1)[:, None], g)
    return (d * st["scale"]).to(_DT[st["dtype"]])


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(st):
    import row_wise_normalization_gb300 as rn

    op = st["op"]
    if op == "embed_fwd":
        return rn.embed_fwd(st["tokens"], st["table"], st["scale"])
    if op == "embed_bwd":
        return rn.embed_bwd(st["dout"], st["tokens"], st["vocab"], st["scale"],
                            dtype=_DT[st["grad"]])
    if op == "logprob_fwd":
        logp, entropy, lse, ids, top = rn.logprob_fwd(st["logits"], st["targets"], st["scale"],
                                                      top=st["top"],
                                                      want_entropy=st["entropy"])
        out = {"logp": logp, "lse": lse}
        if st["entropy"]:
            out["entropy"] = entropy
        if st["top"]:
            out["top_ids"] = ids
            out["top_logp"] = top
        return out
    return rn.logprob_bwd(st["dlogp"], st["logits"], st["targets"], st["lse"], st["scale"],
                          dentropy=st["dentropy"],
                          entropy=st["ent"] if st["dentropy"] is not None else None)


def run(state):
    if own:
        return _own(state)
    return {"embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd,
            "logprob_fwd": _plain_logprob_fwd, "logprob_bwd": _plain_logprob_bwd}[
                state["op"]](state)


# ---------------------------------------------------------------------------
# bytes and operations no implementation can do without
# ---------------------------------------------------------------------------
def _distinct(n, vocab, pad):
    """Expected number of different ids among n draws."""
    n = n * (1.0 - pad)
    v = np.arange(1, vocab + 1, dtype=np.float64)
    p = np.log((v + 1.0) / v) / math.log(vocab + 1.0)
    return float(-np.expm1(n * np.log1p(-np.minimum(p, 1 - 1e-12))).sum()) + (1 if pad else 0)


def work(case):
    es = _SIZE[case["dtype"]]
    isz = 4 if case["itype"] == "i32" else 8
    if case["op"] == "embed_fwd":
        n, d = case["n"], case["d"]
        rows = min(_distinct(n, case["vocab"], case["pad"]), n)
        return {"bytes": int(rows * d * es + n * d * es + n * isz), "flops": n * d}
    if case["op"] == "embed_bwd":
        n, d, vocab = case["n"], case["d"], case["vocab"]
        return {"bytes": int(n * d * es + n * isz + vocab * d * _SIZE[case["grad"]]),
                "flops": 2 * n * d}
    rows, vocab = case["rows"], case["vocab"]
    if case["op"] == "logprob_fwd":
        out = 4 * (2 + (1 if case["entropy"] else 0)) + case["top"] * (4 + isz)
        # subtract, scale, exponential, sum; the entropy's product and sum; the
        # comparison that finds alternatives
        per = 4 + (2 if case["entropy"] else 0) + (1 if case["top"] else 0)
        return {"bytes": rows * vocab * es + rows * (isz + out), "flops": rows * vocab * per}
    per = 4 + (3 if case["entropy"] else 0)
    live = rows if case["entropy"] else int(rows * (1.0 - case["pad"]))
    return {"bytes": (live + rows) * vocab * es + rows * (isz + 8 + (8 if case["entropy"] else 0)),
            "flops": live * vocab * per}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op, scale = case["op"], case["scale"]
    if op == "embed_fwd":
        w = torch.cat([st["table"], st["table"].new_zeros((1, case["d"]))])
        t = st["tokens"].long()
        t[(t < 0) | (t >= case["vocab"])] = case["vocab"]     # the row of zeros
        return torch.index_select(w, 0, t).double().mul_(scale)
    if op == "embed_bwd":
        # ids in order, their rows' running sums cut where the id changes
        t, order = torch.sort(st["tokens"].long(), stable=True)
        keep = (t >= 0) & (t < case["vocab"])
        t, order = t[keep], order[keep]
        out = torch.zeros((case["vocab"], case["d"]), dtype=torch.float64, device="cuda")
        ids, counts = torch.unique_consecutive(t, return_counts=True)
        ends = counts.cumsum(0)
        for j in range(0, case["d"], 512):
            run_ = st["dout"][order, j:j + 512].double().cumsum(0)
            at = run_[ends - 1]
            at[1:] -= run_[ends[:-1] - 1]
            out[ids, j:j + 512] = at
        return out.mul_(scale)
    parts = []
    step = max(1, (1 << 27) // case["vocab"])
    rows = case["rows"]
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = st["logits"][a:b].double()
        t = st["targets"][a:b].long()
        col = torch.arange(case["vocab"], device="cuda")
        hit = col[None, :] == t[:, None]          # no column where there is no target
        if op == "logprob_fwd":
            lse = torch.logsumexp(x * scale, dim=1)
            lq = x * scale - lse[:, None]
            lq = torch.where(torch.isinf(lse)[:, None], torch.full_like(lq, -math.inf), lq)
            o = {"logp": torch.where(hit, lq, torch.zeros_like(lq)).sum(1), "lse": lse}
            if case["entropy"]:
                o["entropy"] = -(torch.xlogy(lq.exp(), lq.exp())).sum(1)
            if case["top"]:
                ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
                o["top_ids"] = ids.to(_IT[case["itype"]])
                o["top_logp"] = lq.gather(1, ids)
            parts.append(o)
        else:
            # the gradient through the softmax: s * (v - q * sum(v)), where v
            # is the gradient of each log probability
            lq = x * scale - st["lse"][a:b].double()[:, None]
            q = lq.exp()
            v = hit * st["dlogp"][a:b].double()[:, None]
            d = v - q * v.sum(1, keepdim=True)
            if case["entropy"]:
                h = st["ent"][a:b].double()[:, None]
                d = d - st["dentropy"][a:b].double()[:, None] * (torch.xlogy(q, q) + q * h)
            parts.append(d * scale)
    if op == "logprob_bwd":
        return torch.cat(parts)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}
