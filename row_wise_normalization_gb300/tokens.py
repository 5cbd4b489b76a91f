"""The token operators: embedding rows and their gradient, log probabilities and
their gradient (torch binding; the C entry points are in include/rownorm.h).

A decoding step waits for the host side of these calls, not for their kernels
(a few microseconds each), so the checks take the common case (contiguous CUDA
tensors on the current device) by a few lookups and leave the rest to the package's
general ones.
"""
from __future__ import annotations

from functools import partial

import torch

from . import _check_f32_cuda, _empty_like_home, _rows_of, capi

_FLOATS = {torch.float32: capi.RN_DTYPE_F32, torch.bfloat16: capi.RN_DTYPE_BF16,
           torch.float16: capi.RN_DTYPE_F16}
_INDEX = {torch.int32: capi.RN_INDEX_I32, torch.int64: capi.RN_INDEX_I64}
_F32 = torch.float32


class _Unloaded:
    """Loads the library at the first call, and stands aside."""

    def __getattr__(self, name):
        global _C
        _C = capi.load()
        return getattr(_C, name)


_C = _Unloaded()


def _values(name, t):
    """Storage code of a floating-point tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _FLOATS.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name} (float32, bfloat16 or float16)")
    return code


def _ids(name, t):
    """Index code of a contiguous tensor of ids."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _INDEX.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")
    if not (t.is_cuda and t.is_contiguous()):
        _check_f32_cuda(name, t, t.dtype)
    return code


def _stride(name, t, d, dtype):
    """Row stride of a matrix of rows of d: contiguous of any shape, or a 2-D
    row-strided view."""
    if t.is_cuda and t.dtype is dtype and t.is_contiguous():
        return d
    _check_f32_cuda(name, t, dtype, contiguous=False)
    return _rows_of(name, t, d)[1]


def _row_floats(name, t, rows):
    """Address of an FP32 vector of a value a row (0 for None)."""
    if t is None:
        return 0
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is _F32 and t.is_contiguous()):
        _check_f32_cuda(name, t)
    if t.numel() != rows:
        raise ValueError(f"{name} must have {rows} elements")
    return t.data_ptr()


def _device(*tensors):
    """Index of the one device of a call's CUDA tensors, -1 where all of them
    are in host memory."""
    dev = -1
    for t in tensors:
        if t is not None:
            i = t.get_device()
            if i != dev and i >= 0:
                if dev >= 0:
                    raise ValueError(f"tensors on cuda:{dev} and on cuda:{i}")
                dev = i
    return dev


def _elsewhere(dev, stream):
    """Whether the call needs another device or stream made current first."""
    return stream is not None or (dev >= 0 and dev != torch._C._cuda_getDevice())


class _On:
    """Makes the call's device current and, where the caller gives a stream of
    its own, that stream too, so that the memory the call allocates belongs to the
    stream that uses it."""

    def __init__(self, dev, stream):
        at = torch.device("cuda", dev) if dev >= 0 else None
        if isinstance(stream, int):
            # (handle 0: the legacy default stream, torch's default stream)
            stream = (torch.cuda.ExternalStream(stream, device=at) if stream
                      else torch.cuda.default_stream(at))
        elif stream is not None and at is not None and stream.device != at:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to {at}")
        self._inner = [torch.cuda.stream(stream)]
        if at is not None:
            self._inner.insert(0, torch.cuda.device(at))

    def __enter__(self):
        for c in self._inner:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._inner):
            c.__exit__(*exc)


def _stream(dev):
    """Handle of the current stream of the call's device (of the current device,
    where every tensor is in host memory)."""
    return (torch._C._cuda_getCurrentRawStream(dev) if dev >= 0
            else torch.cuda.current_stream().cuda_stream)


def _maker(home, dev):
    """What allocates a call's outputs, given their shape and dtype: on the call's device,
    or in host memory like `home`."""
    if home.is_cuda:
        return partial(torch.empty, device=home.device)
    if dev >= 0:
        return partial(torch.empty, device=torch.device("cuda", dev))
    return partial(_empty_like_home, home)


def embed_fwd(tokens, table, scale: float = 1.0, *, out=None, stream=None):
    """Embedding rows ``scale * table[tokens]``.

    tokens: int32 or int64 ids of any shape; an id outside ``[0, vocab)`` gives a
    row of zeros. table: ``[vocab, d]``, float32, bfloat16 or float16, contiguous
    or a row-strided view. Returns ``out`` of shape ``tokens.shape + (d,)`` in the
    table's type (``out`` may also be passed as a 2-D row-strided view).
    """
    code = _values("table", table)
    it = _ids("tokens", tokens)
    if table.dim() != 2:
        raise ValueError("table must be 2-D")
    vocab, d = table.shape
    dtype = table.dtype
    ldt = _stride("table", table, d, dtype)
    dev = _device(table, tokens, out)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return embed_fwd(tokens, table, scale, out=out)
    n = tokens.numel()
    if out is None:
        out, ldo = _maker(table, dev)((*tokens.shape, d), dtype=dtype), d
    else:
        if out.numel() != n * d or out.shape[-1:] != (d,):
            raise ValueError(f"out must hold {n} rows of {d}")
        ldo = _stride("out", out, d, dtype)
    st = _C.embed_fwd(code, it, tokens.data_ptr(), table.data_ptr(), ldt, out.data_ptr(), ldo, n,
                      int(vocab), d, float(scale), _stream(dev))
    if st:
        capi.check(st)
    return out


def embed_bwd(dout, tokens, vocab: int, scale: float = 1.0, *, dtype=None, dtable=None,
              accumulate: bool = False, workspace=None, stream=None):
    """Gradient of ``embed_fwd`` with respect to the table.

    dout: the rows' gradient, shape ``tokens.shape + (d,)`` (or a 2-D row-strided
    view). Returns ``dtable`` of shape ``[vocab, d]`` in ``dtype`` (dout's type
    unless given; float32 is the other choice), every row written; with
    ``accumulate`` the sums are added to the ``dtable`` passed in.
    ``workspace``: a contiguous CUDA tensor of at least
    ``capi.embed_bwd_workspace_size(n, vocab, d)`` bytes (allocated if not given).
    """
    code = _values("dout", dout)
    it = _ids("tokens", tokens)
    n = tokens.numel()
    if dout.dim() < 1:
        raise ValueError("dout must have a last dimension")
    d = dout.shape[-1]
    if dout.numel() != n * d:
        raise ValueError(f"dout must hold {n} rows of {d}")
    lddo = _stride("dout", dout, d, dout.dtype)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs a dtable to add to")
        gdtype = dout.dtype if dtype is None else dtype
    else:
        gdtype = dtable.dtype
        if dtype is not None and dtype != gdtype:
            raise TypeError(f"dtable is {gdtype}, dtype says {dtype}")
    if gdtype is not dout.dtype and gdtype is not _F32:
        raise TypeError(f"dtable must be {dout.dtype} or float32")
    dev = _device(dout, tokens, dtable, workspace)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return embed_bwd(dout, tokens, vocab, scale, dtype=dtype, dtable=dtable,
                             accumulate=accumulate, workspace=workspace)
    if dtable is None:
        dtable, ldg = _maker(dout, dev)((vocab, d), dtype=gdtype), d
    else:
        if tuple(dtable.shape) != (vocab, d):
            raise ValueError(f"dtable must be of shape [{vocab}, {d}]")
        ldg = _stride("dtable", dtable, d, gdtype)
    if workspace is None:
        nbytes = capi.embed_bwd_workspace_size(n, vocab, d)
        workspace = torch.empty(nbytes, dtype=torch.uint8,
                                device=dtable.device if dtable.is_cuda else "cuda")
    else:
        if not (workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor")
        nbytes = workspace.numel() * workspace.element_size()
    st = _C.embed_bwd(code, _FLOATS[gdtype], it, dout.data_ptr(), lddo, tokens.data_ptr(),
                      dtable.data_ptr(), ldg, n, int(vocab), d, float(scale), 1 if accumulate else
                      0, workspace.data_ptr(), nbytes, _stream(dev))
    if st:
        capi.check(st)
    return dtable


def logprob_fwd(logits, targets=None, scale: float = 1.0, *, top: int = 0,
                want_entropy: bool = True, stream=None):
    """Log probabilities over the last dimension of ``logits`` times ``scale`` (the
    inverse temperature).

    logits: float32, bfloat16 or float16, contiguous or a 2-D row-strided view.
    targets: int32 or int64 columns of shape ``logits.shape[:-1]``; one outside
    ``[0, vocab)`` gets 0. Returns ``(logp, entropy, lse, top_ids, top_logp)``:
    the targets' log probabilities (None without targets), the entropies (None
    without ``want_entropy``), the log-sum-exps, and the ``top`` (at most 32)
    largest columns with their log probabilities, shape ``[..., top]``, largest
    first and the lowest column first among equal ones (None with ``top`` 0).
    Values are float32; top_ids has targets' type (int64 without targets).
    """
    code = _values("logits", logits)
    lead = logits.shape
    if not lead:
        raise ValueError("logits must have a last dimension")
    vocab, lead = lead[-1], lead[:-1]
    ldl = _stride("logits", logits, vocab, logits.dtype)
    rows = lead.numel()
    it, itype, tgt = capi.RN_INDEX_I64, torch.int64, 0
    if targets is not None:
        it, itype, tgt = _ids("targets", targets), targets.dtype, targets.data_ptr()
        if targets.numel() != rows:
            raise ValueError(f"targets must have {rows} elements")
    dev = _device(logits, targets)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return logprob_fwd(logits, targets, scale, top=top, want_entropy=want_entropy)
    new = _maker(logits, dev)
    logp = entropy = ids = top_logp = None
    a_logp = a_entropy = a_ids = a_top = 0
    if targets is not None:
        logp = new(lead, dtype=_F32)
        a_logp = logp.data_ptr()
    if want_entropy:
        entropy = new(lead, dtype=_F32)
        a_entropy = entropy.data_ptr()
    lse = new(lead, dtype=_F32)
    if top > 0:
        lead = (*lead, top)
        ids = new(lead, dtype=itype)
        top_logp = new(lead, dtype=_F32)
        a_ids, a_top = ids.data_ptr(), top_logp.data_ptr()
    st = _C.logprob_fwd(code, it, logits.data_ptr(), ldl, tgt, a_logp, a_entropy, lse.data_ptr(),
                        a_ids, a_top, rows, vocab, int(top), float(scale), _stream(dev))
    if st:
        capi.check(st)
    return logp, entropy, lse, ids, top_logp


def logprob_bwd(dlogp, logits, targets, lse, scale: float = 1.0, *, dentropy=None, entropy=None,
                dlogits=None, stream=None):
    """Gradient of ``logprob_fwd``'s log probabilities (dlogp) and, where
    ``dentropy`` is given with the forward call's ``entropy``, of its entropies,
    with respect to the logits. dlogp may be None (then targets too). ``dlogits``:
    allocated in the logits' type unless given; it may be ``logits`` itself.
    """
    code = _values("logits", logits)
    shape = logits.shape
    if not shape:
        raise ValueError("logits must have a last dimension")
    vocab = shape[-1]
    ldl = _stride("logits", logits, vocab, logits.dtype)
    rows = shape[:-1].numel()
    it, tgt = capi.RN_INDEX_I64, 0
    if targets is not None:
        it, tgt = _ids("targets", targets), targets.data_ptr()
        if targets.numel() != rows:
            raise ValueError(f"targets must have {rows} elements")
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    a_dlogp = _row_floats("dlogp", dlogp, rows)
    a_dentropy = _row_floats("dentropy", dentropy, rows)
    a_lse = _row_floats("lse", lse, rows)
    a_entropy = _row_floats("entropy", entropy, rows)
    dev = _device(logits, dlogp, targets, lse, dentropy, entropy, dlogits)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return logprob_bwd(dlogp, logits, targets, lse, scale, dentropy=dentropy,
                               entropy=entropy, dlogits=dlogits)
    if dlogits is None:
        dlogits, ldd = _maker(logits, dev)(shape, dtype=logits.dtype), vocab
    else:
        if dlogits.shape != shape:
            raise ValueError("dlogits must be shaped like logits")
        ldd = _stride("dlogits", dlogits, vocab, logits.dtype)
    st = _C.logprob_bwd(code, it, a_dlogp, a_dentropy, logits.data_ptr(), ldl, tgt, a_lse,
                        a_entropy, dlogits.data_ptr(), ldd, rows, vocab, float(scale), _stream(dev))
    if st:
        capi.check(st)
    return dlogits
