"""The token operators (embedding rows and their gradient, log probabilities and their
gradient) and the head operators (norms of queries and keys with the position rotation, their
gradient, a paged cache of keys and values): torch binding; the C entry points are in
include/rownorm.h.

A decoding step waits for the host side of these calls, not for their kernels
(a few microseconds each), so the checks take the common case (contiguous CUDA
tensors on the current device) by a few lookups and leave the rest to the package's
general ones.
"""
from __future__ import annotations

import ctypes
from functools import partial

import torch

from . import _check_f32_cuda, _empty_like_home, _rows_of, capi

_FLOATS = {torch.float32: capi.RN_DTYPE_F32, torch.bfloat16: capi.RN_DTYPE_BF16,
           torch.float16: capi.RN_DTYPE_F16}
_INDEX = {torch.int32: capi.RN_INDEX_I32, torch.int64: capi.RN_INDEX_I64}
_F32 = torch.float32
_E4M3 = torch.float8_e4m3fn


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


# ---------------------------------------------------------------------------
# The head operators. Rows are heads of tokens: tensors of shape [tokens, heads, d] or
# [batch, len, heads, d] with contiguous rows and any other strides (column blocks of a packed
# projection, transposed head-major tensors). A tensor's rows go to the library as its address,
# heads, and batch, token and head strides. Plain calls are made by the native module (see _Unfound);
# what follows each of those is the general way: outputs passed in, host memory, another device or
# stream, and what is wrong with a call.
# ---------------------------------------------------------------------------
class _InPython:
    """Takes no call: each goes the way below, in Python."""

    def _none(self, *args):
        return None

    qk_rope_fwd = qk_rope_bwd = kv_append = kv_gather = kv_slots = _none


class _Unfound:
    """Finds the native module that marshals plain calls (csrc/binding.cpp), at the first one,
    and stands aside for it. Its functions take a call whole and return its outputs as a
    tuple, or None for one that is not plain, which the functions here then check and make."""

    def __getattr__(self, name):
        global _B
        lib = capi.load()
        _B = _InPython()
        try:
            from . import _binding
        except ImportError:
            pass
        else:
            # (made for this PyTorch: another's objects are laid out differently)
            if torch.__version__.split("+")[0] == _binding.torch_version:
                _binding.use(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in
                               ("qk_rope_fwd", "qk_rope_bwd", "qk_rope_bwd_workspace_size",
                                "kv_append", "kv_gather", "kv_slots")))
                _B = _binding
        return getattr(_B, name)


_B = _Unfound()
_NO_ROWS = (0, 0, 0, 0, 0)
_heads, _qk, _empty = capi.heads, capi.qk, torch.empty
_NONE = _heads(*_NO_ROWS)


def _tensors(**named):
    """Tensors, or None for what is not given."""
    for name, t in named.items():
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _rows(name, t, want, dtype):
    """A tensor's rows; its shape and dtype have to be as given."""
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != want:
        raise ValueError(f"{name} must be of shape {list(want)}, got {list(t.shape)}")
    if not t.is_cuda or t.dtype is not dtype:
        _check_f32_cuda(name, t, dtype, contiguous=False)
    if len(want) == 3:
        ts, hs, one = t.stride()
        bs = 0
    else:
        bs, ts, hs, one = t.stride()
    if one != 1 and t.numel():
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), want[-2], bs, ts, hs


def _new_rows(home, shape, dtype, dev):
    """(tensor, packed rows) of an output that the call allocates, contiguous."""
    t = (_empty(shape, dtype=dtype, device=home.device) if home.is_cuda else
         _maker(home, dev)(shape, dtype=dtype))
    h, d = shape[-2:]
    return t, _heads(t.data_ptr(), h, shape[1] * h * d if len(shape) == 4 else 0, h * d, d)


def _first(name, t):
    """Storage code and shape of the tensor that sets them."""
    code = _values(name, t)
    shape = t.shape
    if len(shape) != 3 and len(shape) != 4:
        raise ValueError(f"{name} must be [tokens, heads, d] or [batch, len, heads, d]")
    return code, shape


def _beside(name, t, shape):
    """The shape that a tensor of other heads of the same tokens has to have."""
    heads = t.shape[-2] if t.dim() > 1 else -1
    return ((shape[0], heads, shape[2]) if len(shape) == 3 else
            (shape[0], shape[1], heads, shape[3]))


def _weight(name, w, d, dtype):
    if w is None:
        return 0
    if not (isinstance(w, torch.Tensor) and w.is_cuda and w.dtype is dtype and w.is_contiguous()):
        _check_f32_cuda(name, w, dtype)
    if w.numel() != d:
        raise ValueError(f"{name} must have {d} elements")
    return w.data_ptr()


def _turn(positions, table, n):
    """(address of positions, of table, rows, stride, rot, index code)."""
    if table is None:
        return 0, 0, 0, 0, 0, 0
    if not (isinstance(table, torch.Tensor) and table.is_cuda and table.dtype is _F32):
        _check_f32_cuda("table", table, _F32, contiguous=False)
    shape = table.shape
    if len(shape) != 2 or table.stride(1) != 1:
        raise ValueError("table must be 2-D with contiguous rows")
    rows, rot = shape
    if rot == 0:
        return 0, 0, 0, 0, 0, 0
    it = _ids("positions", positions)
    if positions.numel() != n:
        raise ValueError(f"positions must have {n} elements")
    return (positions.data_ptr(), table.data_ptr(), rows, table.stride(0) if rows > 1 else rot,
            rot, it)


def qk_rope_fwd(q, k, positions=None, table=None, wq=None, wk=None, eps: float = 1e-5, *,
                norm=None, interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Queries and keys, each head normed (RMS) and turned by its token's position.

    q, k: ``[tokens, heads, d]`` or ``[batch, len, heads, d]`` (float32, bfloat16 or
    float16, one type; d even, at most 512); k may be None. table: float32 ``[positions,
    rot]``, a row the cosines of rot / 2 angles, then their sines; the first ``rot`` values
    of a row are turned, in pairs (i, i + rot / 2) or, with ``interleaved``, (2i, 2i + 1).
    positions: int32 or int64, one a token; a token whose position is outside the table gets
    rows of zeros. Without a table nothing is turned. wq, wk: ``[d]``, the norms' weights;
    unless ``norm`` says so, rows are normed if one of them is given. Returns ``(q_out, k_out)``
    (allocated contiguous unless given; each may be its input itself).
    """
    if q_out is None and k_out is None and stream is None:
        out = _B.qk_rope_fwd(q, k, positions, table, wq, wk, eps, norm, interleaved)
        if out is not None:
            return out
    _tensors(q=q, k=k, positions=positions, table=table, wq=wq, wk=wk, q_out=q_out, k_out=k_out)
    code, shape = _first("q", q)
    dtype, d, len_ = q.dtype, shape[-1], shape[-3]
    batch = 1 if len(shape) == 3 else shape[0]
    if norm is None:
        norm = wq is not None or wk is not None
    pos, tab, trows, tstride, rot, it = _turn(positions, table, batch * len_)
    dev = _device(q, k, positions, table, wq, wk, q_out, k_out)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return qk_rope_fwd(q, k, positions, table, wq, wk, eps, norm=norm,
                               interleaved=interleaved, q_out=q_out, k_out=k_out)
    r_q = _rows("q", q, shape, dtype)
    if q_out is None:
        q_out, p_q = _new_rows(q, shape, dtype, dev)
    else:
        p_q = _heads(*_rows("q_out", q_out, shape, dtype))
    r_k, p_k = _NO_ROWS, _NONE
    if k is not None:
        kshape = _beside("k", k, shape)
        r_k = _rows("k", k, kshape, dtype)
        if k_out is None:
            k_out, p_k = _new_rows(k, kshape, dtype, dev)
        else:
            p_k = _heads(*_rows("k_out", k_out, kshape, dtype))
    elif k_out is not None:
        raise ValueError("k_out without k")
    st = _C.qk_rope_fwd(
        _qk(*r_q, *r_k, _weight("wq", wq, d, dtype), _weight("wk", wk, d, dtype), pos, tab, trows,
            tstride, rot, batch, len_, d, code, it, 1 if norm else 0, 1 if interleaved else 0, eps,
            0), p_q, p_k, _stream(dev))
    if st:
        capi.check(st)
    return q_out, k_out


_BWD_BYTES = {}      # workspace of qk_rope_bwd by width


def qk_rope_bwd(dq_out, dk_out, q, k, positions=None, table=None, wq=None, wk=None,
                eps: float = 1e-5, *, norm=None, interleaved: bool = False,
                param_grads: bool = True, dq=None, dk=None, dwq=None, dwk=None, workspace=None,
                stream=None):
    """Gradient of ``qk_rope_fwd``: dq_out and dk_out are what reaches its outputs, the other
    arguments are as there (without a norm q and k may be None). Returns ``(dq, dk, dwq,
    dwk)`` in the inputs' type, dk None without dk_out, dwq and dwk None without their weights
    or without ``param_grads``. dq and dk may be passed in, dq_out and dk_out (or q and k)
    themselves among them. ``workspace``: a contiguous CUDA tensor of at least
    ``capi.qk_rope_bwd_workspace_size(d)`` bytes (allocated if not given).
    """
    if (dq is None and dk is None and dwq is None and dwk is None and workspace is None
            and stream is None):
        out = _B.qk_rope_bwd(dq_out, dk_out, q, k, positions, table, wq, wk, eps, norm,
                             interleaved, param_grads)
        if out is not None:
            return out
    _tensors(dq_out=dq_out, dk_out=dk_out, q=q, k=k, positions=positions, table=table, wq=wq,
             wk=wk, dq=dq, dk=dk, dwq=dwq, dwk=dwk, workspace=workspace)
    code, shape = _first("dq_out", dq_out)
    dtype, d, len_ = dq_out.dtype, shape[-1], shape[-3]
    batch = 1 if len(shape) == 3 else shape[0]
    if norm is None:
        norm = wq is not None or wk is not None
    pos, tab, trows, tstride, rot, it = _turn(positions, table, batch * len_)
    dev = _device(dq_out, dk_out, q, k, positions, table, wq, wk, dq, dk, dwq, dwk, workspace)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return qk_rope_bwd(dq_out, dk_out, q, k, positions, table, wq, wk, eps, norm=norm,
                               interleaved=interleaved, param_grads=param_grads, dq=dq, dk=dk,
                               dwq=dwq, dwk=dwk, workspace=workspace)
    p_gq = _heads(*_rows("dq_out", dq_out, shape, dtype))
    if dq is None:
        dq, p_dq = _new_rows(dq_out, shape, dtype, dev)
    else:
        p_dq = _heads(*_rows("dq", dq, shape, dtype))
    r_q = _rows("q", q, shape, dtype) if norm else (0, shape[-2], 0, 0, 0)
    r_k, p_gk, p_dk = _NO_ROWS, _NONE, _NONE
    if dk_out is not None:
        kshape = _beside("dk_out", dk_out, shape)
        p_gk = _heads(*_rows("dk_out", dk_out, kshape, dtype))
        if dk is None:
            dk, p_dk = _new_rows(dk_out, kshape, dtype, dev)
        else:
            p_dk = _heads(*_rows("dk", dk, kshape, dtype))
        r_k = _rows("k", k, kshape, dtype) if norm else (0, kshape[-2], 0, 0, 0)
    elif dk is not None:
        raise ValueError("dk without dk_out")
    a_wq, a_wk = _weight("wq", wq, d, dtype), _weight("wk", wk, d, dtype)
    a_dwq = a_dwk = a_ws = nbytes = 0
    if param_grads and norm:
        if wq is not None:
            if dwq is None:
                dwq = _maker(dq_out, dev)((d,), dtype=dtype)
            a_dwq = _weight("dwq", dwq, d, dtype)
        if wk is not None:
            if dwk is None:
                dwk = _maker(dq_out, dev)((d,), dtype=dtype)
            a_dwk = _weight("dwk", dwk, d, dtype)
    if (dwq is not None and not a_dwq) or (dwk is not None and not a_dwk):
        raise ValueError("dwq and dwk need param_grads, the norm and its weights")
    if a_dwq or a_dwk:
        if workspace is None:
            nbytes = _BWD_BYTES.get(d)
            if nbytes is None:
                nbytes = _BWD_BYTES[d] = capi.qk_rope_bwd_workspace_size(d)
            workspace = torch.empty(nbytes, dtype=torch.uint8,
                                    device=dq_out.device if dq_out.is_cuda else "cuda")
        else:
            if not (workspace.is_cuda and workspace.is_contiguous()):
                raise ValueError("workspace must be a contiguous CUDA tensor")
            nbytes = workspace.numel() * workspace.element_size()
        a_ws = workspace.data_ptr()
    st = _C.qk_rope_bwd(
        _qk(*r_q, *r_k, a_wq, a_wk, pos, tab, trows, tstride, rot, batch, len_, d, code, it,
            1 if norm else 0, 1 if interleaved else 0, eps, 0), p_gq, p_gk, p_dq, p_dk, a_dwq,
        a_dwk, a_ws, nbytes, _stream(dev))
    if st:
        capi.check(st)
    return dq, dk, dwq, dwk


def _cache(k_cache, v_cache, dtype, k_scale, v_scale):
    """Packed rn_cache of ``[pages, page_size, heads, d]`` tensors, heads, d, d_v."""
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    kshape, vshape, cdtype = k_cache.shape, v_cache.shape, k_cache.dtype
    if cdtype is not _E4M3 and cdtype is not dtype:
        raise TypeError(f"k_cache must be {dtype} or {_E4M3}, got {cdtype}")
    if not (k_cache.is_cuda and v_cache.is_cuda and v_cache.dtype is cdtype):
        _check_f32_cuda("k_cache", k_cache, cdtype, contiguous=False)
        _check_f32_cuda("v_cache", v_cache, cdtype, contiguous=False)
    if len(kshape) != 4 or len(vshape) != 4:
        raise ValueError("k_cache and v_cache must be [pages, page_size, heads, d]")
    pages, page, heads, d = kshape
    if vshape != kshape and vshape[:3] != kshape[:3]:
        raise ValueError("k_cache and v_cache must hold the same pages, tokens and heads")
    dv = vshape[3]
    kp, ks, kh, k1 = k_cache.stride()
    vp, vs, vh, v1 = v_cache.stride()
    if (k1 != 1 or v1 != 1) and k_cache.numel():
        raise ValueError("k_cache and v_cache must have contiguous rows")
    return (capi.cache(k_cache.data_ptr(), v_cache.data_ptr(), kp, ks, kh, vp, vs, vh, pages, page,
                       dv, capi.RN_DTYPE_E4M3 if cdtype is _E4M3 else _FLOATS[cdtype], k_scale,
                       v_scale, 0), heads, d, dv)


def kv_append(k, v, slots, k_cache, v_cache, positions=None, table=None, wk=None,
              eps: float = 1e-5, *, q=None, wq=None, norm=None, interleaved: bool = False,
              k_scale: float = 1.0, v_scale: float = 1.0, q_out=None, stream=None):
    """Appends keys and values to a paged cache, the keys normed and turned as by
    ``qk_rope_fwd`` on the way; with ``q``, its queries too, in the same launch.

    k, v (and q): ``[tokens, heads, d]`` or ``[batch, len, heads, d]``; v may have a width of
    its own. slots: int32 or int64, one a token (of positions' type): page times page size
    plus the token's place in its page, each at most once; a token whose slot is outside the
    cache (-1: padding) is not stored. k_cache, v_cache: ``[pages, page_size, heads, d]`` with
    contiguous rows and any other strides, of k's type or float8_e4m3fn; an 8-bit cache holds
    values divided by k_scale and v_scale (FP32 quotients, rounded to nearest even), at most 448 in
    size. Returns ``q_out`` (None without q), which may be passed in, q itself among them.
    """
    if q_out is None and stream is None:
        out = _B.kv_append(k, v, slots, k_cache, v_cache, positions, table, wk, eps, q, wq, norm,
                           interleaved, k_scale, v_scale)
        if out is not None:
            return out[0]
    _tensors(k=k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache, positions=positions,
             table=table, wk=wk, q=q, wq=wq, q_out=q_out)
    code, shape = _first("k", k)
    dtype, hk, d, len_ = k.dtype, shape[-2], shape[-1], shape[-3]
    batch = 1 if len(shape) == 3 else shape[0]
    n = batch * len_
    if norm is None:
        norm = wq is not None or wk is not None
    it = _ids("slots", slots)
    if slots.numel() != n:
        raise ValueError(f"slots must have {n} elements")
    pos, tab, trows, tstride, rot, pit = _turn(positions, table, n)
    if rot and pit != it:
        raise TypeError(f"slots and positions must have one type, got {slots.dtype} and "
                        f"{positions.dtype}")
    dev = _device(k, v, slots, k_cache, v_cache, positions, table, wk, q, wq, q_out)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_append(k, v, slots, k_cache, v_cache, positions, table, wk, eps, q=q, wq=wq,
                             norm=norm, interleaved=interleaved, k_scale=k_scale,
                             v_scale=v_scale, q_out=q_out)
    a_c, heads, dk, dv = _cache(k_cache, v_cache, dtype, k_scale, v_scale)
    if heads != hk or dk != d:
        raise ValueError(f"k_cache holds {heads} heads of {dk}, k has {hk} of {d}")
    r_k = _rows("k", k, shape, dtype)
    p_v = _heads(*_rows("v", v, shape if dv == d else (*shape[:-1], dv), dtype))
    r_q, p_q = _NO_ROWS, _NONE
    if q is not None:
        qshape = _beside("q", q, shape)
        r_q = _rows("q", q, qshape, dtype)
        if q_out is None:
            q_out, p_q = _new_rows(q, qshape, dtype, dev)
        else:
            p_q = _heads(*_rows("q_out", q_out, qshape, dtype))
    elif q_out is not None or wq is not None:
        raise ValueError("q_out and wq need q")
    st = _C.kv_append(
        _qk(*r_q, *r_k, _weight("wq", wq, d, dtype), _weight("wk", wk, d, dtype), pos, tab, trows,
            tstride, rot, batch, len_, d, code, it, 1 if norm else 0, 1 if interleaved else 0, eps,
            0), p_q, p_v, a_c, slots.data_ptr(), _stream(dev))
    if st:
        capi.check(st)
    return q_out


def kv_gather(k_cache, v_cache, slots, *, dtype=None, k_scale: float = 1.0, v_scale: float = 1.0,
              k_out=None, v_out=None, stream=None):
    """The rows of ``slots`` (int32 or int64, any shape of them, repeats allowed) out of a
    paged cache: ``(k, v)`` of shape ``[tokens, heads, d]``, rows of zeros where a slot is
    outside the cache. An 8-bit cache's values are multiplied by their scales and come in
    ``dtype`` (bfloat16 unless given); otherwise dtype is the cache's. k_out, v_out may be
    passed in (contiguous rows, any other strides).
    """
    if k_out is None and v_out is None and stream is None:
        out = _B.kv_gather(k_cache, v_cache, slots, dtype, k_scale, v_scale)
        if out is not None:
            return out
    _tensors(k_cache=k_cache, v_cache=v_cache, slots=slots, k_out=k_out, v_out=v_out)
    if k_cache is None:
        raise TypeError("k_cache must be a torch.Tensor")
    if dtype is None:
        dtype = (k_out.dtype if k_out is not None else
                 torch.bfloat16 if k_cache.dtype is _E4M3 else k_cache.dtype)
    code = _FLOATS.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32, bfloat16 or float16)")
    it = _ids("slots", slots)
    n = slots.numel()
    dev = _device(k_cache, v_cache, slots, k_out, v_out)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_gather(k_cache, v_cache, slots, dtype=dtype, k_scale=k_scale,
                             v_scale=v_scale, k_out=k_out, v_out=v_out)
    a_c, heads, d, dv = _cache(k_cache, v_cache, dtype, k_scale, v_scale)
    if k_out is None:
        k_out = _maker(k_cache, dev)((n, heads, d), dtype=dtype)
        p_k = _heads(k_out.data_ptr(), heads, 0, heads * d, d)
    else:
        p_k = _heads(*_rows("k_out", k_out, (n, heads, d), dtype))
    if v_out is None:
        v_out = _maker(v_cache, dev)((n, heads, dv), dtype=dtype)
        p_v = _heads(v_out.data_ptr(), heads, 0, heads * dv, dv)
    else:
        p_v = _heads(*_rows("v_out", v_out, (n, heads, dv), dtype))
    st = _C.kv_gather(a_c, d, slots.data_ptr(), it, n, code, p_k, p_v, _stream(dev))
    if st:
        capi.check(st)
    return k_out, v_out


def kv_slots(page_table, starts, offsets, n: int, page_size: int, *, slots=None, positions=None,
             stream=None):
    """Slots and positions of the ``n`` tokens of a ragged batch: ``(slots, positions)``.

    Tokens ``offsets[b] .. offsets[b + 1]`` belong to sequence b, whose first new token has
    position ``starts[b]`` and whose pages are ``page_table[b]``; tokens of no sequence get -1.
    page_table ``[sequences, width]`` (contiguous rows), starts ``[sequences]``, offsets
    ``[sequences + 1]``: int32 or int64, one type, which is the outputs' too. The results are
    what ``kv_append`` and ``qk_rope_fwd`` take for every layer of a step; with starts of 0,
    what ``kv_gather`` takes for whole sequences.
    """
    if slots is None and positions is None and stream is None:
        out = _B.kv_slots(page_table, starts, offsets, n, page_size)
        if out is not None:
            return out
    _tensors(page_table=page_table, starts=starts, offsets=offsets, slots=slots,
             positions=positions)
    if page_table is None:
        raise TypeError("page_table must be a torch.Tensor")
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be 2-D")
    it = _ids("offsets", offsets)
    dtype = offsets.dtype
    seqs, width = shape
    if not page_table.is_cuda or page_table.dtype is not dtype:
        _check_f32_cuda("page_table", page_table, dtype, contiguous=False)
    ld, one = page_table.stride()
    if one != 1 and width > 1 and seqs:
        raise ValueError("page_table must have contiguous rows")
    if _ids("starts", starts) != it:
        raise TypeError(f"starts must be {dtype}, got {starts.dtype}")
    if starts.numel() != seqs or offsets.numel() != seqs + 1:
        raise ValueError(f"starts must have {seqs} elements, offsets {seqs + 1}")
    dev = _device(page_table, starts, offsets, slots, positions)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_slots(page_table, starts, offsets, n, page_size, slots=slots,
                            positions=positions)
    if slots is None:
        slots = _maker(offsets, dev)(n, dtype=dtype)
    elif _ids("slots", slots) != it or slots.numel() != n:
        raise ValueError(f"slots must be {dtype} with {n} elements")
    if positions is None:
        positions = _maker(offsets, dev)(n, dtype=dtype)
    elif _ids("positions", positions) != it or positions.numel() != n:
        raise ValueError(f"positions must be {dtype} with {n} elements")
    st = _C.kv_slots(it, page_table.data_ptr(), ld if seqs > 1 else width, width,
                     starts.data_ptr(), offsets.data_ptr(), seqs, page_size, slots.data_ptr(),
                     positions.data_ptr(), n, _stream(dev))
    if st:
        capi.check(st)
    return slots, positions
