"""Row-wise LayerNorm / RMSNorm on GB300 (sm_103a), and the token operators on
either side of them (embedding rows, log probabilities).

A thin torch-facing binding over the C ABI of ``librownorm.so``
(include/rownorm.h): it checks tensor shapes and dtypes, allocates outputs
with torch when the caller does not pass them, and hands raw device pointers
and the current CUDA stream to the library. Every arithmetic step runs in the
library's CUDA kernels; if the library is missing, calls raise.
"""
from __future__ import annotations

from . import capi
from .capi import RowNormError, load  # noqa: F401

__all__ = ["ln_fwd", "rms_fwd", "ln_fwd_residual", "rms_fwd_residual", "ln_fwd_batched",
           "rms_fwd_batched", "ln_bwd", "rms_bwd", "embed_fwd", "embed_bwd", "logprob_fwd",
           "logprob_bwd", "capi", "RowNormError", "load"]


def _stream_handle(t, stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(t.device if t.is_cuda else None)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _empty_like_home(x, shape, dtype=None):
    import torch

    dtype = torch.float32 if dtype is None else dtype
    if x.is_cuda:
        return torch.empty(shape, dtype=dtype, device=x.device)
    return torch.empty(shape, dtype=dtype, pin_memory=x.is_pinned())


_PAGEABLE = {}


def _pageable_ok():
    """Whether the current GPU reads pageable host memory (asked once per
    device)."""
    import torch

    if not torch.cuda.is_available():
        return False
    dev = torch.cuda.current_device()
    if dev not in _PAGEABLE:
        _PAGEABLE[dev] = capi.pageable_host_access()
    return _PAGEABLE[dev]


def _dtype_code(t):
    import torch

    codes = {torch.float32: capi.RN_DTYPE_F32, torch.bfloat16: capi.RN_DTYPE_BF16,
             torch.float16: capi.RN_DTYPE_F16}
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return codes[t.dtype]


def _check_f32_cuda(name, t, dtype=None, contiguous=True):
    """Contiguous, of the expected dtype (FP32 unless given), and addressable
    by the GPU: a CUDA tensor, a pinned CPU tensor, or, on a GPU that reads
    pageable host memory (GB300), any CPU tensor (the kernel reads or writes
    host tensors over the host link)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not (t.is_cuda or t.is_pinned() or (t.device.type == "cpu" and _pageable_ok())):
        raise ValueError(f"{name} must be a CUDA tensor or a pinned CPU tensor (this GPU "
                         f"does not read pageable host memory)")
    want = torch.float32 if dtype is None else dtype
    if t.dtype != want:
        raise TypeError(f"{name} must be {want}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows_of(name, t, d):
    """(rows, row stride) of x or y: a contiguous tensor of rows of d, or a
    2-D tensor whose rows are d contiguous elements at a stride >= d (a column
    block of a wider matrix)."""
    if t.is_contiguous():
        return (t.numel() // d if d else 0), d
    if t.dim() == 2 and t.shape[1] == d and t.stride(1) == 1 and t.stride(0) >= d:
        return t.shape[0], t.stride(0)
    raise ValueError(f"{name} must be contiguous, or 2-D with unit column stride and a row "
                     f"stride >= its width")


def ln_fwd(x, gamma, beta, eps: float = 1e-5, *, y=None, mean=None, rstd=None, stream=None,
           variant: int = capi.RN_VARIANT_AUTO):
    """LayerNorm forward over the last dimension of ``x``.

    x, gamma, beta (and y) are float32, bfloat16 or float16 -- all the same
    type; statistics are computed in FP32. Returns ``(y, mean, rstd)``: y like
    x; mean and rstd FP32 of shape x.shape[:-1]. Tensors are CUDA tensors or
    pinned CPU tensors, or any CPU tensors on a GPU that reads pageable host
    memory (read or written by the kernel over the host link);
    outputs not passed in are allocated where x lives. x and y may also be
    2-D row-strided views (``big[:, a:a + d]``): the kernels then read and
    write the rows in place.
    """
    code = _dtype_code(x)
    _check_f32_cuda("x", x, x.dtype, contiguous=False)
    d = x.shape[-1]
    rows, ldx = _rows_of("x", x, d)
    for n, t in (("gamma", gamma), ("beta", beta)):
        _check_f32_cuda(n, t, x.dtype)
        if t.numel() != d:
            raise ValueError(f"{n} must have {d} elements")
    if y is None:
        y = _empty_like_home(x, x.shape, x.dtype)
    if mean is None:
        mean = _empty_like_home(x, x.shape[:-1])
    if rstd is None:
        rstd = _empty_like_home(x, x.shape[:-1])
    _check_f32_cuda("y", y, x.dtype, contiguous=False)
    if y.numel() != x.numel() or y.shape[-1] != d:
        raise ValueError("y must be shaped like x")
    _, ldy = _rows_of("y", y, d)
    for n, t in (("mean", mean), ("rstd", rstd)):
        _check_f32_cuda(n, t)
        if t.numel() != rows:
            raise ValueError(f"{n} must have {rows} elements")
    if ldx == d and ldy == d:
        st = capi.ln_fwd_typed(code, variant, x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                               y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, d,
                               float(eps), _stream_handle(x, stream))
    else:
        st = capi.ln_fwd_strided(code, variant, x.data_ptr(), ldx, gamma.data_ptr(),
                                 beta.data_ptr(), y.data_ptr(), ldy, mean.data_ptr(),
                                 rstd.data_ptr(), rows, d, float(eps), _stream_handle(x, stream))
    capi.check(st)
    return y, mean, rstd


def rms_fwd(x, w, eps: float = 1e-5, *, y=None, stream=None,
            variant: int = capi.RN_VARIANT_AUTO):
    """RMSNorm forward over the last dimension of ``x`` (float32, bfloat16 or
    float16; w of the same type); returns y. x and y may be 2-D row-strided
    views, as in ln_fwd."""
    code = _dtype_code(x)
    _check_f32_cuda("x", x, x.dtype, contiguous=False)
    d = x.shape[-1]
    rows, ldx = _rows_of("x", x, d)
    _check_f32_cuda("w", w, x.dtype)
    if w.numel() != d:
        raise ValueError(f"w must have {d} elements")
    if y is None:
        y = _empty_like_home(x, x.shape, x.dtype)
    _check_f32_cuda("y", y, x.dtype, contiguous=False)
    if y.numel() != x.numel() or y.shape[-1] != d:
        raise ValueError("y must be shaped like x")
    _, ldy = _rows_of("y", y, d)
    if ldx == d and ldy == d:
        st = capi.rms_fwd_typed(code, variant, x.data_ptr(), w.data_ptr(), y.data_ptr(), rows, d,
                                float(eps), _stream_handle(x, stream))
    else:
        st = capi.rms_fwd_strided(code, variant, x.data_ptr(), ldx, w.data_ptr(), y.data_ptr(),
                                  ldy, rows, d, float(eps), _stream_handle(x, stream))
    capi.check(st)
    return y


def _batched(op, problems, eps, stream):
    if not problems:
        return []
    x0 = problems[0][0]
    code = _dtype_code(x0)
    items, outs = [], []
    for k, pr in enumerate(problems):
        x, params = pr[0], pr[1:]
        _check_f32_cuda(f"problem {k} x", x, x0.dtype)
        d = x.shape[-1]
        rows = x.numel() // d if d else 0
        for t in params:
            _check_f32_cuda(f"problem {k} parameter", t, x0.dtype)
            if t.numel() != d:
                raise ValueError(f"problem {k}: parameters must have {d} elements")
        y = _empty_like_home(x, x.shape, x.dtype)
        if op == capi.RN_OP_LN:
            mean = _empty_like_home(x, x.shape[:-1])
            rstd = _empty_like_home(x, x.shape[:-1])
            items.append((x.data_ptr(), params[0].data_ptr(), params[1].data_ptr(), y.data_ptr(),
                          mean.data_ptr(), rstd.data_ptr(), rows, d))
            outs.append((y, mean, rstd))
        else:
            items.append((x.data_ptr(), params[0].data_ptr(), 0, y.data_ptr(), 0, 0, rows, d))
            outs.append(y)
    fn = capi.ln_fwd_batched if op == capi.RN_OP_LN else capi.rms_fwd_batched
    capi.check(fn(code, capi.problems(items), len(items), float(eps), _stream_handle(x0, stream)))
    return outs


def ln_fwd_batched(problems, eps: float = 1e-5, *, stream=None):
    """LayerNorm of many small tensors in as few launches as possible.

    ``problems``: a sequence of ``(x, gamma, beta)``, contiguous, all of one
    dtype (float32, bfloat16 or float16). Returns a list of ``(y, mean,
    rstd)``, one per problem. Problems of width <= 1024 share one launch per
    128; wider ones get their own.
    """
    return _batched(capi.RN_OP_LN, problems, eps, stream)


def rms_fwd_batched(problems, eps: float = 1e-5, *, stream=None):
    """RMSNorm of many small tensors: ``problems`` is a sequence of ``(x, w)``;
    returns the list of y."""
    return _batched(capi.RN_OP_RMS, problems, eps, stream)


def _check_like(name, t, numel):
    _check_f32_cuda(name, t)
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements")


def ln_fwd_residual(x, res, gamma, beta, eps: float = 1e-5, *, h=None, y=None, mean=None,
                    rstd=None, write_h: bool = True, stream=None,
                    variant: int = capi.RN_VARIANT_AUTO):
    """h = x + res, then LayerNorm of h over the last dimension, in one kernel.

    Returns ``(h, y, mean, rstd)``; h is None when ``write_h`` is False and no
    h tensor is passed. Tensors are CUDA tensors or host tensors as for ln_fwd.
    """
    _check_f32_cuda("x", x)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    _check_like("res", res, x.numel())
    _check_like("gamma", gamma, d)
    _check_like("beta", beta, d)
    if h is None and write_h:
        h = _empty_like_home(x, x.shape)
    y = _empty_like_home(x, x.shape) if y is None else y
    mean = _empty_like_home(x, x.shape[:-1]) if mean is None else mean
    rstd = _empty_like_home(x, x.shape[:-1]) if rstd is None else rstd
    if h is not None:
        _check_like("h", h, x.numel())
    _check_like("y", y, x.numel())
    _check_like("mean", mean, rows)
    _check_like("rstd", rstd, rows)
    st = capi.ln_fwd_residual_variant(variant, x.data_ptr(), res.data_ptr(), gamma.data_ptr(),
                                      beta.data_ptr(), h.data_ptr() if h is not None else 0,
                                      y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), rows, d,
                                      float(eps), _stream_handle(x, stream))
    capi.check(st)
    return h, y, mean, rstd


def rms_fwd_residual(x, res, w, eps: float = 1e-5, *, h=None, y=None, write_h: bool = True,
                     stream=None, variant: int = capi.RN_VARIANT_AUTO):
    """h = x + res, then RMSNorm of h over the last dimension, in one kernel.

    Returns ``(h, y)``; h is None when ``write_h`` is False and none is passed.
    """
    _check_f32_cuda("x", x)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    _check_like("res", res, x.numel())
    _check_like("w", w, d)
    if h is None and write_h:
        h = _empty_like_home(x, x.shape)
    y = _empty_like_home(x, x.shape) if y is None else y
    if h is not None:
        _check_like("h", h, x.numel())
    _check_like("y", y, x.numel())
    st = capi.rms_fwd_residual_variant(variant, x.data_ptr(), res.data_ptr(), w.data_ptr(),
                                       h.data_ptr() if h is not None else 0, y.data_ptr(), rows,
                                       d, float(eps), _stream_handle(x, stream))
    capi.check(st)
    return h, y


def _workspace(op, rows, d, device, workspace):
    import torch

    if workspace is not None:
        return workspace
    nbytes = capi.bwd_workspace_size(op, rows, d)
    return torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=device)


def ln_bwd(dy, x, gamma, mean, rstd, *, dx=None, dgamma=None, dbeta=None,
           param_grads: bool = True, workspace=None, stream=None):
    """LayerNorm backward from the forward's saved mean and rstd. dy, x and
    gamma are float32, bfloat16 or float16 (one type; dx and the parameter
    gradients come back in it); mean and rstd are FP32. Returns ``(dx,
    dgamma, dbeta)`` (the last two None when ``param_grads`` is False).
    ``workspace``: a float32 CUDA tensor for the parameter-gradient partials
    (allocated if not given)."""
    import torch

    code = _dtype_code(x)
    for n, t in (("dy", dy), ("x", x), ("gamma", gamma)):
        _check_f32_cuda(n, t, x.dtype)
    for n, t in (("mean", mean), ("rstd", rstd)):
        _check_f32_cuda(n, t)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    dx = torch.empty_like(x) if dx is None else dx
    if param_grads:
        dgamma = torch.empty(d, dtype=x.dtype, device=x.device) if dgamma is None else dgamma
        dbeta = torch.empty(d, dtype=x.dtype, device=x.device) if dbeta is None else dbeta
        ws = _workspace(capi.RN_OP_LN, rows, d, x.device, workspace)
    else:
        dgamma = dbeta = ws = None
    st = capi.ln_bwd_typed(code, dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), mean.data_ptr(),
                           rstd.data_ptr(), dx.data_ptr(),
                           dgamma.data_ptr() if dgamma is not None else 0,
                           dbeta.data_ptr() if dbeta is not None else 0, rows, d,
                           ws.data_ptr() if ws is not None else 0,
                           ws.numel() * 4 if ws is not None else 0, _stream_handle(x, stream))
    capi.check(st)
    return dx, dgamma, dbeta


def rms_bwd(dy, x, w, eps: float = 1e-5, *, dx=None, dw=None, param_grads: bool = True,
            workspace=None, stream=None):
    """RMSNorm backward (float32, bfloat16 or float16 tensors of one type).
    Returns ``(dx, dw)``."""
    import torch

    code = _dtype_code(x)
    for n, t in (("dy", dy), ("x", x), ("w", w)):
        _check_f32_cuda(n, t, x.dtype)
    d = x.shape[-1]
    rows = x.numel() // d if d else 0
    dx = torch.empty_like(x) if dx is None else dx
    if param_grads:
        dw = torch.empty(d, dtype=x.dtype, device=x.device) if dw is None else dw
        ws = _workspace(capi.RN_OP_RMS, rows, d, x.device, workspace)
    else:
        dw = ws = None
    st = capi.rms_bwd_typed(code, dy.data_ptr(), x.data_ptr(), w.data_ptr(), dx.data_ptr(),
                            dw.data_ptr() if dw is not None else 0, rows, d, float(eps),
                            ws.data_ptr() if ws is not None else 0,
                            ws.numel() * 4 if ws is not None else 0, _stream_handle(x, stream))
    capi.check(st)
    return dx, dw


# ---------------------------------------------------------------------------
# token operators
#
# A decoding step waits for the host side of these calls, not for their kernels
# (a few microseconds each), so what they check is written to be checked fast:
# types by one dictionary, contiguous device tensors first, the current device
# and stream left alone unless the call names others.
# ---------------------------------------------------------------------------
_CODES = {}


def _codes():
    import torch

    if not _CODES:
        _CODES.update({torch.float32: capi.RN_DTYPE_F32, torch.bfloat16: capi.RN_DTYPE_BF16,
                       torch.float16: capi.RN_DTYPE_F16, torch.int32: capi.RN_INDEX_I32,
                       torch.int64: capi.RN_INDEX_I64})
    return _CODES


def _values(name, t):
    """The storage code of a floating-point tensor."""
    try:
        code = _codes()[t.dtype]
        if t.dtype.is_floating_point:
            return code
    except (AttributeError, KeyError):
        pass
    if not hasattr(t, "dtype"):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise TypeError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")


def _ids(name, t):
    """The index code of a contiguous tensor of ids."""
    try:
        code = _codes()[t.dtype]
        if not t.dtype.is_floating_point:
            if not (t.is_cuda and t.is_contiguous()):
                _check_f32_cuda(name, t, t.dtype)
            return code
    except (AttributeError, KeyError):
        pass
    if not hasattr(t, "dtype"):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise TypeError(f"{name} must be int32 or int64, got {t.dtype}")


def _row_floats(name, t, rows):
    """Address of an FP32 vector of a value a row (0 for None)."""
    if t is None:
        return 0
    import torch

    if not (getattr(t, "is_cuda", False) and t.dtype is torch.float32 and t.is_contiguous()):
        _check_f32_cuda(name, t)
    if t.numel() != rows:
        raise ValueError(f"{name} must have {rows} elements")
    return t.data_ptr()


def _matrix(name, t, d, dtype):
    """(rows, row stride) of a typed matrix of rows of d (see _rows_of)."""
    if t.is_cuda and t.dtype is dtype and t.is_contiguous() and d > 0:
        return t.numel() // d, d
    _check_f32_cuda(name, t, dtype, contiguous=False)
    return _rows_of(name, t, d)


def _device_of(tensors):
    """The one device of a call's CUDA tensors (None where all are in host
    memory)."""
    dev = None
    for t in tensors:
        if t is not None and t.is_cuda:
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise ValueError(f"tensors on {dev} and on {t.device}")
    return dev


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _elsewhere(dev, stream):
    """Whether a call needs another device or stream made current first."""
    import torch

    return stream is not None or (dev is not None and dev.index != torch.cuda.current_device())


class _On:
    """Makes the call's device current and, where the caller gives a stream of
    its own, that stream too, so that the memory the call allocates belongs to the
    stream that uses it."""

    def __init__(self, dev, stream):
        import torch

        if isinstance(stream, int):
            # (handle 0: the legacy default stream, torch's default stream)
            stream = (torch.cuda.ExternalStream(stream, device=dev) if stream
                      else torch.cuda.default_stream(dev))
        elif stream is not None and dev is not None and stream.device != dev:
            raise ValueError(f"stream belongs to {stream.device}, the tensors to {dev}")
        self._inner = [torch.cuda.stream(stream)]
        if dev is not None:
            self._inner.insert(0, torch.cuda.device(dev))

    def __enter__(self):
        for c in self._inner:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self._inner):
            c.__exit__(*exc)


def _current_stream(dev):
    """Handle of the current stream of the call's device (of the current device,
    where every tensor is in host memory)."""
    import torch

    if dev is None:
        return torch.cuda.current_stream().cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _new(home, dev, shape, dtype):
    """An output on the call's device, or in host memory like `home`."""
    import torch

    if dev is not None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _empty_like_home(home, shape, dtype)


def embed_fwd(tokens, table, scale: float = 1.0, *, out=None, stream=None):
    """Embedding rows ``scale * table[tokens]``.

    tokens: int32 or int64 ids of any shape; an id outside ``[0, vocab)`` gives a
    row of zeros. table: ``[vocab, d]``, float32, bfloat16 or float16, contiguous
    or a row-strided view. Returns ``out`` of shape ``tokens.shape + (d,)`` in the
    table's type (``out`` may also be passed as a 2-D row-strided view).
    """
    dtype = getattr(table, "dtype", None)
    code = _values("table", table)
    it = _ids("tokens", tokens)
    if table.dim() != 2:
        raise ValueError("table must be 2-D")
    vocab, d = table.shape
    _, ldt = _matrix("table", table, d, dtype)
    dev = _device_of((table, tokens, out))
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return embed_fwd(tokens, table, scale, out=out)
    n = tokens.numel()
    if out is None:
        out, ldo = _new(table, dev, (*tokens.shape, d), dtype), d
    else:
        if out.numel() != n * d or out.shape[-1:] != (d,):
            raise ValueError(f"out must hold {n} rows of {d}")
        _, ldo = _matrix("out", out, d, dtype)
    capi.check(capi.embed_fwd(code, it, tokens.data_ptr(), table.data_ptr(), ldt, out.data_ptr(),
                              ldo, n, vocab, d, float(scale), _current_stream(dev)))
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
    import torch

    code = _values("dout", dout)
    it = _ids("tokens", tokens)
    n = tokens.numel()
    if dout.dim() < 1:
        raise ValueError("dout must have a last dimension")
    d = dout.shape[-1]
    if dout.numel() != n * d:
        raise ValueError(f"dout must hold {n} rows of {d}")
    _, lddo = _matrix("dout", dout, d, dout.dtype)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs a dtable to add to")
        gdtype = dout.dtype if dtype is None else dtype
    else:
        gdtype = dtable.dtype
        if dtype is not None and dtype != gdtype:
            raise TypeError(f"dtable is {gdtype}, dtype says {dtype}")
    if gdtype not in (dout.dtype, torch.float32):
        raise TypeError(f"dtable must be {dout.dtype} or float32")
    dev = _device_of((dout, tokens, dtable, workspace))
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return embed_bwd(dout, tokens, vocab, scale, dtype=dtype, dtable=dtable,
                             accumulate=accumulate, workspace=workspace)
    if dtable is None:
        dtable, ldg = _new(dout, dev, (vocab, d), gdtype), d
    else:
        if tuple(dtable.shape) != (vocab, d):
            raise ValueError(f"dtable must be of shape [{vocab}, {d}]")
        _, ldg = _matrix("dtable", dtable, d, gdtype)
    if workspace is None:
        nbytes = capi.embed_bwd_workspace_size(n, vocab, d)
        workspace = torch.empty(nbytes, dtype=torch.uint8,
                                device=dev if dev is not None else "cuda")
    else:
        if not (workspace.is_cuda and workspace.is_contiguous()):
            raise ValueError("workspace must be a contiguous CUDA tensor")
        nbytes = workspace.numel() * workspace.element_size()
    capi.check(capi.embed_bwd(code, _values("dtable", dtable), it, dout.data_ptr(), lddo,
                              tokens.data_ptr(), dtable.data_ptr(), ldg, n, vocab, d,
                              float(scale), 1 if accumulate else 0, workspace.data_ptr(), nbytes,
                              _current_stream(dev)))
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
    import torch

    code = _values("logits", logits)
    if logits.dim() < 1:
        raise ValueError("logits must have a last dimension")
    vocab = logits.shape[-1]
    rows, ldl = _matrix("logits", logits, vocab, logits.dtype)
    lead = logits.shape[:-1]
    it, itype, tgt = capi.RN_INDEX_I64, torch.int64, 0
    if targets is not None:
        it, itype, tgt = _ids("targets", targets), targets.dtype, targets.data_ptr()
        if targets.numel() != rows:
            raise ValueError(f"targets must have {rows} elements")
    dev = _device_of((logits, targets))
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return logprob_fwd(logits, targets, scale, top=top, want_entropy=want_entropy)
    f32 = torch.float32
    logp = entropy = ids = top_logp = None
    if targets is not None:
        logp = _new(logits, dev, lead, f32)
    if want_entropy:
        entropy = _new(logits, dev, lead, f32)
    lse = _new(logits, dev, lead, f32)
    if top > 0:
        ids = _new(logits, dev, (*lead, top), itype)
        top_logp = _new(logits, dev, (*lead, top), f32)
    capi.check(capi.logprob_fwd(code, it, logits.data_ptr(), ldl, tgt, _ptr(logp), _ptr(entropy),
                                lse.data_ptr(), _ptr(ids), _ptr(top_logp), rows, vocab, int(top),
                                float(scale), _current_stream(dev)))
    return logp, entropy, lse, ids, top_logp


def logprob_bwd(dlogp, logits, targets, lse, scale: float = 1.0, *, dentropy=None, entropy=None,
                dlogits=None, stream=None):
    """Gradient of ``logprob_fwd``'s log probabilities (dlogp) and, where
    ``dentropy`` is given with the forward call's ``entropy``, of its entropies,
    with respect to the logits. dlogp may be None (then targets too). ``dlogits``:
    allocated in the logits' type unless given; it may be ``logits`` itself.
    """
    code = _values("logits", logits)
    if logits.dim() < 1:
        raise ValueError("logits must have a last dimension")
    vocab = logits.shape[-1]
    rows, ldl = _matrix("logits", logits, vocab, logits.dtype)
    it, tgt = capi.RN_INDEX_I64, 0
    if targets is not None:
        it, tgt = _ids("targets", targets), targets.data_ptr()
        if targets.numel() != rows:
            raise ValueError(f"targets must have {rows} elements")
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    rows_of = [_row_floats(n, t, rows) for n, t in (("dlogp", dlogp), ("dentropy", dentropy),
                                                    ("lse", lse), ("entropy", entropy))]
    dev = _device_of((logits, dlogp, targets, lse, dentropy, entropy, dlogits))
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return logprob_bwd(dlogp, logits, targets, lse, scale, dentropy=dentropy,
                               entropy=entropy, dlogits=dlogits)
    if dlogits is None:
        dlogits, ldd = _new(logits, dev, logits.shape, logits.dtype), vocab
    else:
        if dlogits.numel() != logits.numel() or dlogits.shape[-1] != vocab:
            raise ValueError("dlogits must be shaped like logits")
        _, ldd = _matrix("dlogits", dlogits, vocab, logits.dtype)
    capi.check(capi.logprob_bwd(code, it, rows_of[0], rows_of[1], logits.data_ptr(), ldl, tgt,
                                rows_of[2], rows_of[3], dlogits.data_ptr(), ldd, rows, vocab,
                                float(scale), _current_stream(dev)))
    return dlogits
