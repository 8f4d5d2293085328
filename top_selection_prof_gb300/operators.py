"""The operators around the selection (include/topk.h): a sparse autoencoder's step with BatchTopK.

    acts = tk.linear(x, w_enc, b_enc, act="relu")                 # (rows, n)
    vals, idx = tk.select_global(acts, K)                         # or tk.select(acts, k): k features a row
    y = tk.decode(vals, idx, w_dec, rows, bias=b_dec)             # (rows, d)
    dvals, dw_dec, db_dec = tk.decode_backward(dy, vals, idx, w_dec)
    dx, dw_enc, db_enc = tk.linear_backward_selected(dvals, vals, idx, x, w_enc, act="relu")
    norm = tk.clip_grad_norm_([dw_enc, db_enc, dw_dec, db_dec], 1.0)

As for the selection, every step runs in the library's CUDA kernels; this
module checks tensors, allocates outputs and passes pointers and the stream.
Inputs are float32 or bfloat16 CUDA tensors, all of one dtype and device in a
call; matrices may be strided by row, with their last dimension contiguous.

stream=: the stream that a call runs on, the current one by default.  As with
torch's own streams the caller orders another one (wait_stream) after what makes
the inputs and before what uses the outputs; their memory is kept for both
streams.  Nothing is recorded for autograd: outputs never require gradients, and
the *_backward functions are what an autograd.Function calls.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import TOPK_ACT_GELU, TOPK_ACT_NONE, TOPK_ACT_RELU, TOPK_ACT_SILU, TOPK_BF16, TOPK_F32

_ACTS = {"none": TOPK_ACT_NONE, "relu": TOPK_ACT_RELU, "gelu": TOPK_ACT_GELU, "silu": TOPK_ACT_SILU}
_CODES = {torch.float32: TOPK_F32, torch.bfloat16: TOPK_BF16}


def _act(act: str) -> int:
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError("act must be one of %s, got %r" % (", ".join(_ACTS), act)) from None


def _first(t):
    """dtype code of the tensor that the call's others are checked against."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("input must be a CUDA tensor (the engine has no CPU path)")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("operators take float32 or bfloat16 tensors, got %s" % t.dtype)
    return code


def _like(t, dtype, device, name):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device:
        raise TypeError("%s must be a %s tensor on %s" % (name, dtype, device))


def _matrix(t, rows, cols, name):
    """Distance between the rows of t, which must be (rows, cols) with contiguous rows that do not overlap."""
    if t.shape != (rows, cols):
        raise ValueError("%s must have shape (%d, %d), got %s" % (name, rows, cols, tuple(t.shape)))
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    if rows <= 1:
        return cols
    if s0 < cols:
        raise ValueError("the rows of %s must not overlap" % name)
    return s0


def _vector(t, dtype, device, n, name):
    _like(t, dtype, device, name)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d values" % (name, n))
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """An output: memory of the stream that writes it (the current one may still read what memory of its own held), kept
    until the current one, too, has done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


_FUNCTIONS = {}


def _call(name, device, stream, tensors, *args):
    """lib.<name>(*args, stream); with a stream of the caller's, the call's tensors are kept until it has run."""
    fn = _FUNCTIONS.get(name)
    if fn is None:
        fn = _FUNCTIONS[name] = getattr(_lib.get(), name)
    index = device.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc:
        _lib.check(rc, name)


def linear(x, w, bias=None, act: str = "none", residual=None, save_pre: bool = False, out=None, stream=None):
    """act(x w^T + bias) + residual, with x (rows, inner) and w (outer, inner).

    save_pre=True returns (y, pre) with pre = x w^T + bias, for linear_backward.  out: where y is written
    (it may be the residual)."""
    code = _first(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (rows, inner)")
    rows, inner = x.shape
    dtype, device = x.dtype, x.device
    _like(w, dtype, device, "w")
    outer = w.shape[0]
    ldx, ldw = _matrix(x, rows, inner, "x"), _matrix(w, outer, inner, "w")
    pb = None if bias is None else _vector(bias, dtype, device, outer, "bias")
    pr, ldr = None, 0
    if residual is not None:
        _like(residual, dtype, device, "residual")
        pr, ldr = residual.data_ptr(), _matrix(residual, rows, outer, "residual")
    if out is None:
        out, ldy = _empty((rows, outer), dtype, device, stream), outer
    else:
        _like(out, dtype, device, "out")
        ldy = _matrix(out, rows, outer, "out")
    pre = _empty((rows, outer), dtype, device, stream) if save_pre else None
    _call("topk_linear", device, stream, (x, w, bias, residual, out, pre), x.data_ptr(), ldx, w.data_ptr(), ldw, pb, pr,
          ldr, code, rows, inner, outer, _act(act), out.data_ptr(), ldy, pre.data_ptr() if save_pre else None, outer)
    return (out, pre) if save_pre else out


def linear_backward(dy, x, w, pre=None, act: str = "none", need=(True, True, True), stream=None):
    """(dx, dw, dbias) of linear from dy (rows, outer); None where `need` is false.

    pre: what linear kept with save_pre (needed unless act is "none"; with "relu" and no residual, its output serves)."""
    code = _first(dy)
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D (rows, outer)")
    rows, outer = dy.shape
    dtype, device = dy.dtype, dy.device
    _like(x, dtype, device, "x")
    _like(w, dtype, device, "w")
    if w.dim() != 2:
        raise ValueError("w must be 2-D (outer, inner)")
    inner = w.shape[1]
    lddy, ldx, ldw = _matrix(dy, rows, outer, "dy"), _matrix(x, rows, inner, "x"), _matrix(w, outer, inner, "w")
    a, ldp = _act(act), 0
    if a != TOPK_ACT_NONE:
        if pre is None:
            raise ValueError("act %r needs pre" % act)
        _like(pre, dtype, device, "pre")
        ldp = _matrix(pre, rows, outer, "pre")
    else:
        pre = None
    dx = _empty((rows, inner), dtype, device, stream) if need[0] else None
    dw = _empty((outer, inner), dtype, device, stream) if need[1] else None
    db = _empty((outer,), dtype, device, stream) if need[2] else None
    _call("topk_linear_backward", device, stream, (dy, x, w, pre, dx, dw, db), dy.data_ptr(), lddy, x.data_ptr(), ldx,
          w.data_ptr(), ldw, None if pre is None else pre.data_ptr(), ldp, code, rows, inner, outer, a,
          None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
          None if db is None else db.data_ptr())
    return dx, dw, db


def _places(idx, rows, device):
    """(count, per_row) of a selection's positions: 1-D flat ones, or (rows, k) row-local ones."""
    if not isinstance(idx, torch.Tensor) or idx.dtype is not torch.int64 or idx.device != device:
        raise TypeError("idx must be an int64 tensor on %s" % device)
    if not idx.is_contiguous():
        raise ValueError("idx must be contiguous")
    if idx.dim() == 1:
        return idx.shape[0], 0
    if idx.dim() != 2 or idx.shape[0] != rows:
        raise ValueError("idx must be 1-D (flat positions) or (rows, k) with %d rows" % rows)
    return idx.shape[1], 1


def _of_places(t, idx, dtype, device, name):
    _like(t, dtype, device, name)
    if t.shape != idx.shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous with idx's shape %s" % (name, tuple(idx.shape)))
    return t.data_ptr()


def linear_backward_selected(dvals, vals, idx, x, w, act: str = "relu", need=(True, True, True), stream=None):
    """(dx, dw, dbias) of linear when only the selected outputs carry a gradient.

    dvals, vals: gradient and value at each selected place; idx: flat positions (1-D, from select_global) or
    row-local ones ((rows, k), from select); act: "relu" or "none".  None where `need` is false."""
    code = _first(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (rows, inner)")
    rows, inner = x.shape
    dtype, device = x.dtype, x.device
    _like(w, dtype, device, "w")
    outer = w.shape[0]
    ldx, ldw = _matrix(x, rows, inner, "x"), _matrix(w, outer, inner, "w")
    count, per_row = _places(idx, rows, device)
    pd, pv = _of_places(dvals, idx, dtype, device, "dvals"), _of_places(vals, idx, dtype, device, "vals")
    dx = _empty((rows, inner), dtype, device, stream) if need[0] else None
    dw = _empty((outer, inner), dtype, device, stream) if need[1] else None
    db = _empty((outer,), dtype, device, stream) if need[2] else None
    _call("topk_linear_backward_selected", device, stream, (dvals, vals, idx, x, w, dx, dw, db), pd, pv,
          idx.data_ptr(), count, per_row, x.data_ptr(), ldx, w.data_ptr(), ldw, code, rows, inner, outer, _act(act),
          None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
          None if db is None else db.data_ptr())
    return dx, dw, db


def decode(vals, idx, w, rows: int, bias=None, stream=None):
    """Reconstruction (rows, d): y[r] = bias + sum of vals_s w[c_s] over row r's selected places; w is (n, d)."""
    code = _first(w)
    if w.dim() != 2:
        raise ValueError("w must be 2-D (n, d)")
    n, d = w.shape
    dtype, device = w.dtype, w.device
    ldw = _matrix(w, n, d, "w")
    count, per_row = _places(idx, rows, device)
    pv = _of_places(vals, idx, dtype, device, "vals")
    pb = None if bias is None else _vector(bias, dtype, device, d, "bias")
    y = _empty((rows, d), dtype, device, stream)
    _call("topk_decode", device, stream, (vals, idx, w, bias, y), pv, idx.data_ptr(), count, per_row, w.data_ptr(), ldw,
          pb, code, rows, n, d, y.data_ptr())
    return y


def decode_backward(dy, vals, idx, w, need=(True, True, True), stream=None):
    """(dvals, dw, dbias) of decode from dy (rows, d); None where `need` is false."""
    code = _first(dy)
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D (rows, d)")
    rows, d = dy.shape
    dtype, device = dy.dtype, dy.device
    _like(w, dtype, device, "w")
    n = w.shape[0]
    lddy, ldw = _matrix(dy, rows, d, "dy"), _matrix(w, n, d, "w")
    count, per_row = _places(idx, rows, device)
    pv = _of_places(vals, idx, dtype, device, "vals")
    dv = _empty(vals.shape, dtype, device, stream) if need[0] else None
    dw = _empty((n, d), dtype, device, stream) if need[1] else None
    db = _empty((d,), dtype, device, stream) if need[2] else None
    _call("topk_decode_backward", device, stream, (dy, vals, idx, w, dv, dw, db), dy.data_ptr(), lddy, pv,
          idx.data_ptr(), count, per_row, w.data_ptr(), ldw, code, rows, n, d, None if dv is None else dv.data_ptr(),
          None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr())
    return dv, dw, db


_ARRAYS = {}


def _table(tensors, name):
    """(pointers, counts, dtypes) of contiguous tensors on one device, as the host arrays the library reads."""
    num = len(tensors)
    arrays = _ARRAYS.get(num)
    if arrays is None:
        arrays = _ARRAYS[num] = (ctypes.c_void_p * num, ctypes.c_int64 * num, ctypes.c_int * num)
    where, codes, ptrs, counts = tensors[0].get_device() if num else -1, [], [], []
    for t in tensors:
        code = _CODES.get(t.dtype)
        if code is None or t.get_device() != where or where < 0:
            _first(t)
            raise TypeError("%s must lie on one device" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        codes.append(code)
        ptrs.append(t.data_ptr())
        counts.append(t.numel())
    return arrays[0](*ptrs), arrays[1](*counts), arrays[2](*codes)


def _norm(tensors, max_norm, out, stream):
    """out None: in place (max_norm None: the norm alone)."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("needs at least one tensor")
    ptrs, counts, codes = _table(tensors, "tensors")
    device = tensors[0].device
    norm = _empty((), torch.float32, device, stream)
    if max_norm is None:
        _call("topk_grad_norm", device, stream, (*tensors, norm), ptrs, counts, codes, len(tensors), norm.data_ptr())
        return norm
    if out is None:
        outs, out = ptrs, ()
    else:
        out = list(out)
        outs, out_counts, out_codes = _table(out, "out")
        if out_counts[:] != counts[:] or out_codes[:] != codes[:] or (out and out[0].device != device):
            raise ValueError("out must match the tensors' sizes, dtypes and device")
    _call("topk_clip_grad_norm", device, stream, (*tensors, *out, norm), ptrs, outs, counts, codes, len(tensors),
          float(max_norm), norm.data_ptr())
    return norm


def grad_norm(tensors, stream=None):
    """The norm of the tensors taken as one vector: a float32 scalar on their device."""
    return _norm(tensors, None, None, stream)


def clip_grad_norm(tensors, max_norm: float, out, stream=None):
    """Writes tensors * min(1, max_norm / (norm + 1e-6)) to the tensors of `out`; returns the norm before that."""
    if out is None:
        raise ValueError("out must be a list of tensors (clip_grad_norm_ works in place)")
    return _norm(tensors, max_norm, out, stream)


def clip_grad_norm_(tensors, max_norm: float, stream=None):
    """clip_grad_norm in place."""
    return _norm(tensors, max_norm, None, stream)
