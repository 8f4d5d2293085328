"""Operators of a language model around the selection (include/topk.h).

    tokens, logprobs = tk.sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)   # u: one random number a row

    vals, idx = tk.select(router_logits, k)                       # k experts a token
    xs, place, offsets = tk.dispatch(x, idx, experts)             # expert e: xs[offsets[e]:offsets[e + 1]]
    y = tk.combine(ys, place, weights)                            # the way back
    dys, dweights = tk.combine_backward(dy, ys, place, weights)
    dx = tk.combine(dxs, place)                                   # dispatch's gradient

    keys, values, score, kept, lengths = tk.evict(keys, values, score, lengths, keep, recent=64, weights=attention)
    slots = tk.replace_(keys, values, score, positions, lengths, key, value, recent=64, weights=attention)

As in operators.py: float32 or bfloat16 CUDA tensors with contiguous last dimensions, every step in the library's
kernels, stream= as there, nothing recorded for autograd.
"""
from __future__ import annotations

import struct

import torch

from .operators import _CODES, _call, _empty, _first, _like, _matrix, _of_places, _vector

_F32, _I64 = torch.float32, torch.int64
_VIEW = struct.Struct("4q").pack    # a topk_view_t


def _by_row(v, dtype, device, rows, name):
    """(number, pointer) of a parameter that is a number or a tensor with one value a row."""
    if isinstance(v, torch.Tensor):
        return 0, _vector(v, dtype, device, rows, name)
    return v, None


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """(tokens, logprobs): a token of each row of logits (rows, n), drawn with u (rows,), float32 in [0, 1).

    Kept are the tokens that weigh at least min_p times the likeliest, of those the first top_k (0: all), of those the
    shortest prefix with a share of top_p; u then picks among them in the order of their logits (equal ones by index).
    temperature (0: the largest logit), top_k, top_p and min_p: numbers, or tensors with one value a row (float32;
    top_k int32).  NaN and -inf are never drawn; a row without anything else gives -1.  logprobs (float32): the logarithm
    of the token's share of what was kept."""
    code = _first(logits)
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D (rows, n)")
    rows, n = logits.shape
    device = logits.device
    ld = _matrix(logits, rows, n, "logits")
    pu = _vector(u, _F32, device, rows, "u")
    t, pt = _by_row(temperature, _F32, device, rows, "temperature")
    k, pk = _by_row(top_k, torch.int32, device, rows, "top_k")
    p, pp = _by_row(top_p, _F32, device, rows, "top_p")
    m, pm = _by_row(min_p, _F32, device, rows, "min_p")
    tokens = _empty((rows,), _I64, device, stream)
    logprobs = _empty((rows,), _F32, device, stream)
    used = (logits, u, temperature if pt else None, top_k if pk else None, top_p if pp else None, min_p if pm else None, tokens, logprobs)
    _call("topk_sample", device, stream, used, logits.data_ptr(), ld, code, rows, n, pu, t, pt, k, pk, p, pp, m, pm,
          tokens.data_ptr(), logprobs.data_ptr())
    return tokens, logprobs


def _choices(t, tokens, device, name):
    """k of an int64 tensor (tokens, k)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I64 or t.device != device:
        raise TypeError("%s must be an int64 tensor on %s" % (name, device))
    shape = t.shape
    if len(shape) != 2 or (tokens is not None and shape[0] != tokens) or shape[1] < 1 or not t.is_contiguous():
        raise ValueError("%s must be contiguous with shape (tokens, k), k >= 1, got %s" % (name, tuple(shape)))
    return shape[1]


def dispatch(x, idx, experts: int, stream=None):
    """(xs, place, offsets): the rows of x (tokens, d) in the order of their experts.

    idx (tokens, k), int64: each token's experts, as select gives them; one out of range (-1: dropped) has none.
    xs (tokens * k, d): the rows of expert e are xs[offsets[e]:offsets[e + 1]], in the order of their tokens; rows left over
    at the end are zeros.  place (tokens, k): each choice's row in xs, or -1.  offsets (experts + 1,): int64."""
    code = _first(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D (tokens, d)")
    tokens, d = x.shape
    dtype, device = x.dtype, x.device
    ldx = _matrix(x, tokens, d, "x")
    k = _choices(idx, tokens, device, "idx")
    xs = _empty((tokens * k, d), dtype, device, stream)
    place = _empty((tokens, k), _I64, device, stream)
    offsets = _empty((max(experts, 0) + 1,), _I64, device, stream)
    _call("topk_dispatch", device, stream, (x, idx, xs, place, offsets), x.data_ptr(), ldx, idx.data_ptr(), code, tokens, k,
          experts, d, xs.data_ptr(), place.data_ptr(), offsets.data_ptr())
    return xs, place, offsets


def combine(ys, place, weights=None, stream=None):
    """y (tokens, d): y[t] = sum of weights[t, j] ys[place[t, j]] over j; places out of range add nothing.

    place (tokens, k) as from dispatch; weights (tokens, k) of ys's dtype, or None: all 1 (dispatch's gradient)."""
    code = _first(ys)
    if ys.dim() != 2:
        raise ValueError("ys must be 2-D (rows, d)")
    rows, d = ys.shape
    dtype, device = ys.dtype, ys.device
    ldys = _matrix(ys, rows, d, "ys")
    k = _choices(place, None, device, "place")
    pw = None if weights is None else _of_places(weights, place, dtype, device, "weights")
    y = _empty((place.shape[0], d), dtype, device, stream)
    _call("topk_combine", device, stream, (ys, place, weights, y), ys.data_ptr(), ldys, rows, place.data_ptr(), pw, code,
          place.shape[0], k, d, y.data_ptr())
    return y


def combine_backward(dy, ys, place, weights=None, need=(True, True), stream=None):
    """(dys, dweights) of combine from dy (tokens, d); None where `need` is false."""
    code = _first(dy)
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D (tokens, d)")
    tokens, d = dy.shape
    dtype, device = dy.dtype, dy.device
    _like(ys, dtype, device, "ys")
    if ys.dim() != 2:
        raise ValueError("ys must be 2-D (rows, d)")
    rows = ys.shape[0]
    lddy, ldys = _matrix(dy, tokens, d, "dy"), _matrix(ys, rows, d, "ys")
    k = _choices(place, tokens, device, "place")
    pw = None if weights is None else _of_places(weights, place, dtype, device, "weights")
    dys = _empty((rows, d), dtype, device, stream) if need[0] else None
    dw = _empty((tokens, k), dtype, device, stream) if need[1] else None
    _call("topk_combine_backward", device, stream, (dy, ys, place, weights, dys, dw), dy.data_ptr(), lddy, ys.data_ptr(), ldys,
          rows, place.data_ptr(), pw, code, tokens, k, d, None if dys is None else dys.data_ptr(),
          None if dw is None else dw.data_ptr())
    return dys, dw


def _view(t, dtype, index, shape, name):
    """A topk_view_t of a tensor (batch, heads, rows, values), or without the dimension of rows, whose values are contiguous."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        raise TypeError("%s must be a %s tensor on cuda:%d" % (name, dtype, index))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    by = t.stride()
    if by[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must be contiguous along its last dimension" % name)
    return _VIEW(t.data_ptr(), by[0], by[1], by[2])


def _cache(keys, values, score, lengths, weights):
    """Checks what evict and replace_ have in common: ((batch, heads, capacity, key dim, value dim), dtype, device index, views of
    keys, values and score, lengths' pointer, (weights' view, dtype, group, queries, the cache's dtype))."""
    code = _first(keys)
    shape = keys.shape
    if len(shape) != 4:
        raise ValueError("keys must be 4-D (batch, heads, capacity, dim)")
    batch, heads, capacity, kd = shape
    dtype, index = keys.dtype, keys.get_device()
    if not isinstance(values, torch.Tensor) or values.dim() != 4:
        raise ValueError("values must be 4-D (batch, heads, capacity, dim)")
    vd = values.shape[3]
    views = (_view(keys, dtype, index, shape, "keys"), _view(values, dtype, index, (batch, heads, capacity, vd), "values"),
             _view(score, _F32, index, (batch, heads, capacity), "score"))
    if not isinstance(lengths, torch.Tensor) or lengths.dtype is not _I64 or lengths.get_device() != index:
        raise TypeError("lengths must be an int64 tensor on cuda:%d" % index)
    if lengths.shape != (batch,) or not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous with %d values" % batch)
    if weights is None:
        added = None, code, 1, 0, code
    else:
        if not isinstance(weights, torch.Tensor) or weights.dtype not in _CODES or weights.dim() != 4:
            raise TypeError("weights must be a 4-D float32 or bfloat16 tensor (batch, query heads, queries, capacity)")
        _, query_heads, queries, _ = weights.shape
        if query_heads < heads or query_heads % heads:
            raise ValueError("weights must have a multiple of the cache's %d heads, got %d" % (heads, query_heads))
        view = _view(weights, weights.dtype, index, (batch, query_heads, queries, capacity), "weights")
        added = view, _CODES[weights.dtype], query_heads // heads, queries, code
    return (batch, heads, capacity, kd, vd), dtype, index, views, lengths.data_ptr(), added


def evict(keys, values, score, lengths, keep: int, recent: int = 0, weights=None, stream=None):
    """(keys, values, score, kept, lengths): a cache cut down to `keep` positions of each head.

    keys, values (batch, heads, capacity, dim); score (batch, heads, capacity), float32: the attention weight that each
    position has had; lengths (batch,), int64: the positions that hold tokens.  What stays: the last `recent` ones and
    those of the others with the largest scores (equal ones by position), in the order of their positions.
    weights (batch, query heads, queries, capacity), float32 or bfloat16: what the queries of each head's group gave,
    added first (a NaN counts as 0).  kept (batch, heads, keep): positions, -1 behind the new lengths, where rows and
    scores are zeros.  Nothing is changed in place."""
    sizes, dtype, _, views, pl, added = _cache(keys, values, score, lengths, weights)
    batch, heads, _, kd, vd = sizes
    device, rows = keys.device, max(keep, 0)
    ok, ov = _empty((batch, heads, rows, kd), dtype, device, stream), _empty((batch, heads, rows, vd), dtype, device, stream)
    osc, kept = _empty((batch, heads, rows), _F32, device, stream), _empty((batch, heads, rows), _I64, device, stream)
    ol = _empty((batch,), _I64, device, stream)
    _call("topk_evict", device, stream, (keys, values, score, lengths, weights, ok, ov, osc, kept, ol), *views, pl, *added, *sizes,
          keep, recent, ok.data_ptr(), ov.data_ptr(), osc.data_ptr(), kept.data_ptr(), ol.data_ptr())
    return ok, ov, osc, kept, ol


def replace_(keys, values, score, positions, lengths, key, value, recent: int = 0, weights=None, stream=None):
    """Puts one new token into each sequence's cache, in place; returns the slots (batch, heads) that it took.

    lengths (batch,): tokens before it.  While there are fewer than slots it takes the next one; then the one whose
    score is least, of those that hold positions before the last `recent` (equal ones: the lowest slot).  key, value
    (batch, heads, dim); positions (batch, heads, capacity), int64: the position in each slot; weights as in evict, by slot,
    added to the scores first.  The slot's score becomes 0.  lengths is not changed."""
    sizes, dtype, index, views, pl, added = _cache(keys, values, score, lengths, weights)
    batch, heads, capacity, kd, vd = sizes
    device = keys.device
    at = _view(positions, _I64, index, (batch, heads, capacity), "positions")
    k, v = _view(key, dtype, index, (batch, heads, kd), "key"), _view(value, dtype, index, (batch, heads, vd), "value")
    slots = _empty((batch, heads), _I64, device, stream)
    _call("topk_replace", device, stream, (keys, values, score, positions, lengths, key, value, weights, slots), *views, at, pl, k, v,
          *added, *sizes, recent, slots.data_ptr())
    return slots
