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
kernels, stream= as there, nothing recorded for autograd.  The calls are checked and made by a compiled module
(csrc/language_calls.cpp): for a decoding step's they would take longer in Python than on the GPU.
"""
from __future__ import annotations

import os

import torch

from . import _lib

CALLS_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_language_calls.so")
_module = None


def _calls():
    """The compiled module; raises if it has not been built for this torch (there is no fallback)."""
    global _module
    if _module is None:
        _lib.get()
        try:
            from . import _language_calls
        except ImportError as e:
            why = "cannot be loaded (%s): was it built with another torch?  Run" % e if os.path.exists(CALLS_PATH) else "is not built; run"
            raise RuntimeError("_language_calls.so %s `python -m top_selection_prof_gb300.build`" % why) from e
        _module = _language_calls
    return _module


def _call(name, stream, *args):
    """The module's function on the current stream, or on `stream`: its inputs are then kept until it has run, its outputs
    are memory of that stream, kept for the current one too."""
    fn = getattr(_module or _calls(), name)
    if stream is None:
        out = fn(*args)
    else:
        if isinstance(args[0], torch.Tensor) and args[0].is_cuda and args[0].device != stream.device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, args[0].device))
        with torch.cuda.stream(stream):
            out = fn(*args)
        if type(out) is not int:
            for t in args:
                if isinstance(t, torch.Tensor):
                    t.record_stream(stream)
            for t in out if type(out) is tuple else (out,):
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(t.device))
    if type(out) is int:
        _lib.check(out, "topk_" + name)
    return out


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """(tokens, logprobs): a token of each row of logits (rows, n), drawn with u (rows,), float32 in [0, 1).

    Kept are the tokens that weigh at least min_p times the likeliest, of those the first top_k (0: all), of those the
    shortest prefix with a share of top_p; u then picks among them in the order of their logits (equal ones by index).
    temperature (0: the largest logit), top_k, top_p and min_p: numbers, or tensors with one value a row (float32;
    top_k int32).  NaN and -inf are never drawn; a row without anything else gives -1.  logprobs (float32): the logarithm
    of the token's share of what was kept."""
    return _call("sample", stream, logits, u, temperature, top_k, top_p, min_p)


def dispatch(x, idx, experts: int, stream=None):
    """(xs, place, offsets): the rows of x (tokens, d) in the order of their experts.

    idx (tokens, k), int64: each token's experts, as select gives them; one out of range (-1: dropped) has none.
    xs (tokens * k, d): the rows of expert e are xs[offsets[e]:offsets[e + 1]], in the order of their tokens; rows left over
    at the end are zeros.  place (tokens, k): each choice's row in xs, or -1.  offsets (experts + 1,): int64."""
    return _call("dispatch", stream, x, idx, experts)


def combine(ys, place, weights=None, stream=None):
    """y (tokens, d): y[t] = sum of weights[t, j] ys[place[t, j]] over j; places out of range add nothing.

    place (tokens, k) as from dispatch; weights (tokens, k) of ys's dtype, or None: all 1 (dispatch's gradient)."""
    return _call("combine", stream, ys, place, weights)


def combine_backward(dy, ys, place, weights=None, need=(True, True), stream=None):
    """(dys, dweights) of combine from dy (tokens, d); None where `need` is false."""
    return _call("combine_backward", stream, dy, ys, place, weights, *need)


def evict(keys, values, score, lengths, keep: int, recent: int = 0, weights=None, stream=None):
    """(keys, values, score, kept, lengths): a cache cut down to `keep` positions of each head.

    keys, values (batch, heads, capacity, dim); score (batch, heads, capacity), float32: the attention weight that each
    position has had; lengths (batch,), int64: the positions that hold tokens.  What stays: the last `recent` ones and
    those of the others with the largest scores (equal ones by position), in the order of their positions.
    weights (batch, query heads, queries, capacity), float32 or bfloat16: what the queries of each head's group gave,
    added first (a NaN counts as 0).  kept (batch, heads, keep): positions, -1 behind the new lengths, where rows and
    scores are zeros.  Nothing is changed in place."""
    return _call("evict", stream, keys, values, score, lengths, keep, recent, weights)


def replace_(keys, values, score, positions, lengths, key, value, recent: int = 0, weights=None, stream=None):
    """Puts one new token into each sequence's cache, in place; returns the slots (batch, heads) that it took.

    lengths (batch,): tokens before it.  While there are fewer than slots it takes the next one; then the one whose
    score is least, of those whose position is below lengths - recent (equal ones: the lowest slot; none: slot -1, and
    nothing is stored).  key, value (batch, heads, dim); positions (batch, heads, capacity), int64: the position in each
    slot; weights as in evict, by slot, added to the scores first.  The slot's score becomes 0.  lengths is not changed.
    As after torch's in-place operators, a backward pass that saved one of the four tensors before raises an error."""
    return _call("replace", stream, keys, values, score, positions, lengths, key, value, recent, weights)
