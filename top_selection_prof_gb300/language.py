"""Operators of a language model around the selection (include/topk.h).

    tokens, logprobs = tk.sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)   # u: one random number a row

As in operators.py: float32 or bfloat16 CUDA tensors with contiguous last dimensions, every step in the library's
kernels, stream= as there, nothing recorded for autograd.
"""
from __future__ import annotations

import torch

from .operators import _call, _empty, _first, _matrix, _vector


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
    f32 = torch.float32
    pu = _vector(u, f32, device, rows, "u")
    t, pt = _by_row(temperature, f32, device, rows, "temperature")
    k, pk = _by_row(top_k, torch.int32, device, rows, "top_k")
    p, pp = _by_row(top_p, f32, device, rows, "top_p")
    m, pm = _by_row(min_p, f32, device, rows, "min_p")
    tokens = _empty((rows,), torch.int64, device, stream)
    logprobs = _empty((rows,), f32, device, stream)
    _call("topk_sample", device, stream, (logits, u, *(v for v in (temperature, top_k, top_p, min_p) if isinstance(v, torch.Tensor)),
                                          tokens, logprobs), logits.data_ptr(), ld, code, rows, n, pu, t, pt, k, pk, p, pp, m, pm,
          tokens.data_ptr(), logprobs.data_ptr())
    return tokens, logprobs
