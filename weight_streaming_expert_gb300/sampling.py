"""Python face of include/sampling.h: the next token of each row of logits.
Argument marshalling only: the work runs in the library's kernel."""
from __future__ import annotations

import torch

from . import native as N
from .attention import _elsewhere, _On, _plain


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, return_probs: bool = False,
           stream=None):
    """logits fp32 [M, V] (as ``LmHead`` returns them; rows may be strided), u
    fp32 [M] in [0, 1).  temperature, top_p, min_p fp32 [M] and top_k int32 [M],
    each or None (off): <= 0 is greedy for the temperature and off for top_k
    and min_p, top_p >= 1 is off.  Returns int32 tokens [M] (-1 for a row
    without a logit above -inf), with ``return_probs`` also each token's
    probability among those that stayed, fp32 [M]."""
    index = logits.get_device()
    if index < 0 or logits.dim() != 2 or logits.dtype != torch.float32 or logits.stride(1) != 1:
        raise ValueError("logits must be an fp32 CUDA tensor [rows, vocab] with contiguous rows")
    if _elsewhere(index, stream):
        with _On(index, stream):
            return _sample(index, logits, u, temperature, top_k, top_p, min_p, tokens, return_probs)
    return _sample(index, logits, u, temperature, top_k, top_p, min_p, tokens, return_probs)


def _sample(index, logits, u, temperature, top_k, top_p, min_p, tokens, return_probs):
    M, V = logits.shape
    dev = logits.device
    _plain("u", u, torch.float32, index, M)
    for name, t, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if t is not None:
            _plain(name, t, dt, index, M)
    if tokens is None:
        tokens = torch.empty(M, dtype=torch.int32, device=dev)
    else:
        _plain("tokens", tokens, torch.int32, index, M)
    probs = torch.empty(M, dtype=torch.float32, device=dev) if return_probs else None
    status = N.lib().moe_sample(
        logits.data_ptr(), logits.stride(0), M, V, u.data_ptr(),
        None if temperature is None else temperature.data_ptr(), None if top_k is None else top_k.data_ptr(),
        None if top_p is None else top_p.data_ptr(), None if min_p is None else min_p.data_ptr(), tokens.data_ptr(), None if probs is None else probs.data_ptr(),
        torch._C._cuda_getCurrentRawStream(index))
    if status:
        N.check("moe_sample", status)
    return (tokens, probs) if return_probs else tokens
