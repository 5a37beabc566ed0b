"""Python face of include/sampling.h: the next token of each row of logits.
The arguments are looked over and passed on by the extension module
(csrc/python_calls.cpp)."""
from __future__ import annotations

import torch

from . import native as N
from .attention import _elsewhere, _On, _plain, _tensor


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, return_probs: bool = False,
           stream=None):
    """logits fp32 [M, V] (as ``LmHead`` returns them; rows may be strided), u
    fp32 [M] in [0, 1).  temperature, top_p, min_p fp32 [M] and top_k int32 [M],
    each or None (off): <= 0 is greedy for the temperature and off for top_k
    and min_p, top_p >= 1 is off.  Returns int32 tokens [M] (-1 for a row
    without a logit above -inf), with ``return_probs`` also each token's
    probability among those that stayed, fp32 [M]."""
    _tensor("logits", logits)
    index = logits.get_device()
    if index >= 0 and _elsewhere(index, stream):
        with _On(index, stream):
            return sample(logits, u, temperature, top_k, top_p, min_p, tokens, return_probs)
    got = N.calls().sample(torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0, logits, u, temperature,
                           top_k, top_p, min_p, tokens, return_probs)
    if isinstance(got, int):
        if got < 0:
            _explain(index, logits, u, temperature, top_k, top_p, min_p, tokens)
        N.check("moe_sample", got)
    if tokens is None:
        return got
    return (tokens, got[1]) if return_probs else tokens


def _explain(index, logits, u, temperature, top_k, top_p, min_p, tokens):
    if (index < 0 or logits.dim() != 2 or logits.dtype != torch.float32
            or (logits.shape[1] > 1 and logits.stride(1) != 1)):
        raise ValueError("logits must be an fp32 CUDA tensor [rows, vocab] with contiguous rows")
    M = logits.shape[0]
    for name, t, dt in (("u", u, torch.float32), ("temperature", temperature, torch.float32),
                        ("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32),
                        ("min_p", min_p, torch.float32), ("tokens", tokens, torch.int32)):
        if t is not None or name == "u":
            _plain(name, t, dt, index, M)
    raise ValueError("an argument of sample is not a tensor, or has over 2^31 elements")
