"""Python face of include/sampling.h: the next token of each row of logits.
Argument marshalling only: the work runs in the library's kernel."""
from __future__ import annotations

import torch

from . import native as N
from .attention import _on, _plain
from .layer import _ptr, _stream_ptr


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None, return_probs: bool = False,
           stream=None):
    """logits fp32 [M, V] (as ``LmHead`` returns them; rows may be strided), u
    fp32 [M] in [0, 1).  temperature, top_p, min_p fp32 [M] and top_k int32 [M],
    each or None (off): <= 0 is greedy for the temperature and off for top_k
    and min_p, top_p >= 1 is off.  Returns int32 tokens [M] (-1 for a row
    without a logit above -inf), with ``return_probs`` also each token's
    probability among those that stayed, fp32 [M]."""
    if logits.dim() != 2 or logits.dtype != torch.float32 or not logits.is_cuda or logits.stride(1) != 1:
        raise ValueError("logits must be an fp32 CUDA tensor [rows, vocab] with contiguous rows")
    M, V = logits.shape
    dev = logits.device
    _plain("u", u, torch.float32, dev, M)
    for name, t, dt in (("temperature", temperature, torch.float32), ("top_k", top_k, torch.int32),
                        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32)):
        if t is not None:
            _plain(name, t, dt, dev, M)
    probs = None
    with _on(dev, stream):
        if tokens is None:
            tokens = torch.empty(M, dtype=torch.int32, device=dev)
        else:
            _plain("tokens", tokens, torch.int32, dev, M)
        if return_probs:
            probs = torch.empty(M, dtype=torch.float32, device=dev)
        N.check("moe_sample", N.lib().moe_sample(_ptr(logits), logits.stride(0), M, V, _ptr(u), _ptr(temperature),
                                                 _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(tokens), _ptr(probs),
                                                 _stream_ptr(stream)))
    return (tokens, probs) if return_probs else tokens
