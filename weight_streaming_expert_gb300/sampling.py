"""Python face of include/sampling.h: penalties, biases and grammar masks on
the logits (``adjust_logits``) and the next token of each row (``sample``).
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


def adjust_logits(logits, history=None, spans=None, repetition=None, presence=None, frequency=None, bias_ids=None,
                  bias_values=None, bias_starts=None, allowed=None, out=None, stream=None):
    """What stands between the logits and the draw.  logits fp32 [M, V], rows
    may be strided.  Each argument or None (left out):

    history int32 [n] and spans int32 [M, 3]: row m's tokens are
    history[begin:end], those from ``answer`` on its own answer, with (begin,
    answer, end) = spans[m]; rows may share them (drafts of one sequence see one
    token more from row to row).  Tokens of either kind are divided by
    repetition[m] where above 0, else multiplied with it; those of the answer
    lose frequency[m] for each time and presence[m] once (fp32 [M]).
    bias_ids int32 [k], bias_values fp32 [k], bias_starts int32 [M + 1]: row m
    adds the entries bias_starts[m] .. bias_starts[m + 1] - 1; of several for a
    token the last holds.
    allowed int32 [M, ceil(V / 32)] (rows may be one, expanded): where bit v % 32
    of word v // 32 is 0 token v becomes -inf.

    Returns out: a new tensor, or the given one, which may be logits itself
    (then only what changes is written)."""
    _tensor("logits", logits)
    index = logits.get_device()
    if index >= 0 and _elsewhere(index, stream):
        with _On(index, stream):
            return adjust_logits(logits, history, spans, repetition, presence, frequency, bias_ids, bias_values,
                                 bias_starts, allowed, out)
    got = N.calls().adjust_logits(torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0, logits, history, spans,
                                  repetition, presence, frequency, bias_ids, bias_values, bias_starts, allowed, out)
    if isinstance(got, int):
        if got < 0:
            _explain_adjust(index, logits, history, spans, repetition, presence, frequency, bias_ids, bias_values,
                            bias_starts, allowed, out)
        N.check("moe_adjust_logits", got)
    return got if out is None else out


def _explain_adjust(index, logits, history, spans, repetition, presence, frequency, bias_ids, bias_values, bias_starts,
                    allowed, out):
    def rows(name, t, dtype, what, columns):
        _tensor(name, t)
        if (t.dim() != 2 or t.dtype != dtype or t.get_device() != index or index < 0 or t.shape[0] != logits.shape[0]
                or t.shape[1] != columns or (columns > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name} must be {what} with contiguous rows on the logits' GPU")

    if logits.dim() != 2:
        raise ValueError("logits must be an fp32 CUDA tensor [rows, vocab]")
    M, V = logits.shape
    rows("logits", logits, torch.float32, "an fp32 CUDA tensor [rows, vocab]", V)
    if out is not None:
        rows("out", out, torch.float32, f"an fp32 tensor [{M}, {V}]", V)
    for name, t in (("repetition", repetition), ("presence", presence), ("frequency", frequency)):
        if t is not None:
            _plain(name, t, torch.float32, index, M)
    if history is not None or spans is not None:
        _tensor("history", history)
        _plain("history", history, torch.int32, index, history.numel())
        _tensor("spans", spans)
        _plain("spans", spans, torch.int32, index, M, 3)
    if bias_ids is not None or bias_values is not None or bias_starts is not None:
        _tensor("bias_ids", bias_ids)
        _plain("bias_ids", bias_ids, torch.int32, index, bias_ids.numel())
        _plain("bias_values", bias_values, torch.float32, index, bias_ids.numel())
        _plain("bias_starts", bias_starts, torch.int32, index, M + 1)
    if allowed is not None:
        rows("allowed", allowed, torch.int32, f"an int32 tensor [{M}, {-(-V // 32)}]", -(-V // 32))
    raise ValueError("an argument of adjust_logits has over 2^31 elements")
