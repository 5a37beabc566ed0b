"""Python face of include/attention.h: norms and rotation of queries and keys
into the paged cache (``QKNormRope``) and attention of new tokens over it
(``PagedAttention``).  The arguments are looked over and passed on by the
extension module (csrc/python_calls.cpp); where it finds that one does not fit,
this side says which.  Nothing here is differentiable."""
from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import torch

from . import native as N

_DTYPES = {torch.bfloat16: N.MOE_DTYPE_BF16, torch.float16: N.MOE_DTYPE_FP16}
_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")

class _On:
    """Device and stream of a call that are not the current ones: outputs are
    allocated, and the kernel is launched, inside."""

    def __init__(self, index, stream):
        self._contexts = [torch.cuda.device(index)] + ([] if stream is None else [torch.cuda.stream(stream)])

    def __enter__(self):
        for c in self._contexts:
            c.__enter__()

    def __exit__(self, *e):
        for c in reversed(self._contexts):
            c.__exit__(*e)


def _elsewhere(index, stream):
    """Whether a call on GPU `index` and `stream` needs `_On`."""
    return stream is not None or torch._C._cuda_getDevice() != index


def _tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, not {type(t).__name__}")


def _heads(name, t, dtype, index, dim):
    """t: [tokens, heads, dim], each head's values contiguous."""
    _tensor(name, t)
    if t.dim() != 3 or t.dtype != dtype or t.get_device() != index or t.shape[2] != dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor [tokens, heads, {dim}] with contiguous heads on "
                         f"cuda:{index}")


def _cache(name, t, dtype, index, heads, dim):
    """t: [pages, page_size, heads, dim], each row contiguous."""
    _tensor(name, t)
    if (t.dim() != 4 or t.dtype != dtype or t.get_device() != index or t.shape[2:] != (heads, dim)
            or t.stride()[2:] != (dim, 1)):
        raise ValueError(f"{name} must be a {dtype} tensor [pages, page_size, {heads}, {dim}] with contiguous rows "
                         f"on cuda:{index}")


def _scale(name, t, cache, index):
    """t: the scale bytes of a quantised cache [pages, page_size, heads, dim]."""
    _tensor(name, t)
    pages, page_size, heads = cache.shape[:3]
    if (t.dtype != torch.uint8 or t.get_device() != index or t.shape != (pages, heads, page_size)
            or (page_size > 1 and t.stride(2) != 1)):
        raise ValueError(f"{name} must be a uint8 tensor [{pages}, {heads}, {page_size}] with contiguous rows on "
                         f"cuda:{index}")


def _caches(k_cache, v_cache, k_scale, v_scale, dtype, index, heads, dim):
    """The caches of one layer: of `dtype`, or with scales of E4M3 codes."""
    if k_scale is not None or v_scale is not None:
        dtype = torch.float8_e4m3fn
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _cache(name, t, dtype, index, heads, dim)
    if k_scale is not None or v_scale is not None:
        for name, t, cache in (("k_scale", k_scale, k_cache), ("v_scale", v_scale, v_cache)):
            _scale(name, t, cache, index)


def _plain(name, t, dtype, index, *shape):
    _tensor(name, t)
    if t.dtype != dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{index}")


class QKNormRope:
    """RMS norm of every query and key head, then the rotation of its first
    ``rotary_dim`` values, with keys and values written into the cache.

    Pair i turns by position * inv_freq[i] (default: theta ** (-2i /
    rotary_dim)); pairs are (i, i + rotary_dim / 2), or with ``interleaved``
    (2i, 2i + 1).  Angles are exact modulo a turn at any int32 position."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, theta: float = 10000.0, inv_freq=None,
                 interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        rotary_dim = head_dim if rotary_dim is None else int(rotary_dim)
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if rotary_dim % 16 or not 0 <= rotary_dim <= head_dim:
            raise ValueError("rotary_dim must be a multiple of 16, at most head_dim")
        if inv_freq is None:
            inv_freq = [float(theta) ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != rotary_dim // 2 or not all(map(math.isfinite, inv_freq)):
            raise ValueError("inv_freq must hold rotary_dim / 2 finite numbers")
        self.head_dim, self.rotary_dim, self.interleaved, self.eps = head_dim, rotary_dim, bool(interleaved), float(eps)
        # turns per position as whole parts of 2^64, as signed words
        turns = [round(Fraction(f) / _TWO_PI * (1 << 64)) % (1 << 64) for f in inv_freq]
        words = [t - (1 << 64) if t >> 63 else t for t in turns]
        self.turns = torch.tensor(words, dtype=torch.int64).to(device)
        self.device = self.turns.device
        self._index = self.turns.get_device()

    def forward(self, q, k, v, q_weight, k_weight, positions, slots, k_cache, v_cache, q_out=None, stream=None,
                k_scale=None, v_scale=None):
        """q [T, Hq, D], k and v [T, Hk, D] (views of one projection are fine),
        weights [D] or None, positions int32 [T], slots int64 [T] (a negative
        slot writes nothing), caches [pages, page_size, Hk, D].  Returns q_out
        (a new contiguous tensor, or the given one; it may be q).  With k_scale
        and v_scale (uint8 [pages, Hk, page_size]) the caches are quantised:
        float8_e4m3fn codes, a power of two for each row of a head; no slot may
        be in slots twice then."""
        index = self._index
        if index < 0:
            raise ValueError("the operator was made on the CPU: its calls need a GPU")
        if _elsewhere(index, stream):
            with _On(index, stream):
                return self.forward(q, k, v, q_weight, k_weight, positions, slots, k_cache, v_cache, q_out, None,
                                    k_scale, v_scale)
        got = N.calls().qk_norm_rope(index, torch._C._cuda_getCurrentRawStream(index), self.head_dim, self.rotary_dim,
                                     self.interleaved, self.eps, self.turns, q, k, v, q_weight, k_weight, positions,
                                     slots, k_cache, v_cache, q_out, k_scale, v_scale)
        if isinstance(got, int):
            if got < 0:
                self._explain(index, q, k, v, q_weight, k_weight, positions, slots, k_cache, v_cache, q_out, k_scale,
                              v_scale)
            N.check("moe_qk_norm_rope", got)
        return got if q_out is None else q_out

    def _explain(self, index, q, k, v, q_weight, k_weight, positions, slots, k_cache, v_cache, q_out, k_scale,
                 v_scale):
        _tensor("q", q)
        D, dt = self.head_dim, q.dtype
        if dt not in _DTYPES:
            raise ValueError("q must be bf16 or fp16")
        for name, t in (("q", q), ("k", k), ("v", v)) + ((("q_out", q_out),) if q_out is not None else ()):
            _heads(name, t, dt, index, D)
        _caches(k_cache, v_cache, k_scale, v_scale, dt, index, k.shape[1], D)
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            if t is not None:
                _plain(name, t, dt, index, D)
        _plain("positions", positions, torch.int32, index, q.shape[0])
        _plain("slots", slots, torch.int64, index, q.shape[0])
        raise ValueError("q, k, v, q_out and the caches must agree in tokens, heads and pages")

    __call__ = forward


class PagedAttention:
    """Attention of each sequence's new tokens over its pages of the cache
    (one ``moe_attn_t`` handle: one host thread and stream at a time)."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, device="cuda"):
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.device = torch.empty(0, device=device).device
        self._index = self.device.index
        with torch.cuda.device(self.device):
            h = N.lib().moe_attn_create(n_heads, n_kv_heads, head_dim)
        if not h:
            raise N.MoEError("moe_attn_create", N.MOE_ERR_INVALID_ARG, N.last_error())
        self._h = ctypes.c_void_p(h)
        self._handle = h

    def forward(self, q, k_cache, v_cache, block_table, q_starts, kv_lens, max_q_len: int, scale: float | None = None,
                tree_mask=None, out=None, return_lse: bool = False, stream=None, k_scale=None, v_scale=None,
                prefix_len: int = 0):
        """q [T, Hq, D]; caches [pages, page_size, Hk, D]; block_table int32
        [B, pages of a row] (a view of a wider table, or one row expanded, is
        fine); q_starts int32 [B + 1]; kv_lens int32 [B] (the new tokens
        included); max_q_len: at least the longest chunk, and the nearer to it
        the better a call is laid out; scale: default
        D ** -0.5; tree_mask: int64 [T], bit j of a token's word set where it
        sees its chunk's token j, instead of the chain (chunks up to 64).
        Returns out [T, Hq, D], with ``return_lse`` also fp32 [T, Hq].

        k_scale, v_scale (uint8 [pages, Hk, page_size]): the caches are
        quantised, float8_e4m3fn codes as ``QKNormRope`` writes them.  Chunks of
        more than 64 rows (tokens times heads that share one of the cache) are
        unpacked first, in a workspace that goes by the table's width: give a
        view as narrow as the longest sequence.
        prefix_len: every sequence begins with the same positions, as many, in
        the same whole pages (forks: ``PagedKVCache.shared_prefix``, which says
        from where it pays) and before all new tokens; they are then read once
        for the batch."""
        index = self._index
        if _elsewhere(index, stream):
            with _On(index, stream):
                return self.forward(q, k_cache, v_cache, block_table, q_starts, kv_lens, max_q_len, scale, tree_mask,
                                    out, return_lse, None, k_scale, v_scale, prefix_len)
        got = N.calls().attention(index, torch._C._cuda_getCurrentRawStream(index), self._handle, self.n_heads,
                                  self.n_kv_heads, self.head_dim, q, k_cache, v_cache, block_table, q_starts, kv_lens,
                                  max_q_len, self.head_dim ** -0.5 if scale is None else scale, tree_mask, out,
                                  return_lse, k_scale, v_scale, prefix_len)
        if isinstance(got, int):
            if got < 0:
                self._explain(q, k_cache, v_cache, block_table, q_starts, kv_lens, max_q_len, tree_mask, out, k_scale,
                              v_scale, prefix_len)
            N.check("moe_attn_forward", got)
        if out is None:
            return got
        return (out, got[1]) if return_lse else out

    def _explain(self, q, k_cache, v_cache, block_table, q_starts, kv_lens, max_q_len, tree_mask, out, k_scale, v_scale,
                 prefix_len):
        _tensor("q", q)
        index, D, dt = self._index, self.head_dim, q.dtype
        if dt not in _DTYPES or q.dim() != 3 or q.shape[1] != self.n_heads:
            raise ValueError(f"q must be a bf16 or fp16 tensor [tokens, {self.n_heads}, {D}]")
        _heads("q", q, dt, index, D)
        _caches(k_cache, v_cache, k_scale, v_scale, dt, index, self.n_kv_heads, D)
        if not isinstance(prefix_len, int) or not 0 <= prefix_len < 1 << 31:
            raise ValueError("prefix_len must be an int of 0 or more")
        _tensor("block_table", block_table)
        if (block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.get_device() != index
                or block_table.stride(1) != 1):
            raise ValueError(f"block_table must be an int32 tensor [batch, pages] with contiguous rows on cuda:{index}")
        B = block_table.shape[0]
        _plain("q_starts", q_starts, torch.int32, index, B + 1)
        _plain("kv_lens", kv_lens, torch.int32, index, B)
        if tree_mask is not None:
            _plain("tree_mask", tree_mask, torch.int64, index, q.shape[0])
        if out is not None:
            _heads("out", out, dt, index, D)
        raise ValueError("the caches must have one shape, out q's, max_q_len must be an int of 0 or more and scale a "
                         "number")

    __call__ = forward

    def status(self) -> int:
        """Synchronises; returns the sticky device status (0 = ok) and clears it."""
        return N.lib().moe_attn_get_status(self._h)

    def close(self):
        if getattr(self, "_h", None):
            N.lib().moe_attn_destroy(self._h)
            self._h, self._handle = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
