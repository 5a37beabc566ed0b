"""Python face of include/attention.h: norms and rotation of queries and keys
into the paged cache (``QKNormRope``) and attention of new tokens over it
(``PagedAttention``).  Argument marshalling only: the work runs in the
library's kernels.  Nothing here is differentiable."""
from __future__ import annotations

import contextlib
import ctypes
import math
from fractions import Fraction

import torch

from . import native as N
from .layer import _ptr, _stream_ptr

_DTYPES = {torch.bfloat16: N.MOE_DTYPE_BF16, torch.float16: N.MOE_DTYPE_FP16}
_NO_CONTEXT = contextlib.nullcontext()
_TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def _on(device, stream):
    """Context in which outputs are allocated: the call's device and stream, so
    that the allocator orders their reuse after the kernel."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.type != "cuda":
        return _NO_CONTEXT
    return _NO_CONTEXT if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _heads(name, t, dtype, device, dim):
    """t: [tokens, heads, dim], each head's values contiguous."""
    if t.dim() != 3 or t.dtype != dtype or t.device != device or t.shape[2] != dim or (t.stride(2) != 1 and dim > 1):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [tokens, heads, {dim}] with contiguous heads")


def _cache(name, t, dtype, device, dim):
    """t: [pages, page_size, kv_heads, dim], each row contiguous."""
    if (t.dim() != 4 or t.dtype != dtype or t.device != device or t.shape[3] != dim or t.stride(3) != 1
            or (t.shape[2] > 1 and t.stride(2) != dim)):
        raise ValueError(f"{name} must be a {dtype} CUDA tensor [pages, page_size, kv_heads, {dim}] with contiguous rows")


def _plain(name, t, dtype, device, *shape):
    if t.dtype != dtype or t.device != device or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {list(shape)}")


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
        device = torch.device(device)
        self.turns = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.device = self.turns.device

    def forward(self, q, k, v, q_weight, k_weight, positions, slots, k_cache, v_cache, q_out=None, stream=None):
        """q [T, Hq, D], k and v [T, Hk, D] (views of one projection are fine),
        weights [D] or None, positions int32 [T], slots int64 [T] (a negative
        slot writes nothing), caches [pages, page_size, Hk, D].  Returns q_out
        (a new contiguous tensor, or the given one; it may be q)."""
        T, Hq, D = q.shape
        dt, dev = q.dtype, q.device
        if dt not in _DTYPES or dev != self.device or D != self.head_dim:
            raise ValueError(f"q must be a bf16 or fp16 tensor [tokens, heads, {self.head_dim}] on {self.device}")
        _heads("q", q, dt, dev, D)
        _heads("k", k, dt, dev, D)
        _heads("v", v, dt, dev, D)
        _cache("k_cache", k_cache, dt, dev, D)
        _cache("v_cache", v_cache, dt, dev, D)
        Hk = k.shape[1]
        if k.shape != v.shape or k.shape[0] != T or k_cache.shape != v_cache.shape or k_cache.shape[2] != Hk:
            raise ValueError("q, k, v and the caches must agree in tokens and heads")
        for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
            if w is not None:
                _plain(name, w, dt, dev, D)
        _plain("positions", positions, torch.int32, dev, T)
        _plain("slots", slots, torch.int64, dev, T)
        with _on(dev, stream):
            if q_out is None:
                q_out = torch.empty((T, Hq, D), dtype=dt, device=dev)
            else:
                _heads("q_out", q_out, dt, dev, D)
                if q_out.shape != q.shape:
                    raise ValueError("q_out must have q's shape")
            a = N.moe_qk_norm_rope_args_t(
                _DTYPES[dt], T, Hq, Hk, D, self.rotary_dim, self.interleaved, self.eps, q.data_ptr(), k.data_ptr(),
                v.data_ptr(), q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                None if q_weight is None else q_weight.data_ptr(), None if k_weight is None else k_weight.data_ptr(),
                self.turns.data_ptr(), positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(), q_out.stride(0),
                q_out.stride(1), k_cache.data_ptr(), v_cache.data_ptr(), k_cache.stride(0), k_cache.stride(1),
                v_cache.stride(0), v_cache.stride(1), k_cache.shape[0], k_cache.shape[1])
            N.check("moe_qk_norm_rope", N.lib().moe_qk_norm_rope(ctypes.byref(a), _stream_ptr(stream)))
        return q_out

    __call__ = forward


class PagedAttention:
    """Attention of each sequence's new tokens over its pages of the cache
    (one ``moe_attn_t`` handle: one host thread and stream at a time)."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, device="cuda"):
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.device = torch.empty(0, device=device).device
        with torch.cuda.device(self.device):
            h = N.lib().moe_attn_create(n_heads, n_kv_heads, head_dim)
        if not h:
            raise N.MoEError("moe_attn_create", N.MOE_ERR_INVALID_ARG, N.last_error())
        self._h = ctypes.c_void_p(h)

    def forward(self, q, k_cache, v_cache, block_table, q_starts, kv_lens, max_q_len: int, scale: float | None = None,
                tree_mask=None, out=None, return_lse: bool = False, stream=None):
        """q [T, Hq, D]; caches [pages, page_size, Hk, D]; block_table int32
        [B, pages of a row]; q_starts int32 [B + 1]; kv_lens int32 [B] (the new
        tokens included); max_q_len: at least the longest chunk; scale: default
        D ** -0.5; tree_mask: int64 [T], bit j of a token's word set where it
        sees its chunk's token j, instead of the chain (chunks up to 64).
        Returns out [T, Hq, D], with ``return_lse`` also fp32 [T, Hq]."""
        T, Hq, D = q.shape
        dt, dev = q.dtype, q.device
        if dt not in _DTYPES or dev != self.device or Hq != self.n_heads or D != self.head_dim:
            raise ValueError(f"q must be a bf16 or fp16 tensor [tokens, {self.n_heads}, {self.head_dim}] on {self.device}")
        _heads("q", q, dt, dev, D)
        _cache("k_cache", k_cache, dt, dev, D)
        _cache("v_cache", v_cache, dt, dev, D)
        if k_cache.shape != v_cache.shape or k_cache.shape[2] != self.n_kv_heads:
            raise ValueError(f"the caches must have one shape, with {self.n_kv_heads} heads")
        if block_table.dim() != 2:
            raise ValueError("block_table must be [batch, pages]")
        B = block_table.shape[0]
        if block_table.dtype != torch.int32 or block_table.device != dev or block_table.stride(1) != 1:
            raise ValueError("block_table must be an int32 CUDA tensor [batch, pages] with contiguous rows")
        _plain("q_starts", q_starts, torch.int32, dev, B + 1)
        _plain("kv_lens", kv_lens, torch.int32, dev, B)
        if tree_mask is not None:
            _plain("tree_mask", tree_mask, torch.int64, dev, T)
        lse = None
        with _on(dev, stream):
            if out is None:
                out = torch.empty((T, Hq, D), dtype=dt, device=dev)
            else:
                _heads("out", out, dt, dev, D)
                if out.shape != q.shape:
                    raise ValueError("out must have q's shape")
            if return_lse:
                lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
            a = N.moe_attn_args_t(
                _DTYPES[dt], B, T, max_q_len, D ** -0.5 if scale is None else scale, q.data_ptr(), q.stride(0),
                q.stride(1), k_cache.data_ptr(), v_cache.data_ptr(), k_cache.stride(0), k_cache.stride(1),
                v_cache.stride(0), v_cache.stride(1), k_cache.shape[0], k_cache.shape[1], block_table.data_ptr(),
                block_table.stride(0) if B > 1 else block_table.shape[1], q_starts.data_ptr(), kv_lens.data_ptr(),
                None if tree_mask is None else tree_mask.data_ptr(), out.data_ptr(), out.stride(0), out.stride(1),
                None if lse is None else lse.data_ptr())
            N.check("moe_attn_forward", N.lib().moe_attn_forward(self._h, ctypes.byref(a), _stream_ptr(stream)))
        return (out, lse) if return_lse else out

    __call__ = forward

    def status(self) -> int:
        """Synchronises; returns the sticky device status (0 = ok) and clears it."""
        return N.lib().moe_attn_get_status(self._h)

    def close(self):
        if getattr(self, "_h", None):
            N.lib().moe_attn_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
