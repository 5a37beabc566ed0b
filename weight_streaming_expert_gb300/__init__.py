"""GB300-native small-M routed-MoE decode/verify layer.

The layer (router GEMV -> softmax top-k -> SwiGLU experts -> weighted
combine) runs in hand-written sm_103a CUDA kernels behind the C ABI in
``include/moe.h``; ``MoELayer`` is its Python face.  ``LmHead`` is the bf16
vocabulary projection of the same decode step (``include/lm_head.h``).  The step's
attention half stands in ``include/attention.h`` (``QKNormRope``,
``PagedAttention``, ``PagedKVCache``) and the draw of the next tokens in
``include/sampling.h`` (``sample``).  Importing the package loads nothing; the
CUDA library is loaded (and must exist) on first use.
"""
import importlib

_HOMES = {"MoELayer": "layer", "LmHead": "layer", "tp_slice": "layer", "combine_partials": "layer",
          "QKNormRope": "attention", "PagedAttention": "attention", "PagedKVCache": "cache", "PageTable": "cache",
          "copy_pages": "cache", "copy_rows": "cache", "sample": "sampling"}
__all__ = list(_HOMES)


def __getattr__(name):
    if name in _HOMES:
        return getattr(importlib.import_module("." + _HOMES[name], __name__), name)
    raise AttributeError(name)
