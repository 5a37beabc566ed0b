"""ctypes binding of include/moe.h, lm_head.h, attention.h and sampling.h (same
names; argument marshalling only).

Every step of the layer runs in the CUDA library ``_build/libwse.so``.  There
is no Python or CPU fallback: if the library is missing or fails to load,
``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from . import build_lib

_lock = threading.Lock()
_lib = None

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_CUDA = 3
MOE_ERR_OOM = 4
MOE_ERR_DEVICE_TIMEOUT = 5
MOE_MAX_TOKENS = 64
MOE_LM_HEAD_MAX_TOKENS = 16
MOE_GEMV_MAX_TOKENS = 16
MOE_GEMV_CUDA_CORES = 0
MOE_GEMV_TENSOR_CORES = 1
MOE_FWD_NO_PDL = 0x1
MOE_FWD_GRAPH = 0x2
MOE_FWD_TRACE = 0x4
MOE_FWD_OUT_F32 = 0x8
MOE_FWD_TEST_SKIP_ARRIVAL = 0x40000000
TRACE_SLOTS = 32
MOE_DTYPE_BF16 = 0
MOE_DTYPE_FP16 = 1
MOE_COPY_ROWS_MAX = 64

STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
                4: "MOE_ERR_OOM", 5: "MOE_ERR_DEVICE_TIMEOUT"}


class moe_info_t(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("n_experts", ctypes.c_int), ("topk", ctypes.c_int),
                ("inter", ctypes.c_int), ("max_tokens", ctypes.c_int), ("n_sms", ctypes.c_int),
                ("gateup_stages", ctypes.c_int), ("down_stages", ctypes.c_int),
                ("gateup_tile_bytes", ctypes.c_int), ("down_tile_bytes", ctypes.c_int),
                ("weight_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t),
                ("kernels_per_forward", ctypes.c_int), ("router_split", ctypes.c_int),
                ("smem_bytes", ctypes.c_size_t), ("shared_expert", ctypes.c_int),
                ("routed_scale", ctypes.c_float), ("bias_selection_only", ctypes.c_int),
                ("fp8_experts", ctypes.c_int), ("grid_ctas", ctypes.c_int),
                ("wait_limit_ns", ctypes.c_ulonglong)]


class moe_layer_opts_t(ctypes.Structure):
    _fields_ = [("w_shared_gate_up", ctypes.c_void_p), ("w_shared_down", ctypes.c_void_p),
                ("routed_scale", ctypes.c_float), ("bias_selection_only", ctypes.c_int)]


_i, _l, _p, _f = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class moe_qk_norm_rope_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i), ("n_tokens", _i), ("n_heads", _i), ("n_kv_heads", _i), ("head_dim", _i),
                ("rotary_dim", _i), ("interleaved", _i), ("eps", _f), ("q", _p), ("k", _p), ("v", _p),
                ("q_token_stride", _l), ("q_head_stride", _l), ("k_token_stride", _l), ("k_head_stride", _l),
                ("v_token_stride", _l), ("v_head_stride", _l), ("q_weight", _p), ("k_weight", _p), ("turns", _p),
                ("positions", _p), ("slots", _p), ("q_out", _p), ("q_out_token_stride", _l),
                ("q_out_head_stride", _l), ("k_cache", _p), ("v_cache", _p), ("k_page_stride", _l),
                ("k_row_stride", _l), ("v_page_stride", _l), ("v_row_stride", _l), ("n_pages", _i),
                ("page_size", _i)]


class moe_cache_scales_t(ctypes.Structure):
    _fields_ = [("k_scale", _p), ("v_scale", _p), ("k_page_stride", _l), ("k_head_stride", _l), ("v_page_stride", _l),
                ("v_head_stride", _l)]


class moe_read_e4m3_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i), ("n", _i), ("n_kv_heads", _i), ("head_dim", _i), ("k_cache", _p), ("v_cache", _p),
                ("k_page_stride", _l), ("k_row_stride", _l), ("v_page_stride", _l), ("v_row_stride", _l),
                ("scales", moe_cache_scales_t), ("n_pages", _i), ("page_size", _i), ("slots", _p), ("k_out", _p),
                ("v_out", _p), ("k_token_stride", _l), ("k_head_stride", _l), ("v_token_stride", _l),
                ("v_head_stride", _l)]


class moe_attn_args_t(ctypes.Structure):
    _fields_ = [("dtype", _i), ("batch", _i), ("n_tokens", _i), ("max_q_len", _i), ("scale", _f), ("q", _p),
                ("q_token_stride", _l), ("q_head_stride", _l), ("k_cache", _p), ("v_cache", _p),
                ("k_page_stride", _l), ("k_row_stride", _l), ("v_page_stride", _l), ("v_row_stride", _l),
                ("n_pages", _i), ("page_size", _i), ("block_table", _p), ("table_stride", _i), ("q_starts", _p),
                ("kv_lens", _p), ("tree_mask", _p), ("out", _p), ("out_token_stride", _l), ("out_head_stride", _l),
                ("lse", _p), ("table_pages", _i)]


class moe_attn_opts_t(ctypes.Structure):
    _fields_ = [("scales", ctypes.POINTER(moe_cache_scales_t)), ("prefix_len", _i), ("workspace", _p),
                ("workspace_bytes", ctypes.c_size_t)]


class moe_adjust_logits_args_t(ctypes.Structure):
    _fields_ = [("logits", _p), ("row_stride", _l), ("out", _p), ("out_stride", _l), ("rows", _i), ("vocab", _i),
                ("history", _p), ("n_history", _i), ("spans", _p), ("repetition", _p), ("presence", _p),
                ("frequency", _p), ("bias_ids", _p), ("bias_values", _p), ("n_biases", _i), ("bias_starts", _p),
                ("allowed", _p), ("allowed_stride", _l)]


class MoEError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def library_path() -> str:
    return build_lib.LIB


def lib(build_if_missing: bool = True):
    """The loaded C library with its prototypes declared."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = build_lib.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"CUDA library not built: {path}")
            build_lib.build_library()
        L = ctypes.CDLL(path)
        vp, ci, cu = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint
        i32p = ctypes.POINTER(ctypes.c_int32)
        f32p = ctypes.POINTER(ctypes.c_float)
        ip = ctypes.POINTER(ctypes.c_int)
        L.moe_create.argtypes = [ci, ci, ci, ci, vp, vp, vp]
        L.moe_create.restype = vp
        L.moe_create_ex.argtypes = [ci, ci, ci, ci, vp, vp, vp, ctypes.POINTER(moe_layer_opts_t)]
        L.moe_create_ex.restype = vp
        L.moe_create_fp8.argtypes = [ci, ci, ci, ci, vp, vp, vp, vp, vp]
        L.moe_create_fp8.restype = vp
        L.moe_forward.argtypes = [vp, vp, vp, vp, ci, vp]
        L.moe_forward.restype = ci
        L.moe_forward_ex.argtypes = [vp, vp, vp, vp, vp, ci, vp, cu]
        L.moe_forward_ex.restype = ci
        L.moe_forward_timed.argtypes = [vp, vp, vp, vp, ci, vp, ctypes.POINTER(vp)]
        L.moe_forward_timed.restype = ci
        L.moe_set_router_bias.argtypes = [vp, vp]
        L.moe_set_router_bias.restype = ci
        L.moe_get_status.argtypes = [vp]
        L.moe_get_status.restype = ci
        L.moe_set_grid.argtypes = [vp, ci]
        L.moe_set_grid.restype = ci
        L.moe_set_wait_limit.argtypes = [vp, ctypes.c_ulonglong]
        L.moe_set_wait_limit.restype = ci
        L.moe_combine_partials.argtypes = [vp, ci, ctypes.c_size_t, vp, vp]
        L.moe_combine_partials.restype = ci
        L.moe_get_info.argtypes = [vp, ctypes.POINTER(moe_info_t)]
        L.moe_get_info.restype = ci
        L.moe_read_routing.argtypes = [vp, ci, ip, ip, i32p, i32p, i32p, i32p, f32p, ci]
        L.moe_read_routing.restype = ci
        L.moe_read_trace.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64), ci]
        L.moe_read_trace.restype = ci
        L.moe_route_static.argtypes = [ci, ci, ci, vp, vp, vp, ci, vp, vp, vp]
        L.moe_route_static.restype = ci
        L.moe_route_static_read_status.argtypes = [vp, vp]
        L.moe_route_static_read_status.restype = ci
        L.moe_destroy.argtypes = [vp]
        L.moe_destroy.restype = None
        L.moe_lm_head_create.argtypes = [ci, ci, vp]
        L.moe_lm_head_create.restype = vp
        L.moe_lm_head_forward.argtypes = [vp, vp, vp, ci, vp]
        L.moe_lm_head_forward.restype = ci
        L.moe_lm_head_get_status.argtypes = [vp]
        L.moe_lm_head_get_status.restype = ci
        L.moe_lm_head_destroy.argtypes = [vp]
        L.moe_lm_head_destroy.restype = None
        L.moe_gemv_pack.argtypes = [vp, vp, ci, ci, vp]
        L.moe_gemv_pack.restype = ci
        L.moe_gemv.argtypes = [vp, vp, vp, ci, ci, ci, ci, vp]
        L.moe_gemv.restype = ci
        L.moe_gemv_get_status.argtypes = []
        L.moe_gemv_get_status.restype = ci
        i64 = ctypes.c_int64
        L.moe_qk_norm_rope.argtypes = [ctypes.POINTER(moe_qk_norm_rope_args_t), vp]
        L.moe_qk_norm_rope.restype = ci
        L.moe_qk_norm_rope_e4m3.argtypes = [ctypes.POINTER(moe_qk_norm_rope_args_t), ctypes.POINTER(moe_cache_scales_t),
                                            vp]
        L.moe_qk_norm_rope_e4m3.restype = ci
        L.moe_read_e4m3.argtypes = [ctypes.POINTER(moe_read_e4m3_args_t), vp]
        L.moe_read_e4m3.restype = ci
        L.moe_copy_scales.argtypes = [vp, vp, ci, i64, i64, i64, i64, i64, i64, ci, ci, ci, vp, vp, ci, vp]
        L.moe_copy_scales.restype = ci
        L.moe_attn_create.argtypes = [ci, ci, ci]
        L.moe_attn_create.restype = vp
        L.moe_attn_forward.argtypes = [vp, ctypes.POINTER(moe_attn_args_t), vp]
        L.moe_attn_forward.restype = ci
        L.moe_attn_forward_ex.argtypes = [vp, ctypes.POINTER(moe_attn_args_t), ctypes.POINTER(moe_attn_opts_t), vp]
        L.moe_attn_forward_ex.restype = ci
        L.moe_attn_workspace.argtypes = [vp, ctypes.POINTER(moe_attn_args_t), ctypes.POINTER(moe_attn_opts_t)]
        L.moe_attn_workspace.restype = ctypes.c_size_t
        L.moe_attn_get_status.argtypes = [vp]
        L.moe_attn_get_status.restype = ci
        L.moe_attn_destroy.argtypes = [vp]
        L.moe_attn_destroy.restype = None
        L.moe_copy_pages.argtypes = [vp, vp, ci, i64, i64, i64, i64, ci, i64, vp, vp, ci, vp]
        L.moe_copy_pages.restype = ci
        L.moe_copy_rows.argtypes = [vp, vp, ci, i64, i64, i64, i64, ci, ci, i64, vp, vp, ci, vp]
        L.moe_copy_rows.restype = ci
        L.moe_sample.argtypes = [vp, i64, ci, ci, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_sample.restype = ci
        L.moe_adjust_logits.argtypes = [ctypes.POINTER(moe_adjust_logits_args_t), vp]
        L.moe_adjust_logits.restype = ci
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        _lib = L
        return L


_calls = None


def calls():
    """The extension module of the attention and sampling calls
    (``_build/wse_calls.so``, csrc/python_calls.cpp), loaded on first use."""
    global _calls
    if _calls is None:
        lib()  # it is linked against the library
        with _lock:
            if not os.path.exists(build_lib.CALLS):
                build_lib.build()
            if not os.path.exists(build_lib.CALLS):
                raise RuntimeError(f"extension module not built: {build_lib.CALLS}")
            loader = importlib.machinery.ExtensionFileLoader("wse_calls", build_lib.CALLS)
            spec = importlib.util.spec_from_file_location("wse_calls", build_lib.CALLS, loader=loader)
            module = importlib.util.module_from_spec(spec)
            loader.exec_module(module)
            _calls = module
    return _calls


def last_error() -> str:
    return (lib().moe_last_error() or b"").decode()


def check(fn: str, status: int):
    if status != MOE_OK:
        raise MoEError(fn, status, last_error())
