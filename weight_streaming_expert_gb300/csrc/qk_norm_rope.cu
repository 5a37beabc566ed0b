// qk_norm_rope.cu -- norms of queries and keys per head with the position
// rotation, keys and values written into the paged cache, in one pass
// (include/attention.h).
//
// Per token and head, x its D values:  y = x * rsqrt(mean(x^2) + eps) * w,
// then pair i of the first `rot` values turns by the angle a_i:
//   (y_a, y_b) -> (y_a cos a_i - y_b sin a_i,  y_a sin a_i + y_b cos a_i).
// a_i = position * (turns per position), a number that grows to 10^5 turns
// while only its fraction counts.  Held as a fraction of 2^64 the product
// wraps modulo a whole turn by itself, so the angle has an error of
// position * 2^-65 turns and the 32 leading bits go to sincospif.
//
// Bound by memory: 2 bytes in and 2 out per value.  One CTA per token: the
// rot/2 sine/cosine pairs are computed once per token (one per thread) while
// the heads' 16-byte loads are in flight, and D/8 lanes share a head, so that
// the sum of squares and the pairs' partners are shuffles inside a warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "host_util.cuh"

namespace wse {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeLoads = 4;  // heads a thread has in flight

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const moe_qk_norm_rope_args_t a) {
  constexpr int kLanes = D / 8;                       // lanes of a head
  constexpr int kPerPass = kRopeThreads / kLanes;     // heads of a pass
  __shared__ float2 turn[D / 2];                      // (cos, sin) of this token's angles
  const int tid = threadIdx.x, part = tid % kLanes, row = tid / kLanes;
  const long long t = blockIdx.x;
  const int n_qk = a.n_heads + a.n_kv_heads, n_all = n_qk + a.n_kv_heads;
  const int rot = a.rotary_dim;
  pdl_wait();
  pdl_launch_dependents();

  const long long slot = a.n_kv_heads > 0 ? a.slots[t] : -1;
  const bool keep = slot >= 0 && slot < (long long)a.n_pages * a.page_size;
  const long long page = keep ? slot / a.page_size : 0, off = keep ? slot % a.page_size : 0;
  const T* qw = static_cast<const T*>(a.q_weight);
  const T* kw = static_cast<const T*>(a.k_weight);
  float c[8], s[8];
  bool first = true;
  for (int base = 0; base < n_all; base += kRopeLoads * kPerPass) {
    uint4 raw[kRopeLoads];
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      const int h = base + i * kPerPass + row;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < a.n_heads)
        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + t * a.q_token_stride +
                                                 h * a.q_head_stride + part * 8);
      else if (h < n_qk)
        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + t * a.k_token_stride +
                                                 (h - a.n_heads) * a.k_head_stride + part * 8);
      else if (h < n_all)
        raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + t * a.v_token_stride +
                                                 (h - n_qk) * a.v_head_stride + part * 8);
    }
    if (first) {
      first = false;
      if (tid < rot / 2) {
        const unsigned long long at = (unsigned long long)(long long)a.positions[t] * a.turns[tid];
        float sn, cs;
        sincospif((float)(int)(at >> 32) * 0x1p-31f, &sn, &cs);  // 2 * turns half-turns, turns in [-1/2, 1/2)
        turn[tid] = make_float2(cs, sn);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = part * 8 + j;
        const int pair = kInterleaved ? e / 2 : (e < rot / 2 ? e : e - rot / 2);
        const float2 v = e < rot ? turn[pair] : make_float2(1.f, 0.f);
        c[j] = v.x;
        // the first of a pair takes -sin of its partner, the second +sin
        s[j] = (kInterleaved ? (e & 1) == 0 : e < rot / 2) ? -v.y : v.y;
      }
    }
    // the lane of this head that holds the partners of this lane's values
    const int half = rot / 16, lane = tid & 31;
    const int partner = part < half ? lane + half : (part < 2 * half ? lane - half : lane);
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      const int h = base + i * kPerPass + row;
      const T* e = reinterpret_cast<const T*>(&raw[i]);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(e[j]);
      const T* w = h < a.n_heads ? qw : kw;
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(x[j], x[j], sq);
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
      if (w && h < n_qk) {
        const float r = rsqrtf(sq * (1.f / D) + a.eps);
        const uint4 wraw = *reinterpret_cast<const uint4*>(w + part * 8);
        const T* we = reinterpret_cast<const T*>(&wraw);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * to_f32<T>(we[j]);
      }
      uint4 packed;
      T* o = reinterpret_cast<T*>(&packed);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float other = kInterleaved ? x[j ^ 1] : __shfl_sync(0xffffffffu, x[j], partner);
        // values outside the rotated part stay as they are (0 * inf must not reach them)
        o[j] = from_f32<T>(part * 8 + j < rot ? fmaf(other, s[j], x[j] * c[j]) : x[j]);
      }
      if (h < a.n_heads)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + t * a.q_out_token_stride + h * a.q_out_head_stride +
                                  part * 8) = packed;
      else if (h < n_qk && keep)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.k_cache) + page * a.k_page_stride + off * a.k_row_stride +
                                  (long long)(h - a.n_heads) * D + part * 8) = packed;
      else if (h < n_all && h >= n_qk && keep)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) + page * a.v_page_stride + off * a.v_row_stride +
                                  (long long)(h - n_qk) * D + part * 8) = raw[i];
    }
  }
}

template <typename T>
int launch_rope(const moe_qk_norm_rope_args_t& a, moe_stream_t stream) {
  void (*kernel)(const moe_qk_norm_rope_args_t) = nullptr;
  const bool il = a.interleaved != 0;
  if (a.head_dim == 64) kernel = il ? qk_norm_rope_kernel<T, 64, true> : qk_norm_rope_kernel<T, 64, false>;
  else if (a.head_dim == 128) kernel = il ? qk_norm_rope_kernel<T, 128, true> : qk_norm_rope_kernel<T, 128, false>;
  else kernel = il ? qk_norm_rope_kernel<T, 256, true> : qk_norm_rope_kernel<T, 256, false>;
  return launch_pdl(kernel, dim3((unsigned)a.n_tokens), dim3(kRopeThreads), 0, stream, 1, a);
}

}  // namespace
}  // namespace wse

using namespace wse;

extern "C" int moe_qk_norm_rope(const moe_qk_norm_rope_args_t* a, moe_stream_t stream) {
  if (!a) return fail(MOE_ERR_INVALID_ARG, "null arguments");
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_FP16)
    return fail(MOE_ERR_INVALID_ARG, "dtype = %d: must be MOE_DTYPE_BF16 or MOE_DTYPE_FP16", a->dtype);
  if (a->n_tokens < 0 || a->n_heads < 0 || a->n_kv_heads < 0 || a->n_heads > 65536 || a->n_kv_heads > 65536)
    return fail(MOE_ERR_INVALID_ARG, "n_tokens, n_heads and n_kv_heads must be 0 or more (heads up to 65536)");
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head_dim = %d: must be 64, 128 or 256", a->head_dim);
  if (a->rotary_dim < 0 || a->rotary_dim > a->head_dim || a->rotary_dim % 16)
    return fail(MOE_ERR_INVALID_ARG, "rotary_dim = %d: must be a multiple of 16 up to head_dim", a->rotary_dim);
  if (!(a->eps >= 0.f)) return fail(MOE_ERR_INVALID_ARG, "eps must be 0 or more");
  if (a->n_tokens == 0 || a->n_heads + a->n_kv_heads == 0) return MOE_OK;
  if (a->rotary_dim > 0 && (!a->turns || !a->positions || !aligned(a->turns, 8) || !aligned(a->positions, 4)))
    return fail(MOE_ERR_INVALID_ARG, "turns and positions must be non-null and aligned to their elements");
  if (a->n_heads > 0 && (!a->q || !a->q_out || !aligned(a->q, 16) || !aligned(a->q_out, 16)))
    return fail(MOE_ERR_INVALID_ARG, "q and q_out must be non-null and 16-byte aligned");
  if (a->n_kv_heads > 0 &&
      (!a->k || !a->v || !a->k_cache || !a->v_cache || !aligned(a->k, 16) || !aligned(a->v, 16) ||
       !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !a->slots || !aligned(a->slots, 8)))
    return fail(MOE_ERR_INVALID_ARG, "k, v and the caches must be non-null and 16-byte aligned, slots 8-byte");
  if ((a->q_weight && !aligned(a->q_weight, 16)) || (a->k_weight && !aligned(a->k_weight, 16)))
    return fail(MOE_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
  if ((a->q_token_stride | a->q_head_stride | a->k_token_stride | a->k_head_stride | a->v_token_stride |
       a->v_head_stride | a->q_out_token_stride | a->q_out_head_stride | a->k_page_stride | a->k_row_stride |
       a->v_page_stride | a->v_row_stride) & 7)
    return fail(MOE_ERR_INVALID_ARG, "every stride must be a multiple of 8 elements (16 bytes)");
  if (a->n_kv_heads > 0 && (a->n_pages < 1 || a->page_size < 1))
    return fail(MOE_ERR_INVALID_ARG, "n_pages and page_size must be 1 or more");
  const int rc = check_device();
  if (rc != MOE_OK) return rc;
  return a->dtype == MOE_DTYPE_BF16 ? launch_rope<__nv_bfloat16>(*a, stream) : launch_rope<__half>(*a, stream);
}
