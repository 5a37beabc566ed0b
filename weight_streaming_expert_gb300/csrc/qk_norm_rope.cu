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
// 2 bytes in and 2 out per value.  A warp handles a token, or
// a share of its heads where there are few tokens; D/8 lanes share a head.  A
// lane holds four values of a head's first half and their four partners of the
// second (or four adjacent pairs), so a pair turns inside a thread and only
// the sum of squares crosses lanes.  The sines and cosines of a token are
// computed once by the warp, two or so per lane, while its first heads are on
// their way, and no warp waits for another.
//
// The norm's weights are multiplied into the sines and cosines once per token
// and kind, and the products are done on two fp32 values at a time: the kernel
// is bound by issuing instructions before it is by memory.  16384 tokens of 32
// + 8 heads of 128: 59 us, 5.6 TB/s; with weights and turns one after the other
// and single products 73 us, 70 % of the issue slots.  6 tokens: 3.2 us, a
// launch and two reads one after the other.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "host_util.cuh"

namespace wse {
namespace {

constexpr int kRopeThreads = 256, kRopeWarps = kRopeThreads / 32;
constexpr int kRopeLoads = 4;  // heads a lane has in flight

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
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two fp32 values side by side, whose products are one instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float x, float y) {
  f32x2 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 both(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 x, f32x2 y) {
  f32x2 v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(x), "l"(y));
  return v;
}
__device__ __forceinline__ f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) {
  f32x2 v;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(x), "l"(y), "l"(z));
  return v;
}

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, D == 256 ? 3 : 4) qk_norm_rope_kernel(
    const __grid_constant__ moe_qk_norm_rope_args_t a, int warps_per_token) {
  constexpr int kLanes = D / 8;               // lanes of a head
  constexpr int kHeads = 32 / kLanes;         // heads of a group: what a warp does at a time
  __shared__ float2 turn[kRopeWarps][D / 2];  // (cos, sin) of the warp's token
  const int lane = threadIdx.x & 31, part = lane % kLanes, sub = lane / kLanes;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // tells the compiler that it is uniform
  const long long t = (long long)blockIdx.x * (kRopeWarps / warps_per_token) + warp / warps_per_token;
  const int pairs = a.rotary_dim / 2;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.n_tokens) return;

  // where this lane's first and second four values of a head lie; lanes past
  // the rotated pairs share out the rest in the same way
  const bool turns = part * 4 < pairs;
  int lo = part * 8, hi = part * 8 + 4;
  if (!kInterleaved) {
    lo = turns ? part * 4 : part * 4 + pairs;
    hi = turns ? part * 4 + pairs : part * 4 + D / 2;
  }
  const int apart = hi - lo;
  const long long slot = a.n_kv_heads > 0 ? a.slots[t] : -1;
  const bool keep = slot >= 0 && slot < (long long)a.n_pages * a.page_size;
  const long long page = keep ? slot / a.page_size : 0, row = keep ? slot - page * a.page_size : 0;

  // groups of heads of one kind, so that what differs by kind is decided once
  // for the warp: of queries, then of keys, then of values
  const int q_groups = (a.n_heads + kHeads - 1) / kHeads, kv_groups = (a.n_kv_heads + kHeads - 1) / kHeads;
  const int groups = q_groups + 2 * kv_groups;
  auto kind_of = [&](int g) { return g < q_groups ? 0 : g < q_groups + kv_groups ? 1 : 2; };
  auto head_of = [&](int g, int kind) {
    return (kind == 0 ? g : kind == 1 ? g - q_groups : g - q_groups - kv_groups) * kHeads + sub;
  };
  // where this lane's values of a head begin, in and out
  auto from = [&](int kind, int head) {
    const long long at = kind == 0   ? t * a.q_token_stride + head * a.q_head_stride
                         : kind == 1 ? t * a.k_token_stride + head * a.k_head_stride
                                     : t * a.v_token_stride + head * a.v_head_stride;
    return static_cast<const T*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) + at + lo;
  };
  auto to = [&](int kind, int head) {
    const long long at = kind == 0   ? t * a.q_out_token_stride + head * a.q_out_head_stride
                         : kind == 1 ? page * a.k_page_stride + row * a.k_row_stride + head * D
                                     : page * a.v_page_stride + row * a.v_row_stride + head * D;
    return static_cast<T*>(kind == 0 ? a.q_out : kind == 1 ? a.k_cache : a.v_cache) + at + lo;
  };

  // what a head's values are multiplied with: norm weight times cosine or sine,
  // for this lane's pairs, two at a time.  Halves: own[0, 1] and cross[0, 1]
  // make the first of a pair, own[2, 3] and cross[2, 3] the second, with `own`
  // on that value itself.  Adjacent: own on (x_a, x_a), cross on (x_b, x_b).
  f32x2 own[4], cross[4];
  int made = -1;  // the kind that they are of
  auto factors_of = [&](int kind) {
    if (kind == made) return;
    made = kind;
    float w[8], c[4], sn[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if (const T* weight = static_cast<const T*>(kind == 0 ? a.q_weight : a.k_weight)) {
      const uint2 w0 = *reinterpret_cast<const uint2*>(weight + lo), w1 = *reinterpret_cast<const uint2*>(weight + hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = to_f32<T>(reinterpret_cast<const T*>(&w0)[j]);
        w[4 + j] = to_f32<T>(reinterpret_cast<const T*>(&w1)[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 cs = turns ? turn[warp][part * 4 + j] : make_float2(1.f, 0.f);
      c[j] = cs.x;
      sn[j] = cs.y;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kInterleaved) {
        const float wa = w[2 * j], wb = w[2 * j + 1];
        own[j] = turns ? pair_of(wa * c[j], wa * sn[j]) : pair_of(wa, wb);
        cross[j] = pair_of(-wb * sn[j], wb * c[j]);
      } else {
        const int n = 2 * (j & 1);  // of pairs n, n + 1
        const float* wo = w + (j < 2 ? 0 : 4);
        const float* wc = w + (j < 2 ? 4 : 0);
        const float sign = j < 2 ? -1.f : 1.f;
        own[j] = pair_of(wo[n] * c[n], wo[n + 1] * c[n + 1]);
        cross[j] = pair_of(sign * wc[n] * sn[n], sign * wc[n + 1] * sn[n + 1]);
      }
    }
  };
  // a group's values, normed and turned
  auto finish = [&](uint2& v0, uint2& v1, bool norm) {
    const T* e0 = reinterpret_cast<const T*>(&v0);
    const T* e1 = reinterpret_cast<const T*>(&v1);
    f32x2 x[4], y[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      x[j] = pair_of(to_f32<T>(e0[2 * j]), to_f32<T>(e0[2 * j + 1]));
      x[2 + j] = pair_of(to_f32<T>(e1[2 * j]), to_f32<T>(e1[2 * j + 1]));
    }
    if (norm) {
      f32x2 sq2 = mul2(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) sq2 = fma2(x[j], x[j], sq2);
      float sq = both(sq2).x + both(sq2).y;
#pragma unroll
      for (int m = kLanes / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m);
      const float r = rsqrtf(sq * (1.f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], pair_of(r, r));
    }
    if (turns) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kInterleaved) {
          const float2 v = both(x[j]);
          y[j] = fma2(pair_of(v.y, v.y), cross[j], mul2(pair_of(v.x, v.x), own[j]));
        } else {
          y[j] = fma2(x[j ^ 2], cross[j], mul2(x[j], own[j]));
        }
      }
    } else {  // 0 * inf must not reach these
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = mul2(x[j], own[j]);
    }
    v0 = make_uint2(pack2<T>(both(y[0]).x, both(y[0]).y), pack2<T>(both(y[1]).x, both(y[1]).y));
    v1 = make_uint2(pack2<T>(both(y[2]).x, both(y[2]).y), pack2<T>(both(y[3]).x, both(y[3]).y));
  };
  auto load = [&](uint2& v0, uint2& v1, const T* p) {
    v0 = *reinterpret_cast<const uint2*>(p);
    v1 = *reinterpret_cast<const uint2*>(p + apart);
  };
  auto store = [&](T* p, uint2 v0, uint2 v1) {
    *reinterpret_cast<uint2*>(p) = v0;
    *reinterpret_cast<uint2*>(p + apart) = v1;
  };

  const int g_first = warp % warps_per_token, whole = a.n_heads / kHeads;
  const long long q_step = (long long)warps_per_token * kHeads * a.q_head_stride;
  const long long out_step = (long long)warps_per_token * kHeads * a.q_out_head_stride;
  const T* q = from(0, g_first * kHeads + sub);
  T* out = to(0, g_first * kHeads + sub);
  for (int g0 = g_first; g0 < groups; g0 += kRopeLoads * warps_per_token) {
    const bool queries = g0 + (kRopeLoads - 1) * warps_per_token < whole;  // whole groups of them
    uint2 x0[kRopeLoads], x1[kRopeLoads];
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      const int g = g0 + i * warps_per_token;
      if (queries) {
        load(x0[i], x1[i], q);
        q += q_step;
      } else if (g < groups) {
        const int kind = kind_of(g), head = head_of(g, kind);
        if (head < (kind == 0 ? a.n_heads : a.n_kv_heads)) load(x0[i], x1[i], from(kind, head));
      }
    }
    if (g0 == g_first) {
      for (int i = lane; i < pairs; i += 32) {
        const unsigned long long at = (unsigned long long)(long long)a.positions[t] * a.turns[i];
        float sn, c;
        sincospif((float)(int)(at >> 32) * 0x1p-31f, &sn, &c);  // in half turns, turns in [-1/2, 1/2)
        turn[warp][i] = make_float2(c, sn);
      }
      __syncwarp();
    }
    if (queries) {
      factors_of(0);
      const bool norm = a.q_weight != nullptr;
#pragma unroll
      for (int i = 0; i < kRopeLoads; ++i) {
        finish(x0[i], x1[i], norm);
        store(out, x0[i], x1[i]);
        out += out_step;
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kRopeLoads; ++i) {
      const int g = g0 + i * warps_per_token;
      if (g >= groups) break;
      const int kind = kind_of(g), head = head_of(g, kind);
      if (kind < 2) {
        factors_of(kind);
        finish(x0[i], x1[i], (kind == 0 ? a.q_weight : a.k_weight) != nullptr);
      }
      if (head < (kind == 0 ? a.n_heads : a.n_kv_heads) && (kind == 0 || keep)) store(to(kind, head), x0[i], x1[i]);
    }
  }
}

template <typename T>
int launch_rope(const moe_qk_norm_rope_args_t& a, moe_stream_t stream) {
  void (*kernel)(const moe_qk_norm_rope_args_t, int) = nullptr;
  const bool il = a.interleaved != 0;
  if (a.head_dim == 64) kernel = il ? qk_norm_rope_kernel<T, 64, true> : qk_norm_rope_kernel<T, 64, false>;
  else if (a.head_dim == 128) kernel = il ? qk_norm_rope_kernel<T, 128, true> : qk_norm_rope_kernel<T, 128, false>;
  else kernel = il ? qk_norm_rope_kernel<T, 256, true> : qk_norm_rope_kernel<T, 256, false>;
  // Several warps share a token as long as all CTAs are resident at once (4 per
  // SM): 1001 tokens of 16 + 4 heads of 64 take 4.4 us with 4 warps each, 5.3
  // with 8.  Beyond that a warp each, which works the angles out once: 16384
  // tokens of 32 + 8 heads of 128 take 59 us, with 2 warps 64, with 4 76.
  int warps = kRopeWarps;
  const long long resident = 4ll * sm_count() * kRopeWarps;
  while (warps > 1 && a.n_tokens * (long long)warps > resident) warps /= 2;
  const int tokens = kRopeWarps / warps;
  return launch_pdl(kernel, dim3((unsigned)((a.n_tokens + tokens - 1) / tokens)), dim3(kRopeThreads), 0, stream, 1, a,
                    warps);
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
