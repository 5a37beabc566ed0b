// paged_attention.cu -- attention of a chunk of new tokens over a paged cache
// (include/attention.h).
//
// One warp per (token, query head) walks the positions it sees with a running
// maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "host_util.cuh"

namespace wse {
namespace {

enum : int { kAttnBadPage = 1, kAttnBadLength = 2, kAttnTimeout = 4 };

template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t v) {
  return make_float2(bf16lo(v), bf16hi(v));
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct AttnParams {
  moe_attn_args_t a;
  int n_heads, n_kv_heads;
  int* status;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) paged_attention_kernel(const AttnParams p) {
  constexpr int kWords = D / 64;  // 32-bit words of a lane
  const moe_attn_args_t& a = p.a;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (unit >= (long long)a.n_tokens * p.n_heads) return;
  const int t = (int)(unit / p.n_heads), h = (int)(unit % p.n_heads), kvh = h / (p.n_heads / p.n_kv_heads);
  int b = 0;
  while (b < a.batch && a.q_starts[b + 1] <= t) ++b;
  if (b == a.batch || t < a.q_starts[0]) return;
  const int n = a.q_starts[b + 1] - a.q_starts[b], i = t - a.q_starts[b];
  int kv = a.kv_lens[b];
  const long long room = (long long)a.table_stride * a.page_size;
  if (kv < 0 || kv > room) {
    if (lane == 0) atomicOr(p.status, kAttnBadLength);
    kv = kv < 0 ? 0 : (int)room;
  }
  const int base = kv - n;
  const long long bits = a.tree_mask ? a.tree_mask[t] : 0;
  const int end = a.tree_mask ? kv : min(kv, base + i + 1);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) + t * a.q_token_stride +
                                                        h * a.q_head_stride) + lane * kWords;
  float2 qv[kWords], acc[kWords];
  for (int w = 0; w < kWords; ++w) qv[w] = unpack<T>(q[w]), acc[w] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    if (a.tree_mask && j >= base && !((bits >> min(63, j - base)) & 1)) continue;
    const int page = a.block_table[(long long)b * a.table_stride + j / a.page_size];
    const bool bad = (unsigned)page >= (unsigned)a.n_pages;
    if (bad && lane == 0) atomicOr(p.status, kAttnBadPage);
    const long long off = j % a.page_size;
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.k_cache) + page * a.k_page_stride +
                                                           off * a.k_row_stride + kvh * D) + lane * kWords;
    const uint32_t* vp = reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.v_cache) + page * a.v_page_stride +
                                                           off * a.v_row_stride + kvh * D) + lane * kWords;
    float s = 0.f;
    float2 v[kWords];
    for (int w = 0; w < kWords; ++w) {
      const float2 kx = unpack<T>(bad ? 0u : kp[w]);
      v[w] = unpack<T>(bad ? 0u : vp[w]);
      s = fmaf(qv[w].x, kx.x, fmaf(qv[w].y, kx.y, s));
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale;
    const float top = fmaxf(m, s);
    const float was = m == -INFINITY ? 0.f : __expf(m - top), e = s == -INFINITY ? 0.f : __expf(s - top);
    l = l * was + e;
    for (int w = 0; w < kWords; ++w) acc[w].x = acc[w].x * was + e * v[w].x, acc[w].y = acc[w].y * was + e * v[w].y;
    m = top;
  }
  uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + t * a.out_token_stride + h * a.out_head_stride) +
                lane * kWords;
  const float r = l > 0.f ? 1.f / l : 0.f;
  for (int w = 0; w < kWords; ++w) o[w] = pack<T>(acc[w].x * r, acc[w].y * r);
  if (a.lse && lane == 0) a.lse[unit] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace wse

using namespace wse;

struct moe_attn {
  int n_heads, n_kv_heads, head_dim;
  int* status;
};

extern "C" {

moe_attn_t* moe_attn_create(int n_heads, int n_kv_heads, int head_dim) {
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads > 65536) {
    fail(MOE_ERR_INVALID_ARG, "n_heads = %d must be a multiple of n_kv_heads = %d", n_heads, n_kv_heads);
    return nullptr;
  }
  if (head_dim != 64 && head_dim != 128) {
    fail(MOE_ERR_UNSUPPORTED, "head_dim = %d: must be 64 or 128", head_dim);
    return nullptr;
  }
  if (check_device() != MOE_OK) return nullptr;
  auto* h = new moe_attn{n_heads, n_kv_heads, head_dim, nullptr};
  cudaError_t e = cudaMalloc(&h->status, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, sizeof(int));
  if (e != cudaSuccess) {
    fail_cuda(e, "attention workspace");
    cudaFree(h->status);
    delete h;
    return nullptr;
  }
  return h;
}

int moe_attn_forward(moe_attn_t* h, const moe_attn_args_t* a, moe_stream_t stream) {
  if (!h || !a) return fail(MOE_ERR_INVALID_ARG, "null handle or arguments");
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_FP16)
    return fail(MOE_ERR_INVALID_ARG, "dtype = %d: must be MOE_DTYPE_BF16 or MOE_DTYPE_FP16", a->dtype);
  if (a->batch < 0 || a->n_tokens < 0 || a->max_q_len < 0 || a->table_stride < 0)
    return fail(MOE_ERR_INVALID_ARG, "batch, n_tokens, max_q_len and table_stride must be 0 or more");
  if (!(a->scale > 0.f) || !(a->scale < INFINITY)) return fail(MOE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128 && a->page_size != 256)
    return fail(MOE_ERR_UNSUPPORTED, "page_size = %d: must be 16, 32, 64, 128 or 256", a->page_size);
  if (a->tree_mask && a->max_q_len > 64)
    return fail(MOE_ERR_UNSUPPORTED, "max_q_len = %d: a tree mask has 64 bits", a->max_q_len);
  if (a->batch == 0 || a->n_tokens == 0 || a->max_q_len == 0) return MOE_OK;
  if (a->n_pages < 1) return fail(MOE_ERR_INVALID_ARG, "n_pages = %d < 1", a->n_pages);
  if (!a->q || !a->k_cache || !a->v_cache || !a->out || !aligned(a->q, 16) || !aligned(a->k_cache, 16) ||
      !aligned(a->v_cache, 16) || !aligned(a->out, 16))
    return fail(MOE_ERR_INVALID_ARG, "q, out and the caches must be non-null and 16-byte aligned");
  if (!a->block_table || !a->q_starts || !a->kv_lens || !aligned(a->block_table, 4) || !aligned(a->q_starts, 4) ||
      !aligned(a->kv_lens, 4) || !aligned(a->tree_mask, 8) || !aligned(a->lse, 4))
    return fail(MOE_ERR_INVALID_ARG, "block_table, q_starts and kv_lens must be non-null, and all aligned");
  if ((a->q_token_stride | a->q_head_stride | a->out_token_stride | a->out_head_stride | a->k_page_stride |
       a->k_row_stride | a->v_page_stride | a->v_row_stride) & 7)
    return fail(MOE_ERR_INVALID_ARG, "every stride must be a multiple of 8 elements (16 bytes)");
  const AttnParams p{*a, h->n_heads, h->n_kv_heads, h->status};
  const long long units = (long long)a->n_tokens * h->n_heads;
  void (*kernel)(const AttnParams) =
      a->dtype == MOE_DTYPE_BF16
          ? (h->head_dim == 64 ? paged_attention_kernel<__nv_bfloat16, 64> : paged_attention_kernel<__nv_bfloat16, 128>)
          : (h->head_dim == 64 ? paged_attention_kernel<__half, 64> : paged_attention_kernel<__half, 128>);
  return launch_pdl(kernel, dim3((unsigned)((units + 3) / 4)), dim3(128), 0, stream, 1, p);
}

int moe_attn_get_status(moe_attn_t* h) {
  if (!h) return fail(MOE_ERR_INVALID_ARG, "null handle");
  int st = 0;
  cudaError_t e;
  if ((e = cudaDeviceSynchronize()) != cudaSuccess ||
      (e = cudaMemcpy(&st, h->status, sizeof st, cudaMemcpyDeviceToHost)) != cudaSuccess ||
      (e = cudaMemset(h->status, 0, sizeof st)) != cudaSuccess)
    return fail_cuda(e, "attention status");
  if (st & kAttnTimeout) return fail(MOE_ERR_DEVICE_TIMEOUT, "a bounded wait of the attention kernel ran out");
  if (st)
    return fail(MOE_ERR_INVALID_ARG, "%s%s", st & kAttnBadPage ? "a block table names a page outside the cache; " : "",
                st & kAttnBadLength ? "a length does not fit the block table or max_q_len" : "");
  return MOE_OK;
}

void moe_attn_destroy(moe_attn_t* h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->status);
  delete h;
}

}  // extern "C"
