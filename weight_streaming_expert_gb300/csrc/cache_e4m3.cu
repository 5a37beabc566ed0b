// cache_e4m3.cu -- reading rows of the quantised cache back, and moving its
// scales (include/attention.h).
#include "attention.h"
#include "e4m3.cuh"
#include "host_util.cuh"

namespace wse {
namespace {

constexpr int kReadThreads = 256;

// `lanes` of a warp take a token, 16 codes of it each at a time (so that its slot
// is worked out once for them: with 16 codes of any row a thread the divisions
// took longer than memory); blockIdx.y: keys or values.  D + 1 bytes in and 2 D
// out for each row, but bound by the latency of its waves (slot, then codes and
// scale, then the stores) and by issue: 16384 tokens of 4 heads of 128 11.2 us
// (memory needs 7.5), 73 % of the issue slots, DRAM 14 %; with four tokens a lane
// in flight and fewer threads 12.9.  6 tokens 1.7 us, a launch.
__global__ void __launch_bounds__(kReadThreads, 8)
    read_e4m3_kernel(const __grid_constant__ moe_read_e4m3_args_t a, int lanes) {
  const bool values = blockIdx.y != 0;
  const int per_head = a.head_dim / 16, per_token = a.n_kv_heads * per_head;
  const long long t = (long long)blockIdx.x * (kReadThreads / lanes) + threadIdx.x / lanes;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.n) return;
  const long long slot = a.slots[t];
  const bool there = slot >= 0 && slot < (long long)a.n_pages * a.page_size;
  const long long page = slot >> 32 ? slot / a.page_size : (unsigned)slot / (unsigned)a.page_size;
  const long long row = slot - page * a.page_size;
  const uint8_t* codes = values ? static_cast<const uint8_t*>(a.v_cache) + page * a.v_page_stride + row * a.v_row_stride
                                : static_cast<const uint8_t*>(a.k_cache) + page * a.k_page_stride + row * a.k_row_stride;
  const uint8_t* scale = values ? static_cast<const uint8_t*>(a.scales.v_scale) + page * a.scales.v_page_stride + row
                                : static_cast<const uint8_t*>(a.scales.k_scale) + page * a.scales.k_page_stride + row;
  const long long scale_head = values ? a.scales.v_head_stride : a.scales.k_head_stride;
  char* out = values ? static_cast<char*>(a.v_out) + t * a.v_token_stride * 2
                     : static_cast<char*>(a.k_out) + t * a.k_token_stride * 2;
  const long long head_stride = (values ? a.v_head_stride : a.k_head_stride) * 2;
  for (int u = threadIdx.x % lanes; u < per_token; u += lanes) {
    const int head = u / per_head, part = u - head * per_head;
    uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    if (there) {
      const uint4 c = *reinterpret_cast<const uint4*>(codes + u * 16);
      expand_e4m3(c, power_of_two(exponent_of(scale[head * scale_head])), a.dtype == MOE_DTYPE_BF16, v);
    }
    uint4* to = reinterpret_cast<uint4*>(out + head * head_stride + part * 32);
    to[0] = make_uint4(v[0], v[1], v[2], v[3]);
    to[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

struct CopyScalesArgs {
  uint8_t* pool[2];
  int64_t layer_stride[2], page_stride[2], head_stride[2];
  int64_t n_slots;
  int page_size, n_heads, n;
  const int64_t* src;
  const int64_t* dst;
};

constexpr int kScaleHeads = kReadThreads / MOE_COPY_ROWS_MAX;  // of a CTA

// One CTA moves the scales of all rows for kScaleHeads heads of a layer: every
// thread has read its byte before any thread writes.
__global__ void __launch_bounds__(kReadThreads) copy_scales_kernel(const CopyScalesArgs a) {
  const int which = blockIdx.y & 1;
  const long long layer = blockIdx.y >> 1;
  const int i = threadIdx.x / kScaleHeads;
  const long long head = (long long)blockIdx.x * kScaleHeads + threadIdx.x % kScaleHeads;
  pdl_wait();
  pdl_launch_dependents();
  uint8_t* base = a.pool[which] + layer * a.layer_stride[which] + head * a.head_stride[which];
  uint8_t v = 0;
  long long d = -1;
  if (i < a.n && head < a.n_heads) {
    const long long s = a.src[i];
    d = a.dst[i];
    if (s < 0 || s >= a.n_slots || d >= a.n_slots) d = -1;
    if (d >= 0) v = base[s / a.page_size * a.page_stride[which] + s % a.page_size];
  }
  __syncthreads();
  if (d >= 0) base[d / a.page_size * a.page_stride[which] + d % a.page_size] = v;
}

}  // namespace
}  // namespace wse

using namespace wse;

extern "C" {

int moe_read_e4m3(const moe_read_e4m3_args_t* a, moe_stream_t stream) {
  if (!a) return fail(MOE_ERR_INVALID_ARG, "null arguments");
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_FP16)
    return fail(MOE_ERR_INVALID_ARG, "dtype = %d: must be MOE_DTYPE_BF16 or MOE_DTYPE_FP16", a->dtype);
  if (a->n < 0 || a->n_kv_heads < 0 || a->n_kv_heads > 65536)
    return fail(MOE_ERR_INVALID_ARG, "n and n_kv_heads must be 0 or more (heads up to 65536)");
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return fail(MOE_ERR_UNSUPPORTED, "head_dim = %d: must be 64, 128 or 256", a->head_dim);
  if (a->n == 0 || a->n_kv_heads == 0) return MOE_OK;
  if (a->n_pages < 1 || a->page_size < 1)
    return fail(MOE_ERR_INVALID_ARG, "n_pages and page_size must be 1 or more");
  if (!a->slots || !aligned(a->slots, 8)) return fail(MOE_ERR_INVALID_ARG, "slots must be non-null and 8-byte aligned");
  if (!a->k_cache || !a->v_cache || !a->k_out || !a->v_out || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) ||
      !aligned(a->k_out, 16) || !aligned(a->v_out, 16) || !a->scales.k_scale || !a->scales.v_scale)
    return fail(MOE_ERR_INVALID_ARG, "the caches, scales and outputs must be non-null, caches and outputs 16-byte aligned");
  if ((a->k_page_stride | a->k_row_stride | a->v_page_stride | a->v_row_stride) & 15)
    return fail(MOE_ERR_INVALID_ARG, "every stride of the caches must be a multiple of 16 bytes");
  if ((a->k_token_stride | a->k_head_stride | a->v_token_stride | a->v_head_stride) & 7)
    return fail(MOE_ERR_INVALID_ARG, "every stride of the outputs must be a multiple of 8 elements (16 bytes)");
  const int rc = check_device();
  if (rc != MOE_OK) return rc;
  int lanes = 1;
  while (lanes < 32 && lanes < a->n_kv_heads * (a->head_dim / 16)) lanes *= 2;
  const long long tokens = kReadThreads / lanes;  // of a CTA
  return launch_pdl(read_e4m3_kernel, dim3((unsigned)((a->n + tokens - 1) / tokens), 2), dim3(kReadThreads), 0, stream, 1,
                    *a, lanes);
}

int moe_copy_scales(void* k_scales, void* v_scales, int n_layers, int64_t k_layer_stride, int64_t v_layer_stride,
                    int64_t k_page_stride, int64_t v_page_stride, int64_t k_head_stride, int64_t v_head_stride,
                    int n_pages, int page_size, int n_kv_heads, const int64_t* src, const int64_t* dst, int n,
                    moe_stream_t stream) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n > MOE_COPY_ROWS_MAX) return fail(MOE_ERR_UNSUPPORTED, "n = %d exceeds %d", n, MOE_COPY_ROWS_MAX);
  if (!k_scales || !v_scales) return fail(MOE_ERR_INVALID_ARG, "the scales must be non-null");
  if (n_layers < 1 || n_layers > 32767 || n_pages < 1 || page_size < 1 || n_kv_heads < 1 || n_kv_heads > 65536)
    return fail(MOE_ERR_INVALID_ARG, "n_layers must be in 1..32767, n_kv_heads in 1..65536, n_pages and page_size 1 or "
                                     "more");
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 8) || !aligned(dst, 8))
    return fail(MOE_ERR_INVALID_ARG, "src and dst must be non-null and 8-byte aligned");
  const CopyScalesArgs a{{static_cast<uint8_t*>(k_scales), static_cast<uint8_t*>(v_scales)},
                         {k_layer_stride, v_layer_stride},
                         {k_page_stride, v_page_stride},
                         {k_head_stride, v_head_stride},
                         (int64_t)n_pages * page_size, page_size, n_kv_heads, n, src, dst};
  const int rc = check_device();
  if (rc != MOE_OK) return rc;
  return launch_pdl(copy_scales_kernel, dim3((unsigned)((n_kv_heads + kScaleHeads - 1) / kScaleHeads), 2u * n_layers),
                    dim3(kReadThreads), 0, stream, 1, a);
}

}  // extern "C"
