// cache_pages.cu -- moving pages and rows of the paged cache
// (include/attention.h).
//
// A copy is bound by memory: each moved byte is read and written once.
#include "attention.h"
#include "host_util.cuh"

namespace wse {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 4;                                  // 16-byte loads a thread has in flight
constexpr int kCopyChunk = kCopyThreads * kCopyLoads * 16;     // bytes a CTA moves

struct CopyPagesArgs {
  char* pool[2];
  int64_t layer_stride[2], page_stride[2];
  int64_t page_bytes;
  int n_pages, chunks;  // chunks of a page
  const int32_t* src;
  const int32_t* dst;
};

// One CTA moves one chunk of one page of one layer of one pool: blockIdx.x =
// pair * chunks + chunk, blockIdx.y = 2 * layer + pool.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyPagesArgs a) {
  const int pair = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int which = blockIdx.y & 1;
  const long long layer = blockIdx.y >> 1;
  pdl_wait();
  pdl_launch_dependents();
  const int s = a.src[pair], d = a.dst[pair];
  if ((unsigned)s >= (unsigned)a.n_pages || (unsigned)d >= (unsigned)a.n_pages) return;
  char* base = a.pool[which] + layer * a.layer_stride[which];
  const char* from = base + s * a.page_stride[which];
  char* to = base + d * a.page_stride[which];
  const long long at = (long long)chunk * kCopyChunk + threadIdx.x * 16;
  uint4 v[kCopyLoads];
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    const long long o = at + (long long)i * kCopyThreads * 16;
    if (o < a.page_bytes) v[i] = *reinterpret_cast<const uint4*>(from + o);
  }
#pragma unroll
  for (int i = 0; i < kCopyLoads; ++i) {
    const long long o = at + (long long)i * kCopyThreads * 16;
    if (o < a.page_bytes) *reinterpret_cast<uint4*>(to + o) = v[i];
  }
}

struct CopyRowsArgs {
  char* pool[2];
  int64_t layer_stride[2], page_stride[2];
  int64_t row_bytes;
  int64_t n_slots;
  int page_size, n;
  const int64_t* src;
  const int64_t* dst;
};

constexpr int kRowColumns = kCopyThreads / MOE_COPY_ROWS_MAX;  // 16-byte columns of a CTA

// One CTA moves all rows' bytes of kRowColumns columns: every thread has read
// its 16 bytes before any thread writes, so rows may move onto one another.
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const CopyRowsArgs a) {
  const int which = blockIdx.y & 1;
  const long long layer = blockIdx.y >> 1;
  const int i = threadIdx.x / kRowColumns;
  const long long at = ((long long)blockIdx.x * kRowColumns + threadIdx.x % kRowColumns) * 16;
  pdl_wait();
  pdl_launch_dependents();
  char* base = a.pool[which] + layer * a.layer_stride[which];
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  long long d = -1;
  if (i < a.n && at < a.row_bytes) {
    const long long s = a.src[i];
    d = a.dst[i];
    if (s < 0 || s >= a.n_slots || d >= a.n_slots) d = -1;
    if (d >= 0)
      v = *reinterpret_cast<const uint4*>(base + s / a.page_size * a.page_stride[which] +
                                          s % a.page_size * a.row_bytes + at);
  }
  __syncthreads();
  if (d >= 0)
    *reinterpret_cast<uint4*>(base + d / a.page_size * a.page_stride[which] + d % a.page_size * a.row_bytes + at) = v;
}

int check_pools(const void* k, const void* v, int n_layers, int64_t s0, int64_t s1, int64_t s2, int64_t s3,
                int n_pages, int64_t bytes, const char* unit) {
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
    return fail(MOE_ERR_INVALID_ARG, "the pools must be non-null and 16-byte aligned");
  if (n_layers < 1 || n_layers > 32767 || n_pages < 1)
    return fail(MOE_ERR_INVALID_ARG, "n_layers must be in 1..32767 and n_pages 1 or more");
  if (bytes < 16 || ((bytes | s0 | s1 | s2 | s3) & 15))
    return fail(MOE_ERR_INVALID_ARG, "%s and the strides must be multiples of 16 bytes", unit);
  return MOE_OK;
}

}  // namespace
}  // namespace wse

using namespace wse;

extern "C" {

int moe_copy_pages(void* k_pool, void* v_pool, int n_layers, int64_t k_layer_stride, int64_t v_layer_stride,
                   int64_t k_page_stride, int64_t v_page_stride, int n_pages, int64_t page_bytes, const int32_t* src,
                   const int32_t* dst, int n, moe_stream_t stream) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n = %d < 0", n);
  int rc = check_pools(k_pool, v_pool, n_layers, k_layer_stride, v_layer_stride, k_page_stride, v_page_stride,
                       n_pages, page_bytes, "page_bytes");
  if (rc != MOE_OK) return rc;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4))
    return fail(MOE_ERR_INVALID_ARG, "src and dst must be non-null and 4-byte aligned");
  CopyPagesArgs a{{static_cast<char*>(k_pool), static_cast<char*>(v_pool)},
                  {k_layer_stride, v_layer_stride},
                  {k_page_stride, v_page_stride},
                  page_bytes, n_pages, 0, src, dst};
  const int64_t chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk;
  if (chunks * n > 0x7fffffffll) return fail(MOE_ERR_UNSUPPORTED, "%d pages of that size: too many for one call", n);
  a.chunks = (int)chunks;
  if ((rc = check_device()) != MOE_OK) return rc;
  return launch_pdl(copy_pages_kernel, dim3((unsigned)(chunks * n), 2u * n_layers), dim3(kCopyThreads), 0, stream, 1,
                    a);
}

int moe_copy_rows(void* k_pool, void* v_pool, int n_layers, int64_t k_layer_stride, int64_t v_layer_stride,
                  int64_t k_page_stride, int64_t v_page_stride, int n_pages, int page_size, int64_t row_bytes,
                  const int64_t* src, const int64_t* dst, int n, moe_stream_t stream) {
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "n = %d < 0", n);
  if (n > MOE_COPY_ROWS_MAX) return fail(MOE_ERR_UNSUPPORTED, "n = %d exceeds %d", n, MOE_COPY_ROWS_MAX);
  int rc = check_pools(k_pool, v_pool, n_layers, k_layer_stride, v_layer_stride, k_page_stride, v_page_stride,
                       n_pages, row_bytes, "row_bytes");
  if (rc != MOE_OK) return rc;
  if (page_size < 1) return fail(MOE_ERR_INVALID_ARG, "page_size = %d < 1", page_size);
  if (n == 0) return MOE_OK;
  if (!src || !dst || !aligned(src, 8) || !aligned(dst, 8))
    return fail(MOE_ERR_INVALID_ARG, "src and dst must be non-null and 8-byte aligned");
  const CopyRowsArgs a{{static_cast<char*>(k_pool), static_cast<char*>(v_pool)},
                       {k_layer_stride, v_layer_stride},
                       {k_page_stride, v_page_stride},
                       row_bytes, (int64_t)n_pages * page_size, page_size, n, src, dst};
  if ((rc = check_device()) != MOE_OK) return rc;
  const unsigned blocks = (unsigned)((row_bytes / 16 + kRowColumns - 1) / kRowColumns);
  return launch_pdl(copy_rows_kernel, dim3(blocks, 2u * n_layers), dim3(kCopyThreads), 0, stream, 1, a);
}

}  // extern "C"
