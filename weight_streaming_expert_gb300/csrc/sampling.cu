// sampling.cu -- one token per row of logits with temperature, top-k, top-p
// and min-p, from a given uniform number (include/sampling.h).
//
// A row's weights are whole numbers, w_i = floor(2^38 exp((l_i - l0) / T)),
// so every sum below is exact and the same in any order.  With the logits as
// order-preserving integer keys both filters ask the same question: the
// smallest key K in the row such that measure(keys > K) < target, where the
// measure counts tokens (top-k: target k) or sums weights (top-p: target
// p times the weight that top-k left).  It is answered by histograms of
// falling key, each pass refining the bin that holds K.
//
// A row belongs to one thread-block cluster: its CTAs take contiguous slices
// of the vocabulary, hold them in shared memory, and exchange maxima, bins and
// sums through distributed shared memory.  The row is read from memory once;
// what remains is the latency of about a dozen cluster-wide exchanges.
#include <cooperative_groups.h>

#include "host_util.cuh"
#include "sampling.h"

namespace cg = cooperative_groups;

namespace wse {
namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = kSampleThreads;    // of a pass, over the whole cluster
constexpr int kBinBits = 9;
constexpr int kFirstShift = 15;          // the first pass resolves 2^24 keys below the largest: two to three octaves
constexpr int kMaxCluster = 16;
constexpr float kOne = 274877906944.f;   // 2^38
constexpr int kMaxCached = 49152;        // logits of a slice that fit in shared memory
constexpr uint32_t kKeyNegInf = 0x007fffffu;

using u64 = unsigned long long;

struct SampleArgs {
  const float* logits;
  int64_t row_stride;
  int vocab, slice;  // logits of a CTA's slice
  bool cached;       // the slice is held in shared memory
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* probs;
};

// Order-preserving key of a logit: NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (l != l) l = -INFINITY;
  const uint32_t b = __float_as_uint(l + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct Shared {
  u64 hist[kBins];
  u64 sums[kSampleWarps];
  u64 scan[2];   // read by the other CTAs: the CTA's value of a scan, alternating
  u64 found[3];  // read by the other CTAs: a pass's bin + 1 (0: none), the measure before it, its own
  unsigned best;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

struct Cta {
  Shared& s;
  cg::cluster_group cluster;
  int rank, size;
  const float* data;  // this CTA's slice, in shared or global memory
  int seg0, seg1;     // this warp's contiguous part of it
  int warp, lane;
  unsigned phase;

  // Sum of `v` over the CTA (v: one value per warp, uniform in it).
  __device__ u64 cta_sum(u64 v) {
    __syncthreads();
    if (lane == 0) s.sums[warp] = v;
    __syncthreads();
    u64 total = 0;
    for (int w = 0; w < kSampleWarps; ++w) total += s.sums[w];
    return total;
  }
  // Over the cluster: the sum of the CTAs' values before this one, and of all.
  // Two slots in turn: a slot is written again only after another exchange,
  // which every CTA enters after it has read this one.
  __device__ void cluster_scan(u64 mine, u64& below, u64& total) {
    phase ^= 1;
    if (threadIdx.x == 0) s.scan[phase] = mine;
    cluster.sync();
    below = total = 0;
    for (int r = 0; r < size; ++r) {
      const u64 v = *cluster.map_shared_rank(&s.scan[phase], r);
      if (r < rank) below += v;
      total += v;
    }
  }
  __device__ u64 cluster_max(u64 mine) {
    phase ^= 1;
    if (threadIdx.x == 0) s.scan[phase] = mine;
    cluster.sync();
    u64 top = 0;
    for (int r = 0; r < size; ++r) top = max(top, *cluster.map_shared_rank(&s.scan[phase], r));
    return top;
  }

  // The smallest key K in [lo, hi] of the row (of non-zero measure) with
  // measure(keys in (K, hi]) < target; `above` is that measure and `at` the
  // measure of K itself.  target > 0 and hi is in the row.
  template <typename Measure>
  __device__ void select(uint32_t lo, uint32_t hi, double target, Measure measure, uint32_t& key, u64& above,
                         u64& at) {
    above = 0;
    for (bool first = true;; first = false) {
      const uint32_t range = hi - lo;  // keys - 1
      const int fit = max(0, 32 - __clz((int)range) - kBinBits);
      const int shift = first ? min(kFirstShift, fit) : fit;
      s.hist[threadIdx.x] = 0;
      if (threadIdx.x == 0) s.best = 0;
      __syncthreads();
      for (int i = seg0 + lane; i < seg1; i += 32) {
        const uint32_t k = key_of(data[i]);
        if (k < lo || k > hi) continue;
        const u64 m = measure(k);
        if (m) atomicAdd(&s.hist[min((hi - k) >> shift, (uint32_t)kBins - 1)], m);
      }
      cluster.sync();
      // each CTA sums its share of the bins over the cluster, one per thread
      const int per = kBins / size;
      const bool mine = (int)threadIdx.x < per;
      u64 bin = 0;
      if (mine)
        for (int r = 0; r < size; ++r) bin += cluster.map_shared_rank(s.hist, r)[rank * per + threadIdx.x];
      u64 upto = bin;  // inclusive scan over the share
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += o;
      }
      const u64 share = cta_sum(__shfl_sync(0xffffffffu, upto, 31));
      for (int w = 0; w < warp; ++w) upto += s.sums[w];
      u64 below, total;
      cluster_scan(share, below, total);
      const u64 before = above + below + upto - bin;
      const bool good = bin > 0 && (double)before < target;
      if (good) atomicMax(&s.best, threadIdx.x + 1);
      __syncthreads();
      if (s.best == 0 && threadIdx.x == 0) s.found[0] = 0;
      if (good && s.best == threadIdx.x + 1) {
        s.found[0] = rank * per + threadIdx.x + 1;
        s.found[1] = before;
        s.found[2] = bin;
      }
      cluster.sync();
      u64 b = 1;
      for (int r = size - 1; r >= 0; --r) {
        const u64* f = cluster.map_shared_rank(s.found, r);
        if (f[0]) {
          b = f[0];
          above = f[1];
          at = f[2];
          break;
        }
      }
      const uint32_t top = hi - ((uint32_t)(b - 1) << shift);
      if (b < (u64)kBins && top - lo >= (1u << shift)) lo = top - (1u << shift) + 1;
      hi = top;
      if (lo == hi) break;
    }
    key = hi;
  }
};

__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ float cache[];
  __shared__ Shared s;
  const int tid = threadIdx.x;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long m = blockIdx.x / size;
  pdl_wait();
  pdl_launch_dependents();
  const int begin = min(rank * a.slice, a.vocab);
  const int n = min(a.slice, a.vocab - begin);
  const float* row = a.logits + m * a.row_stride + begin;
  const int seg = (n + kSampleThreads - 1) / kSampleThreads * 32;
  Cta c{s, cluster, rank, size, a.cached ? cache : row, 0, 0, tid >> 5, tid & 31, 0};
  c.seg0 = min(n, c.warp * seg);
  c.seg1 = min(n, c.seg0 + seg);

  // the row's largest logit, the lowest id first
  u64 best = 0;
#pragma unroll 8
  for (int i = c.seg0 + c.lane; i < c.seg1; i += 32) {
    const float l = row[i];
    if (a.cached) cache[i] = l;
    best = max(best, (u64)key_of(l) << 32 | (uint32_t)~(begin + i));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, d));
  if (c.lane == 0) s.sums[c.warp] = best;
  __syncthreads();
  for (int w = 0; w < kSampleWarps; ++w) best = max(best, s.sums[w]);
  best = c.cluster_max(best);
  const uint32_t top_key = (uint32_t)(best >> 32);
  const float top = logit_of(top_key);
  const float t = a.temperature ? a.temperature[m] : 1.f;
  if (top_key <= kKeyNegInf || !(t > 0.f)) {
    if (rank == 0 && tid == 0) {
      a.tokens[m] = top_key <= kKeyNegInf ? -1 : (int)~(uint32_t)best;
      if (a.probs) a.probs[m] = top_key <= kKeyNegInf ? 0.f : 1.f;
    }
    cluster.sync();  // the others may still read this CTA's maximum
    return;
  }
  auto weight = [&](uint32_t key) -> u64 {
    const float l = logit_of(key);
    if (l == top) return (u64)kOne;  // an infinite one too
    const float z = (l - top) / t;
    return z == z ? (u64)(expf(z) * kOne) : 0;  // infinitely far below at an infinite temperature: 0
  };

  // the tokens that stay: keys above thr and the first `ties` of the `same`
  // tokens whose key is thr
  uint32_t thr = 0;
  u64 ties = ~0ull, same = 0;
  const int k = a.top_k ? a.top_k[m] : 0;
  const float p = a.top_p ? a.top_p[m] : 1.f;
  u64 above, at, total;
  if (k > 0 && k < a.vocab) {
    c.select(0, top_key, (double)k, [](uint32_t) -> u64 { return 1; }, thr, above, at);
    ties = min((u64)k - above, at);
    same = at;
  }
  if (p < 1.f) {
    u64 sum = 0, below;
    for (int i = c.seg0 + c.lane; i < c.seg1; i += 32) {
      const uint32_t key = key_of(c.data[i]);
      if (key > thr) sum += weight(key);
    }
    c.cluster_scan(c.cta_sum(warp_sum(sum)), below, total);
    const u64 at_thr = same ? weight(thr) : 0;
    total += same ? ties * at_thr : 0;
    double target = (double)p * (double)total;
    if (!(target > 0.)) target = 0.5;  // the first token stays in any case
    uint32_t key;
    c.select(thr, top_key, target, weight, key, above, at);
    const u64 w = weight(key), all = at / w;
    u64 fit = (u64)fmax(1., ceil((target - (double)above) / (double)w));
    // the last of them by the definition's own comparison
    while (fit > 1 && !((double)(above + (fit - 1) * w) < target)) --fit;
    while ((double)(above + fit * w) < target) ++fit;
    ties = min(fit, key == thr && same ? ties : all);
    same = all;
    thr = key;
  }
  const bool partial = same && ties < same;
  const double least = a.min_p ? (double)fminf(a.min_p[m], 1.f) * (double)kOne : 0.;

  // tokens of key thr before this warp's part, where only some of them stay
  u64 tie0 = 0;
  if (partial) {
    u64 mine = 0, all;
    for (int i = c.seg0 + c.lane; i < c.seg1; i += 32) mine += key_of(c.data[i]) == thr;
    mine = c.cta_sum(warp_sum(mine));
    c.cluster_scan(mine, tie0, all);
    for (int w = 0; w < c.warp; ++w) tie0 += s.sums[w];
  }
  // weight of element i (0: it does not stay), all lanes of a warp in step
  auto staying = [&](int i, u64& tie) -> u64 {
    const uint32_t key = i < c.seg1 ? key_of(c.data[i]) : 0u;
    bool stays = i < c.seg1 && (key > thr || !same || key == thr);
    if (partial) {
      const unsigned eq = __ballot_sync(0xffffffffu, i < c.seg1 && key == thr);
      if (key == thr) stays = stays && tie + __popc(eq & ((1u << c.lane) - 1)) < ties;
      tie += __popc(eq);
    }
    if (!stays || (same && key < thr)) return 0;
    const u64 w = weight(key);
    return (double)w >= least ? w : 0;
  };
  u64 sum = 0, tie = tie0, below;
  for (int i = c.seg0; i < c.seg1; i += 32) sum += staying(i + c.lane, tie);
  sum = warp_sum(sum);
  const u64 mine = c.cta_sum(sum);
  c.cluster_scan(mine, below, total);
  const u64 wanted = min((u64)((double)a.u[m] * (double)total), total - 1);
  for (int w = 0; w < c.warp; ++w) below += s.sums[w];
  if (wanted >= below && wanted < below + sum) {  // the token lies in this warp's part
    tie = tie0;
    u64 base = below;
    for (int i = c.seg0; i < c.seg1; i += 32) {
      const u64 w = staying(i + c.lane, tie);
      u64 upto = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
        if (c.lane >= d) upto += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + upto > wanted);
      if (past) {
        if (c.lane == __ffs(past) - 1) {
          a.tokens[m] = begin + i + c.lane;
          if (a.probs) a.probs[m] = (float)((double)w / (double)total);
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  cluster.sync();  // no CTA leaves while another may read its sums
}

}  // namespace
}  // namespace wse

using namespace wse;

extern "C" int moe_sample(const float* logits, int64_t row_stride, int rows, int vocab, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                          int32_t* tokens, float* probs, moe_stream_t stream) {
  if (rows < 0 || rows > 65535) return fail(MOE_ERR_INVALID_ARG, "rows = %d: must be in 0..65535", rows);
  if (vocab < 1 || vocab > MOE_SAMPLE_MAX_VOCAB)
    return fail(MOE_ERR_INVALID_ARG, "vocab = %d: must be in 1..%d", vocab, MOE_SAMPLE_MAX_VOCAB);
  if (rows == 0) return MOE_OK;
  if (!logits || !u || !tokens) return fail(MOE_ERR_INVALID_ARG, "null logits, u or tokens");
  if (!aligned(logits, 4) || !aligned(u, 4) || !aligned(tokens, 4) || !aligned(temperature, 4) ||
      !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(probs, 4))
    return fail(MOE_ERR_INVALID_ARG, "every array must be 4-byte aligned");
  if (row_stride < vocab && rows > 1)
    return fail(MOE_ERR_INVALID_ARG, "row_stride = %lld is smaller than vocab", (long long)row_stride);
  int rc = check_device();
  if (rc != MOE_OK) return rc;
  int cluster = kMaxCluster;
  while (cluster > 1 && (rows * cluster > 1024 || (vocab + cluster - 1) / cluster < kSampleThreads)) cluster /= 2;
  SampleArgs a{logits, row_stride, vocab, (vocab + cluster - 1) / cluster, false, u, temperature, top_k, top_p, min_p,
               tokens, probs};
  a.cached = a.slice <= kMaxCached;
  const size_t smem = a.cached ? (size_t)a.slice * 4 : 0;
  static thread_local int ready = -1;  // device whose kernel attributes this thread has set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    if ((e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4)) ==
        cudaSuccess)
      e = cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return fail_cuda(e, "sampling set-up");
  return launch_pdl(sample_kernel, dim3((unsigned)(rows * cluster)), dim3(kSampleThreads), smem, stream, cluster, a);
}
