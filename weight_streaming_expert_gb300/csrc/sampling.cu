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
// what remains is the latency of the exchanges (one takes about 1 us).  So where a
// filter cuts among the 2048 largest logits, as it mostly does, one pass of
// bins finds those down to the cut, the CTAs hand them to the first one in the
// order of their ids, and it goes on alone.  Up to 512 of them it sorts, which
// places both cuts at once, and strikes out what lies behind (top-k 50
// and top-p 0.95: 19 us instead of 31; sorting 2048 would take longer than the
// passes of bins, top-p 0.5 alone 42 us instead of 31).
//
// 6 rows of 157184 logits: greedy 3.3 us, unfiltered 8.0 us, top-k 50 16 us,
// top-k 50 and top-p 0.95 17 us, top-p 0.95 alone (a cut among 20,000 logits)
// 34 us; the logits' bytes are 0.6 us of that.  The kernel for slices in
// shared memory may use 128 registers, as only one such CTA fits an SM: at 64
// it spills, 19 us instead of 17 for both filters.
#include <cooperative_groups.h>

#include <cstddef>

#include "host_util.cuh"
#include "sampling.h"

namespace cg = cooperative_groups;

namespace wse {
namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBinBits = 12, kBins = 1 << kBinBits;  // of a pass, over the whole cluster
constexpr int kBarBits = 10;             // of the pass that finds the kList largest logits
constexpr int kWindowBits = 24;          // the first pass looks at the 2^24 keys from the largest: two to three octaves
constexpr int kMaxCluster = 16;
constexpr float kOne = 274877906944.f;   // 2^38
constexpr int kMaxCached = 40960;        // logits of a slice that fit in shared memory
constexpr uint32_t kKeyNegInf = 0x007fffffu;
constexpr int kList = 2048;              // largest logits that one CTA can go on with
constexpr int kSorted = 512;             // of them, where sorting is faster than more passes of bins
constexpr int kAllTies = 0x7fffffff;
constexpr int kLimbBits = 13;            // of a weight (39 bits) in a bin's three words
constexpr int kMaxSlice = 1 << (32 - kLimbBits);  // a slice's sums of 13-bit parts fit a word

using u64 = unsigned long long;

struct SampleArgs {
  const float* logits;
  int64_t row_stride;
  int vocab, slice;  // logits of a CTA's slice
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

struct alignas(16) Shared {
  uint32_t hist[3][kBins];   // counts, or the sums of the weights' 13-bit parts, then 64-bit sums over the first two
  uint32_t list_key[kList];  // of the first CTA: the largest logits, by id
  int list_id[kList];
  u64 sums[kSampleWarps];    // of this CTA's warps
  u64 scan[2][kMaxCluster];  // written by the other CTAs: their values of an exchange, alternating
  u64 found[3];              // written by the CTA that found it: a pass's bin, the measure before it, its own
  u64 shared[2];             // of this CTA: what one thread computes for the others
  int tie_end;               // written by the CTA that found it
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}
__device__ __forceinline__ u64 warp_max(u64 v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// The CTAs that work on a row, and this one's part of it: n keys, of which each
// thread has `run` in a row (an odd number: consecutive threads then read
// different banks).
template <bool kCached>
struct Team {
  Shared& s;
  cg::cluster_group cluster;
  int rank, size;   // 0 and 1 once the first CTA goes on alone
  bool alone;       // it does, with the list: its keys and their ids
  const float* row; // before that, the slice's logits, whose ids are begin, begin + 1, ..
  int begin;
  int shift;        // and how far into the memory after the struct their keys begin
  int warp, lane;
  unsigned phase;
  int i0, i1;            // this thread's keys

  __device__ void split(int n) {
    const int run = ((n + kSampleThreads - 1) / kSampleThreads) | 1;
    i0 = min(n, (int)threadIdx.x * run);
    i1 = min(n, i0 + run);
  }
  // Keys in shared memory: of the slice after the struct, or the list's.
  __device__ __forceinline__ uint32_t cached(int i) const {
    const int first = alone ? (int)offsetof(Shared, list_key) / 4 : (int)sizeof(Shared) / 4 + shift;
    return reinterpret_cast<const uint32_t*>(&s)[first + i];
  }
  __device__ __forceinline__ uint32_t key(int i) const { return kCached || alone ? cached(i) : key_of(row[i]); }
  // f(i, keys i .. i + 3) for this thread's keys, four at a time so that their
  // latencies overlap; keys past the end are 0, below every key of a logit and
  // of no weight
  template <typename F>
  __device__ __forceinline__ void each4(F f) const {
    uint32_t k[4];
    for (int i = i0; i < i1; i += 4) {
      if (kCached || alone) {
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = i + j < i1 ? cached(i + j) : 0u;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = i + j < i1 ? key_of(row[i + j]) : 0u;
      }
      f(i, k);
    }
  }
  __device__ __forceinline__ int id(int i) const { return alone ? s.list_id[i] : begin + i; }
  __device__ __forceinline__ void sync() {
    if (size > 1)
      cluster.sync();
    else
      __syncthreads();
  }
  template <typename X>
  __device__ __forceinline__ X* peer(X* mine, int r) const {
    return size > 1 ? cluster.map_shared_rank(mine, r) : mine;
  }

  // Sum of the values of the threads before this one, and of all of the CTA.
  __device__ u64 cta_scan(u64 v, u64& total) {
    u64 upto = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const u64 o = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += o;
    }
    __syncthreads();
    if (lane == 31) s.sums[warp] = upto;
    __syncthreads();
    u64 before = upto - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
      const u64 x = s.sums[w];
      if (w < warp) before += x;
      total += x;
    }
    return before;
  }
  // The same over the team.
  __device__ u64 team_scan(u64 v, u64& total) {
    u64 mine;
    const u64 before = cta_scan(v, mine);
    if (size == 1) {
      total = mine;
      return before;
    }
    const u64 other = exchange(mine);
    total = warp_sum(other);
    return warp_sum(lane < rank ? other : 0) + before;
  }
  __device__ u64 team_max(u64 mine) { return size == 1 ? mine : warp_max(exchange(mine)); }
  // Each CTA's value, the same for all of its threads, to every other: lane r
  // gets CTA r's, 0 past the last.  The values are written into the others'
  // memory, which nobody waits for, instead of read out of it, which takes
  // about half a microsecond.  Two slots in turn: a slot is written again only
  // after another exchange, which every CTA enters after it has read this one.
  __device__ u64 exchange(u64 mine) {
    phase ^= 1;
    if (warp == 0 && lane < size) *cluster.map_shared_rank(&s.scan[phase][rank], lane) = mine;
    cluster.sync();
    return lane < size ? s.scan[phase][lane] : 0;
  }

  // The smallest key K in [lo, hi] of the row (of non-zero measure) with
  // measure(keys in (K, hi]) < target; `above` is that measure and `at` the
  // measure of K itself.  0 < target <= measure of the whole range.  With kOnce
  // only as far as the first bin that holds it: lo and `found` are that bin's
  // smallest and largest possible keys, `above` the measure above the bin, `at`
  // the bin's.
  // kParts: words of a bin, 1 for counts and 3 for weights (a 64-bit add in
  // shared memory is a loop of compare-and-swap, three 32-bit adds are not).
  template <int kParts, int kBits, bool kOnce, typename Measure>
  __device__ void select(uint32_t& lo, uint32_t hi, u64 target, Measure measure, uint32_t& found, u64& above, u64& at) {
    constexpr int kWide = kParts == 1 ? 4 : 2;  // bins of a 16-byte read
    constexpr int kUsed = 1 << kBits;           // bins of a pass
    static_assert(kUsed <= kBins && kUsed / kMaxCluster >= kWide);
    above = 0;
    // The first pass looks only near the top, where the filters usually cut:
    // most of the row then touches no bin.  Where the cut lies below, the next
    // pass covers all the rest.
    uint32_t from = hi - lo >= (1u << kWindowBits) ? hi - (1u << kWindowBits) + 1 : lo;
    for (;;) {
      const int shift = max(0, 32 - __clz((int)(hi - from)) - kBits);
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int b = threadIdx.x; b < kUsed / 4; b += kSampleThreads)
          reinterpret_cast<uint4*>(s.hist[q])[b] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      each4([&](int, const uint32_t (&k)[4]) {
        bool in[4], any = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) any |= in[j] = k[j] >= max(from, 1u) && k[j] <= hi;
        if (!any) return;
        u64 w[4];
        measure(k, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t bin = (hi - k[j]) >> shift;
          if (!in[j]) continue;
          if (kParts == 1) {
            atomicAdd(&s.hist[0][bin], (uint32_t)w[j]);
          } else if (w[j]) {
            atomicAdd(&s.hist[0][bin], (uint32_t)w[j] & ((1u << kLimbBits) - 1));
            atomicAdd(&s.hist[1][bin], (uint32_t)(w[j] >> kLimbBits) & ((1u << kLimbBits) - 1));
            atomicAdd(&s.hist[2][bin], (uint32_t)(w[j] >> (2 * kLimbBits)));
          }
        }
      });
      u64* wide = reinterpret_cast<u64*>(s.hist[0]);
      if (kParts > 1 && size > 1) {
        __syncthreads();
        static_assert(kParts == 1 || kUsed % kSampleThreads == 0);
        u64 sum[kUsed / kSampleThreads];
#pragma unroll
        for (int b = 0; b < kUsed / kSampleThreads; ++b) {
          const int at_b = threadIdx.x + b * kSampleThreads;
          sum[b] = s.hist[0][at_b] + ((u64)s.hist[1][at_b] << kLimbBits) + ((u64)s.hist[2][at_b] << (2 * kLimbBits));
        }
        __syncthreads();
#pragma unroll
        for (int b = 0; b < kUsed / kSampleThreads; ++b) wide[threadIdx.x + b * kSampleThreads] = sum[b];
      }
      sync();
      // each CTA sums its share of the bins over the team, a thread a few bins
      // in a row
      const int share = kUsed / size, own_bins = max(kWide, share / kSampleThreads);
      const int first = rank * share + threadIdx.x * own_bins;
      const bool mine = (int)threadIdx.x * own_bins < share;
      auto bins_of = [&](int b, u64 (&sum)[kWide]) {
        const uint4* bins = reinterpret_cast<const uint4*>(kParts == 1 ? (const void*)(s.hist[0] + b) : wide + b);
        auto add = [&](uint4 v) {
          if (kParts == 1) {
            sum[0] += v.x, sum[1] += v.y, sum[kWide - 2] += v.z, sum[kWide - 1] += v.w;
          } else {
            sum[0] += (u64)v.x | (u64)v.y << 32;
            sum[1] += (u64)v.z | (u64)v.w << 32;
          }
        };
        for (int e = 0; e < kWide; ++e) sum[e] = 0;
        if (size == 1) {  // alone: the words as they are
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int e = 0; e < kWide; ++e) sum[e] += (u64)s.hist[q][b + e] << (q * kLimbBits);
          return;
        }
        uint4 v[kMaxCluster];  // all reads under way at once: each takes about half a microsecond
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          v[r] = r < size ? *cluster.map_shared_rank(bins, r) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) add(v[r]);
      };
      u64 own = 0, part[kWide];
      if (mine)
        for (int e = 0; e < own_bins; e += kWide) {
          bins_of(first + e, part);
          for (int i = 0; i < kWide; ++i) own += part[i];
        }
      u64 total;
      u64 before = team_scan(own, total);
      if (from > lo && above + total < target) {
        above += total;
        hi = from - 1;
        from = lo;
        continue;
      }
      before += above;
      // the bin that the target falls into is one thread's, whose warp tells all
      const bool here = mine && before < target && before + own >= target;
      const unsigned vote = __ballot_sync(0xffffffffu, here);
      if (vote) {
        int b = first;
        u64 bin = 0;
        if (here)
          for (bool done = false; !done; b += kWide) {
            bins_of(b, part);
            for (int i = 0; i < kWide && !done; ++i) {
              bin = part[i];
              done = before + bin >= target;
              if (done)
                b += i - kWide;
              else
                before += bin;
            }
          }
        const int src = __ffs(vote) - 1;
        b = __shfl_sync(0xffffffffu, b, src);
        before = __shfl_sync(0xffffffffu, before, src);
        bin = __shfl_sync(0xffffffffu, bin, src);
        if (lane < size) {
          u64* f = peer(s.found, lane);
          f[0] = b;
          f[1] = before;
          f[2] = bin;
        }
      }
      sync();
      above = s.found[1];
      at = s.found[2];
      hi -= (uint32_t)s.found[0] << shift;
      if (hi - from >= (1u << shift)) from = hi - (1u << shift) + 1;
      lo = from;
      if (from == hi || kOnce) break;
    }
    found = hi;
  }
};

// The lowest whole number that is not below x as a double: n < whole_of(x) is
// the same as (double)n < x, which rounds above 2^53.
__device__ u64 whole_of(double x) {
  u64 n = (u64)ceil(x);
  if (x < 0x1p53) return n;
  for (u64 d = 1024; d > 0; d >>= 1)
    while (n >= d && (double)(n - d) >= x) n -= d;
  return n;
}

// Sorts n words in shared memory by falling value, n a power of two from 64 to
// 1024: a bitonic network, whose steps over distances below 64 stay in a warp.
__device__ void sort_falling(u64* a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      const int i = threadIdx.x, lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
      if (i < n / 2) {
        const u64 x = a[lo], y = a[hi];
        if ((x < y) == ((lo & k) == 0)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      if (j >= 64 || (j == 1 && k >= 64))
        __syncthreads();
      else
        __syncwarp();
    }
}

struct Ones {
  __device__ void operator()(const uint32_t (&)[4], u64 (&w)[4]) const { w[0] = w[1] = w[2] = w[3] = 1; }
};

// x / y to about one unit in the last place: each as the sum of two fp32
// numbers, the quotient of the larger ones corrected once by its remainder.
__device__ float quotient(u64 x, u64 y) {
  const float xh = (float)x, yh = (float)y;
  const float xl = (float)(long long)(x - (u64)xh), yl = (float)(long long)(y - (u64)yh);
  const float q = xh / yh;
  return q + (fmaf(-q, yh, xh) + fmaf(-q, yl, xl)) / yh;
}

template <bool kCached>
__global__ void __launch_bounds__(kSampleThreads, kCached ? 1 : 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const long long m = blockIdx.x / size;
  cluster_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const float t = a.temperature ? a.temperature[m] : 1.f, p = a.top_p ? a.top_p[m] : 1.f;
  const float min_p = a.min_p ? a.min_p[m] : 0.f, u = a.u[m];
  const int k = a.top_k ? a.top_k[m] : 0;
  const int begin = min(rank * a.slice, a.vocab), n = min(a.slice, a.vocab - begin);
  const float* row = a.logits + m * a.row_stride + begin;
  const int shift = (int)(reinterpret_cast<uintptr_t>(row) / 4) & 3;  // logits from a 16-byte border on
  uint32_t* cache = reinterpret_cast<uint32_t*>(smem + sizeof(Shared)) + shift;
  Team<kCached> c{s, cluster, rank, size, false, row, begin, shift, tid >> 5, tid & 31, 0, 0, 0};
  c.split(n);

  // the row's largest logit, the lowest id first
  uint32_t best_key = 0;
  int best_i = 0;
  auto take = [&](int i, uint32_t key) {
    if (kCached) cache[i] = key;
    if (key > best_key) best_key = key, best_i = i;
  };
  // four at a time from the first one at a 16-byte border
  const int head = min(n, -c.shift & 3), fours = (n - head) / 4;
  if (tid < head) take(tid, key_of(row[tid]));
  constexpr int kLoads = 8;  // in flight
  for (int g0 = tid; g0 < fours; g0 += kLoads * kSampleThreads) {
    float4 v[kLoads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l)
      if (g0 + l * kSampleThreads < fours)
        v[l] = reinterpret_cast<const float4*>(row + head)[g0 + l * kSampleThreads];
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int g = g0 + l * kSampleThreads, i = head + 4 * g;
      if (g >= fours) break;
      const uint4 key = make_uint4(key_of(v[l].x), key_of(v[l].y), key_of(v[l].z), key_of(v[l].w));
      if (kCached) reinterpret_cast<uint4*>(cache + head)[g] = key;
      const uint32_t most = max(max(key.x, key.y), max(key.z, key.w));
      if (most > best_key)
        best_key = most, best_i = i + (key.x == most ? 0 : key.y == most ? 1 : key.z == most ? 2 : 3);
    }
  }
  if (tid < n - head - 4 * fours) take(head + 4 * fours + tid, key_of(row[head + 4 * fours + tid]));
  u64 best = warp_max((u64)best_key << 32 | (uint32_t)~(begin + best_i));
  if (c.lane == 0) s.sums[c.warp] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSampleWarps; ++w) best = max(best, s.sums[w]);
  cluster_wait();  // every CTA of the cluster has begun, before the first writes into another's memory
  best = c.team_max(best);
  const uint32_t top_key = (uint32_t)(best >> 32);
  const float top = logit_of(top_key);
  if (top_key <= kKeyNegInf || !(t > 0.f)) {
    if (rank == 0 && tid == 0) {
      a.tokens[m] = top_key <= kKeyNegInf ? -1 : (int)~(uint32_t)best;
      if (a.probs) a.probs[m] = top_key <= kKeyNegInf ? 0.f : 1.f;
    }
    return;
  }
  // d / t, correctly rounded like the operator: a quotient off by at most one
  // unit in the last place, corrected by its exact remainder with a correctly
  // rounded reciprocal, is (Markstein, IBM J. Res. Dev. 34, 1990), as long as
  // nothing leaves the normal range on the way.  Where d is so small that it
  // does, exp gives 1 either way; where d / t overflows the remainder is NaN,
  // which counts as infinitely far below like an infinite d.
  const float inverse = __frcp_rn(t);
  const bool tame = t > 1e-4f && t < 1e4f && top < INFINITY;
  // exp((l - l0) / t) of four keys, without a branch between them; 0 for what
  // is infinitely far below (also at an infinite temperature)
  auto exps = [&](const uint32_t (&key)[4], float (&e)[4]) {
    float z[4];
    if (tame) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float d = logit_of(key[j]) - top, q = d * inverse;
        z[j] = fmaf(fmaf(-q, t, d), inverse, q);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = key[j] == top_key ? 0.f : (logit_of(key[j]) - top) / t;  // top may be infinite
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = fmaxf(expf(z[j]), 0.f);  // of NaN and 0: 0
  };
  // floor(2^38 e) as a high and a low word of 19 bits (e = 1: 2^19 and 0).
  // Adding 2^23 towards minus infinity leaves the whole part in the low bits,
  // and both remainders are exact; conversions would take four times as long.
  auto split = [](float e, uint32_t& high, uint32_t& low) {
    const float h = __fadd_rd(e * 0x1p19f, 0x1p23f);
    high = __float_as_uint(h) & 0x7fffffu;
    low = __float_as_uint(__fadd_rd(fmaf(e, 0x1p38f, (h - 0x1p23f) * -0x1p19f), 0x1p23f)) & 0x7fffffu;
  };
  auto weights = [&](const uint32_t (&key)[4], u64 (&w)[4]) {
    float e[4];
    exps(key, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t high, low;
      split(e[j], high, low);
      w[j] = ((u64)high << 19) + low;
    }
  };
  auto weight = [&](uint32_t key) {
    const uint32_t k[4] = {key, 0u, 0u, 0u};
    u64 w[4];
    weights(k, w);
    return w[0];
  };
  // Weight of this thread's keys from `bar` on, of at least `least`, up to id
  // tie_end for those of key bar itself.  A thread has at most 1025 keys, whose
  // high and low words sum to less than 2^32.
  auto mass_from = [&](uint32_t bar, float least, int tie_end) {
    uint32_t high = 0, low = 0;
    c.each4([&](int i, const uint32_t (&key)[4]) {
      if (max(max(key[0], key[1]), max(key[2], key[3])) < bar) return;
      float e[4];
      exps(key, e);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bool stays = key[j] >= bar && e[j] >= least;
        if (tie_end != kAllTies) stays = stays && (key[j] != bar || c.id(i + j) <= tie_end);
        uint32_t h, l;
        split(stays ? e[j] : 0.f, h, l);
        high += h;
        low += l;
      }
    });
    return ((u64)high << 19) + low;
  };

  const bool by_count = k > 0 && k < a.vocab, by_mass = p < 1.f;
  u64 above, at, total, target = 0;  // target: what top-p leaves, once its share is known
  auto share_of = [&](u64 mass) {
    // 64-bit arithmetic is slow on this GPU: one thread does it for all
    if (tid == 0) {
      const double limit = (double)p * (double)mass;
      s.shared[0] = limit > 0. ? whole_of(limit) : 1;  // 1: the first token stays in any case
    }
    __syncthreads();
    return s.shared[0];
  };
  if (by_mass && !by_count) {
    c.team_scan(mass_from(0, 0.f, kAllTies), total);
    target = share_of(total);
  }
  // the first cut is in [cut_lo, cut_hi], with `before_cut` above
  uint32_t cut_lo = 0, cut_hi = top_key;
  u64 before_cut = 0;
  if (by_count ? k <= kList : by_mass) {
    // the keys down to the bin that the first cut falls into, and how many of
    // them this thread has
    if (a.vocab > kList) {
      if (by_count)
        c.template select<1, kBarBits, true>(cut_lo, top_key, (u64)k, Ones{}, cut_hi, before_cut, at);
      else
        c.template select<3, kBarBits, true>(cut_lo, top_key, target, weights, cut_hi, before_cut, at);
    }
    const uint32_t bar = max(cut_lo, 1u);  // 0 is no key
    u64 count = 0;
    c.each4([&](int, const uint32_t (&key)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) count += key[j] >= bar;
    });
    const int to = (int)c.team_scan(count, total);
    if (total <= kList) {
      uint32_t* list_key = c.peer(s.list_key, 0) + to;
      int* list_id = c.peer(s.list_id, 0) + to;
      if (count)
        c.each4([&](int i, const uint32_t (&key)[4]) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (key[j] >= bar) {
              *list_key++ = key[j];
              *list_id++ = begin + i + j;
            }
        });
      c.sync();
      if (rank != 0) return;
      c.size = 1;
      c.alone = true;
      c.split((int)total);
    }
  }

  const bool sorted = c.alone && total <= kSorted;
  if (sorted) {
    // by falling key and rising id: the list's order is that of the ids
    u64* order = reinterpret_cast<u64*>(s.hist);
    const int n_list = (int)total;
    int padded = 64;
    while (padded < n_list) padded *= 2;
    if (tid < padded) order[tid] = tid < n_list ? (u64)s.list_key[tid] << 32 | (uint32_t)~tid : 0;
    __syncthreads();
    sort_falling(order, padded);
    int stay = by_count ? min(k, n_list) : n_list;
    if (by_mass) {
      // the weights before each, in that order
      const u64 w = tid < stay ? weight((uint32_t)(order[tid] >> 32)) : 0;
      const u64 before = c.cta_scan(w, total);
      if (by_count) target = share_of(total);
      stay = __syncthreads_count(tid < stay && before < target);
    }
    // what does not stay is no key any more
    if (tid >= stay && tid < n_list) s.list_key[~(uint32_t)order[tid]] = 0;
    __syncthreads();
  }

  // the tokens that stay: keys above thr, and of the tokens whose key is thr
  // those up to id tie_end
  uint32_t thr = 1;
  int tie_end = kAllTies;
  u64 ties = 0, same = 0;  // how many of the `same` tokens of key thr stay
  if (by_count && !sorted) {
    c.template select<1, kBinBits, false>(cut_lo, cut_hi, (u64)k - before_cut, Ones{}, thr, above, at);
    ties = (u64)k - before_cut - above;  // at most `at`: k is reached there
    same = at;
  }
  if (by_mass && !sorted) {
    if (by_count) {
      c.team_scan(mass_from(thr + 1, 0.f, kAllTies), total);
      target = share_of(total + ties * weight(thr));
      cut_lo = thr, cut_hi = top_key, before_cut = 0;
    }
    uint32_t key;
    target -= before_cut;
    c.template select<3, kBinBits, false>(cut_lo, cut_hi, target, weights, key, above, at);
    const u64 w = weight(key);
    if (at == w) {
      ties = same = 1;
    } else {
      if (tid == 0) {
        const u64 every = at / w, fit = (target - above + w - 1) / w;
        s.shared[0] = min(fit, key == thr && same ? ties : every);
        s.shared[1] = every;
      }
      __syncthreads();
      ties = s.shared[0];
      same = s.shared[1];
    }
    thr = key;
  }
  if (same && ties < same) {
    // the id of the last of them: the thread that holds it tells all
    u64 count = 0;
    c.each4([&](int, const uint32_t (&key)[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) count += key[j] == thr;
    });
    u64 before = c.team_scan(count, total);
    if (before < ties && ties <= before + count) {
      int i = c.i0;
      for (;; ++i)
        if (c.key(i) == thr && ++before == ties) break;
      for (int r = 0; r < c.size; ++r) *c.peer(&s.tie_end, r) = c.id(i);
    }
    c.sync();
    tie_end = s.tie_end;
  }
  // w >= min_p 2^38 is e >= the least multiple of 2^-38 that is not below
  // min_p: exact in fp32, as 2^38 e and min_p have 24 bits
  const float least = min_p > 0.f ? ceilf(fminf(min_p, 1.f) * kOne) * 0x1p-38f : 0.f;
  const u64 sum = mass_from(thr, least, tie_end);
  u64 before = c.team_scan(sum, total);
  if (tid == 0) s.shared[0] = min((u64)((double)u * (double)total), total - 1);
  __syncthreads();
  const u64 wanted = s.shared[0];
  const unsigned here = __ballot_sync(0xffffffffu, wanted >= before && wanted < before + sum);
  if (here) {  // the token is one of a thread's of this warp: its lanes look through them
    const int src = __ffs(here) - 1;
    const int from = __shfl_sync(0xffffffffu, c.i0, src), to = __shfl_sync(0xffffffffu, c.i1, src);
    before = __shfl_sync(0xffffffffu, before, src);
    for (int i = from + c.lane; i - c.lane < to; i += 32) {
      const uint32_t key[4] = {i < to ? c.key(i) : 0u, 0u, 0u, 0u};
      float e[4];
      exps(key, e);
      const bool stays = i < to && key[0] >= thr && e[0] >= least && (key[0] != thr || c.id(i) <= tie_end);
      uint32_t high, low;
      split(stays ? e[0] : 0.f, high, low);
      const u64 w = ((u64)high << 19) + low;
      u64 upto = w;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, upto, d);
        if (c.lane >= d) upto += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > wanted);
      if (past) {
        if (c.lane == __ffs(past) - 1) {
          a.tokens[m] = c.id(i);
          if (a.probs) a.probs[m] = quotient(w, total);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  // whoever leaves has passed a barrier after all that others do in its memory
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
  static_assert(MOE_SAMPLE_MAX_VOCAB / kMaxCluster <= kMaxSlice && kMaxCached <= kMaxSlice);
  static_assert(sizeof(Shared) % 16 == 0 && sizeof(Shared) + (kMaxCached + 3) * 4 <= 227 * 1024);
  constexpr int kSmem = (int)sizeof(Shared) + (kMaxCached + 3) * 4;
  static thread_local int ready = -1;                // device that this thread has set up
  static thread_local int resident[kMaxCluster + 1];  // clusters of a size that run at once there
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    for (auto kernel : {sample_kernel<true>, sample_kernel<false>}) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    }
    for (int size = 2; size <= kMaxCluster && e == cudaSuccess; size *= 2) {
      cudaLaunchAttribute in_clusters{};
      in_clusters.id = cudaLaunchAttributeClusterDimension;
      in_clusters.val.clusterDim.x = size;
      in_clusters.val.clusterDim.y = in_clusters.val.clusterDim.z = 1;
      cudaLaunchConfig_t config{};
      config.gridDim = dim3((unsigned)size);
      config.blockDim = dim3(kSampleThreads);
      config.dynamicSmemBytes = kSmem;
      config.attrs = &in_clusters;
      config.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&resident[size], sample_kernel<true>, &config);
    }
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return fail_cuda(e, "sampling set-up");
  // CTAs of a row: as many as let all rows run at once, a CTA per SM (7
  // clusters of 16, 15 of 8, 36 of 4, 76 of 2: the groups of SMs that a cluster
  // cannot leave are not all whole): 16 rows of 157184, top-k 50: 32 us with 8,
  // in two waves, 25 us with 4 (top-p 0.95 54 and 56 us).  But not so few that a slice leaves shared memory:
  // 64 rows 48 us with 4, in two waves, 68 us with 2, which read the row from
  // L2 in every pass.
  int cluster = kMaxCluster;
  while (cluster > 1 && (rows > resident[cluster] || (vocab + cluster - 1) / cluster < kSampleThreads) &&
         (vocab + cluster / 2 - 1) / (cluster / 2) <= kMaxCached)
    cluster /= 2;
  SampleArgs a{logits, row_stride, vocab, (vocab + cluster - 1) / cluster, u, temperature, top_k, top_p, min_p,
               tokens, probs};
  const bool cached = a.slice <= kMaxCached;
  const size_t smem = sizeof(Shared) + (cached ? (size_t)(a.slice + 3) * 4 : 0);
  return launch_pdl(cached ? sample_kernel<true> : sample_kernel<false>, dim3((unsigned)(rows * cluster)),
                    dim3(kSampleThreads), smem, stream, cluster, a);
}
