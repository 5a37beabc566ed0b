// paged_attention.cu -- attention of a chunk of new tokens over a paged cache
// (include/attention.h), on the fifth-generation tensor cores.
//
// For a query row q (one token, one head) over the positions it sees:
//   s_j = q.k_j,  m = max_j s_j,  p_j = 2^(c (s_j - m)) with c = scale log2 e,
//   out = sum_j p_j v_j / sum_j p_j,
// in one pass over the positions with a running m: when m grows, what was
// summed so far is multiplied by 2^(c (m_old - m_new)).  Any m gives the same
// quotient, so the sums are only rescaled when m has grown by a factor of more
// than 2^8 in p (p then stays below 2^8: exact enough in fp32 sums, and in
// range for 16-bit probabilities); most rows rescale once or twice in all.
//
// A tile is up to 128 query rows: as many whole tokens of the chunk as fit,
// each with the heads that share a key/value head, so that a page is read once
// for all of them.  Per 64 positions one warp issues S = Q K^T into TMEM (128 x
// 64 fp32), four warps turn S into probabilities, one row a thread with no
// exchange between threads, and write them over S as the 16-bit A operand of
// O += P V, which stays in TMEM.  Each probability is rounded once to the
// element type, as the MMA takes both operands in one 16-bit type: against 64
// bits the outputs are then 1.35 times as far off as by their own rounding
// alone; scores, statistics and sums are fp32.  Two such chains run side by
// side, so that one's products cover the other's exponentials (two tiles in
// turn, and rescaling only where the maximum has grown, are published ideas for
// attention kernels):
//   pair   two tiles of rows over the same positions (chunks of many rows);
//   split  one tile, the even 128 positions in one chain and the odd ones in
//          the other, merged at the end (chunks of up to 128 rows, which are
//          bound by reading the cache).
// A chain has two buffers of 64 positions.  In the pair form the next scores go
// into the one while the softmax works on the other: S as 128 x 64 takes 413
// clocks where 128 x 128 takes 268 for the same positions (the MMA then waits
// for its operands in shared memory), but a chain that waited for its scores
// took 3060 clocks for 128 positions and now takes 2800 (8192 tokens over
// 16384, 32/4 heads of 128: 1375 us before, 1205 us).  The split form waits
// for memory anyway and takes both buffers' scores at once.
// One warp copies the pages with TMA into a ring of 128-position tiles, another
// the queries of the next tile, and in the pair form a third looks through the
// values of positions that some rows do not see.
//
// The work is a list of (sequence, key/value head, tile of rows, 128
// positions) in that order.  Every CTA takes a contiguous share of equal cost,
// computed on the device from the lengths that the call finds there: one long
// sequence spreads over all SMs, many short ones share an SM, and a captured
// graph adapts to lengths that change.  A tile that a boundary cuts leaves
// unnormalised sums with their m; a second, small kernel joins them in a fixed
// order.
//
// What bounds it, and what it reaches on one GB300 (copy 6687 GB/s, bf16 GEMM
// 1897 TFLOP/s in a burst and 1727 sustained):
//   long chunks      the tensor pipe: 2650 of the 2800 clocks per 256 rows by
//                    128 positions are MMAs.  8192 tokens over 16384: 1.17 ms,
//                    1410 TFLOP/s, in a graph, 1.19 ms as a call among others.
//   long decoding    reading the cache: 32 sequences of 2,000 to 32,768
//                    positions, one token each: 132 us, 6.3 TB/s.
//   short calls      latencies: the plan, the first pages, one softmax, the
//                    join: 6 tokens over 8192: 13 us, of which memory needs 2.5.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "attention.h"
#include "host_util.cuh"
#include "tcgen05.cuh"

namespace wse {
namespace {

enum : int { kAttnBadPage = 1, kAttnBadLength = 2, kAttnTimeout = 4 };

constexpr int kTile = 128;                 // query rows of a tile, and positions
constexpr int kHalf = 64;                  // positions of a softmax step
// Two softmax warpgroups, then a warp each for MMAs, copies and queries, and in
// the pair form one for veiled values.
constexpr int kMmaWarp = 8, kCopyWarp = 9, kQueryWarp = 10, kValueWarp = 11;
constexpr int kMaxBatch = 4096;
constexpr int kMaxStages = 10;
constexpr uint32_t kStagingBytes = 8 * 4096;  // 32 rows of 128 bytes for each softmax warp
constexpr float kRescaleLog2 = 8.f;
constexpr int kJoinRows = 4, kJoinGroups = 4;  // rows of a joining CTA, and threads that share a row's parts
constexpr int kFewParts = 4;
constexpr int kMaxSpread = 8;              // key/value heads that neighbouring CTAs work on side by side

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
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t pair_of(uint32_t x, uint32_t y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  return pair_of(__float_as_uint(x), __float_as_uint(y));
}
__device__ __forceinline__ float low_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ void max3(float& top, uint32_t x, uint32_t y) {
  asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
}

// A tile that was cut at the end of CTA c's share: joined from the partial sums
// of CTAs c, c + spread, .., `parts` of them (0: no such tile).
struct Cut {
  int parts, c, b, h, tile;
};
constexpr double kMaxUnits = 2e9;          // of a call: they are counted in 32 bits
constexpr int kMaxParts = 1024;            // CTAs, which is at least the shares of one tile

struct AttnParams {
  moe_attn_args_t a;
  int n_kv_heads, group;
  int tokens;       // of a tile: 128 / group
  int spread;       // CTAs c, c + 1, .., c + spread - 1 do the same share of as many heads
  int* status;
  float* part_o;    // [CTAs][2][rows of an item][D]: unnormalised sums
  float2* part_ml;  // [CTAs][2][rows of an item]: (m, sum of p)
  Cut* cuts;        // [CTAs]: by the CTA, or by_item
  bool by_item;     // one item per sequence and head, no more than CTAs: cut b * heads + h is that item's; `fits` holds
  bool fits;        // the units' sum stays in 32 bits even where sequences name the same tokens
};

// One sequence as the kernel takes it: lengths that do not fit are cut.
struct Seq {
  int q0, n, kv, base;  // first new token, their count, positions, those before the chunk
  bool bad;
};
__device__ __forceinline__ Seq load_seq(const AttnParams& p, int b) {
  const moe_attn_args_t& a = p.a;
  Seq s;
  const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1], kv = a.kv_lens[b];
  const long long room = min(1ll << 30, (long long)a.table_pages * a.page_size);
  s.q0 = max(0, min(q0, a.n_tokens));
  s.n = max(0, min(max(0, min(q1, a.n_tokens)) - s.q0, a.max_q_len));  // both in 0..n_tokens: no overflow
  s.kv = (int)max(0ll, min((long long)kv, room));
  s.bad = s.q0 != q0 || (long long)s.n != (long long)q1 - q0 || s.kv != kv;
  // the chunk's place goes by the lengths as given; what was cut is hidden
  const long long base = (long long)kv - ((long long)q1 - q0);
  s.base = (int)max(-(1ll << 30), min(base, (1ll << 30) - 1));  // base + a token's number stays in 32 bits
  return s;
}
// 128-position tiles that item i of a sequence visits (at least one, which
// writes the zeros of rows that see nothing).  kTiles: query tiles of an item.
template <int kTiles>
__device__ __forceinline__ int units_of(const AttnParams& p, const Seq& s, int i) {
  const int last = min(s.n, (i + 1) * kTiles * p.tokens) - 1;
  const int end = p.a.tree_mask ? s.kv : min(s.kv, max(0, s.base + last + 1));
  return max(1, (end + kTile - 1) / kTile);
}

// The same value in every lane, told to the compiler: MMAs take their operands
// from uniform registers, and a move there per operand took longer than the MMA.
template <typename X>
__device__ __forceinline__ X uniform(X v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// What an item costs besides its units, in units: its queries, the first scores
// and the last sums, which nothing overlaps.  In the pair form as much as two
// units: ragged chunks of 900 to 1500 tokens over 1500 to 6000 take 145 us with
// 0, 124 with 1, 119 with 2, 120 with 3.  In the split form, whose copies run
// ahead, nothing to speak of (decode batch 130 us with 0 and 131 with 1 or 2).
template <int kTiles>
constexpr int kItemCost = kTiles == 2 ? 2 : 0;

// A CTA's next piece of work.
struct Item {
  int b, h, tile, u0, u1, units;
  Seq s;
};

// The list is split into equal shares, of which `spread` neighbouring CTAs do
// the same one, each for a head of its own: what they read of a position lies
// side by side in memory and is read at about the same time.
struct Plan {
  int start, todo;     // where this CTA's share begins, and its length, in units of cost
  int share;           // of every CTA but the last
  int b, h, tile, at;  // h counts groups of `spread` heads; what of the item others have done
  Seq s;               // sequence b
};

template <int kTiles>
struct Walk {
  const AttnParams& p;
  int b, h, tile, at, todo;
  Seq s;
  int loaded;
  __device__ Walk(const AttnParams& p_, const Plan& plan)
      : p(p_), b(plan.b), h(plan.h), tile(plan.tile), at(plan.at), todo(plan.todo), s(plan.s), loaded(plan.b) {}
  __device__ bool next(Item& it) {
    if (todo <= 0) return false;
    for (;;) {
      if (loaded != b) {
        s = load_seq(p, b);
        loaded = b;
      }
      if (tile * kTiles * p.tokens < s.n) break;
      tile = 0;
      if (s.n > 0 && ++h < p.n_kv_heads / p.spread) continue;
      h = 0;
      ++b;
    }
    it.b = b, it.h = h * p.spread + (int)blockIdx.x % p.spread, it.tile = tile, it.s = s;
    it.units = units_of<kTiles>(p, s, tile);
    const int to = min(it.units + kItemCost<kTiles>, at + todo);
    todo -= to - at;
    it.u0 = max(0, at - kItemCost<kTiles>);
    it.u1 = max(0, to - kItemCost<kTiles>);
    at = 0;
    ++tile;
    return it.u1 > 0;  // a share that ends before the item's first unit leaves it to the next
  }
};

// Sum of the lanes' values up to this one's.
__device__ __forceinline__ int scan_up(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  return v;
}

// Positions that not every row of an item sees: those from `lo` on are hidden
// from some rows, those from `hi` on from all.
struct Veil {
  int lo, hi;
};
template <int kTiles>
__device__ __forceinline__ Veil veil_of(const AttnParams& p, const Seq& s, int item) {
  if (p.a.tree_mask) return {max(0, min(s.base, s.kv)), s.kv};
  const int first = item * kTiles * p.tokens, last = min(s.n, first + kTiles * p.tokens) - 1;
  const int lo = max(0, min(s.base + first + 1, s.kv));
  return {lo, max(lo, min(s.base + last + 1, s.kv))};
}

// Elements of a pair that are infinite or NaN: the top bit of each half.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair) {
  constexpr uint32_t kExponent = std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kLowest = std::is_same<T, __nv_bfloat16>::value ? 0x00800080u : 0x04000400u;
  return ((pair & kExponent) + kLowest) & 0x80008000u;  // all ones carry into the sign's place
}
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint4 v) {
  return not_finite<T>(v.x) | not_finite<T>(v.y) | not_finite<T>(v.z) | not_finite<T>(v.w);
}

// Values (128 rows of D in shared memory) whose rows from `lo` on are hidden from
// some rows of the item and from `hi` on from all: a hidden row's probability is
// 0, but 0 * inf and 0 * NaN are NaN.  Rows from `hi` on become zeros: past the
// sequence's end they hold anything.  Of the others only infinities and NaN do;
// true in the lanes that met one.  (Two plain loops: as one, with a branch, it
// was late for the products, ragged chunks 131 us instead of 121.)
template <typename T, int D>
__device__ __forceinline__ bool clean_values(uint8_t* values, int lo, int hi) {
  constexpr int kChunks = D / 8;  // of 16 bytes, of a row
  const int lane = threadIdx.x & 31, past = min(max(hi, 0), kTile);
  auto chunk = [&](int i) {
    return reinterpret_cast<uint4*>(values + (i % kChunks / 8) * (kTile * 128) + i / kChunks * 128 + i % 8 * 16);
  };
  for (int i = past * kChunks + lane; i < kTile * kChunks; i += 32) *chunk(i) = make_uint4(0u, 0u, 0u, 0u);
  bool found = false;
#pragma unroll 1
  for (int i = lo * kChunks + lane; i < past * kChunks; i += 32) {
    uint4* at = chunk(i);
    if (!not_finite<T>(*at)) continue;
    found = true;
    uint32_t* pairs = reinterpret_cast<uint32_t*>(at);
#pragma unroll 1
    for (int k = 0; k < 4; ++k) pairs[k] &= ~((not_finite<T>(pairs[k]) >> 15) * 0xffffu);
  }
  return found;
}

// Where this CTA's share begins, found by each warp for itself: lane l has the
// sequences l * per, .., whose costs (one head's units) cost(b) gives and sum
// to `lane_sum`.
template <int kTiles, bool kChecked, typename Cost>
__device__ __forceinline__ Plan make_plan(const AttnParams& p, int per, long long lane_sum, Cost cost) {
  const int lane = threadIdx.x & 31;
  const int heads = p.n_kv_heads / p.spread, shares = gridDim.x / p.spread;
  if (kChecked && !p.fits) {
    // the host's limit holds for chunks that do not overlap
    long long all = lane_sum;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) all += __shfl_xor_sync(0xffffffffu, all, m);
    if ((double)all * p.n_kv_heads > kMaxUnits) {
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, kAttnBadLength);
      lane_sum = 0;  // no work for anyone (an early return here costs the long chunk 4 %)
    }
  }
  const int sum = (int)lane_sum, upto = scan_up(sum);
  const int total = __shfl_sync(0xffffffffu, upto, 31) * heads;
  Plan plan{};
  // equal shares of whole units: fewer CTAs, and cuts, where there are few
  plan.share = (unsigned)(total + shares - 1) / (unsigned)shares;
  plan.start = min(total, plan.share * (int)(blockIdx.x / p.spread));
  plan.todo = min(total - plan.start, plan.share);
  if (plan.todo == 0) return plan;
  int at = (upto - sum) * heads, own = 0, b = lane * per;
  const bool mine = plan.start >= at && plan.start < upto * heads;
  if (mine)
    for (own = cost(b); plan.start >= at + own * heads; own = cost(++b)) at += own * heads;
  const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  plan.b = __shfl_sync(0xffffffffu, b, src);
  int rest = plan.start - __shfl_sync(0xffffffffu, at, src);
  own = __shfl_sync(0xffffffffu, own, src);
  plan.s = load_seq(p, plan.b);
  plan.h = (unsigned)rest / (unsigned)own;
  rest -= plan.h * own;
  for (int tile = lane;; tile += 32) {  // 32 items at a time
    const int u = tile * kTiles * p.tokens < plan.s.n ? units_of<kTiles>(p, plan.s, tile) + kItemCost<kTiles> : 0;
    const int to = scan_up(u);
    const unsigned past = __ballot_sync(0xffffffffu, to > rest);
    if (past) {
      const int first = __ffs(past) - 1;
      plan.tile = __shfl_sync(0xffffffffu, tile, first);
      plan.at = rest - __shfl_sync(0xffffffffu, to - u, first);
      return plan;
    }
    rest -= __shfl_sync(0xffffffffu, to, 31);
  }
}

// Whether a row has seen nothing where these are its largest score and its sum.
// A row whose scores are all NaN has no largest one either, but its sum is NaN,
// which has to show.
__device__ __forceinline__ bool nothing_seen(float2 ml) { return ml.x == -INFINITY && ml.y == 0.f; }

// The n lowest bits of a word (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }

// Waits with a limit.  The first that runs out sets the CTA's flag, after
// which no wait of the CTA waits any more: every role walks to its end (its
// addresses never depend on data that a wait guards, only on the plan).
struct Waiter {
  volatile int* gone;
  int* status;
  __device__ void operator()(uint32_t bar, uint32_t parity) const {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*gone) return;
      if (global_timer_ns() - t0 > kWaitTimeoutNs) {
        *gone = 1;
        atomicOr(status, kAttnTimeout);
        return;
      }
    }
  }
};

// Adds the infinities and NaN that clean_values has taken out of an item's
// tiles u0 .. u1 - 1 to the rows that see them: whatever its weight, an infinity
// is the sum's then.  For row r of the chain's columns, whose 16-bit output or
// fp32 part (in place `slot`) is in memory already.  Hardly ever called.
template <typename T, int D, bool kPair>
__device__ __noinline__ void add_not_finite(const AttnParams& p, int b, int h, int tile, int u0, int u1, bool cut,
                                            int slot, int chain, int r) {
  constexpr int kTiles = kPair ? 2 : 1, kColumns = kPair ? D : D / 2;
  const moe_attn_args_t& a = p.a;
  const Seq s = load_seq(p, b);
  const int token = (tile * kTiles + (kPair ? chain : 0)) * p.tokens + r / p.group;
  if (r / p.group >= p.tokens || token >= s.n) return;
  const Veil veil = veil_of<kTiles>(p, s, tile);
  const int column0 = kPair ? 0 : chain * kColumns, local = kPair ? chain * kTile + r : r;
  const long long row = s.q0 + token;
  const int head = h * p.group + r % p.group;
  T* out = static_cast<T*>(a.out) + row * a.out_token_stride + head * a.out_head_stride + column0;
  float* part = p.part_o + ((long long)slot * kTiles * kTile + local) * D + column0;
  for (int pos = max(veil.lo, u0 * kTile); pos < min(veil.hi, u1 * kTile); ++pos) {
    const int other = pos - s.base;  // the chunk's token at that position
    if (a.tree_mask ? other >= 64 || (other >= 0 && !((a.tree_mask[row] >> other) & 1)) : other > token) continue;
    const int page = a.block_table[(long long)b * a.table_stride + pos / a.page_size];
    if ((unsigned)page >= (unsigned)a.n_pages) continue;
    const T* v = static_cast<const T*>(a.v_cache) + page * a.v_page_stride + pos % a.page_size * a.v_row_stride +
                 h * D + column0;
    for (int column = 0; column < kColumns; column += 8) {
      if (!not_finite<T>(*reinterpret_cast<const uint4*>(v + column))) continue;
      for (int i = column; i < column + 8; ++i) {
        const float x = (float)v[i];
        if (fabsf(x) < INFINITY) continue;
        if (cut)
          part[i] += x;
        else
          out[i] = (T)((float)out[i] + x);
      }
    }
  }
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int D, bool kPair>
struct Layout {
  static constexpr int kThreads = kPair ? 384 : 352;
  static constexpr uint32_t kTileBytes = kTile * D * 2;          // one tile of Q, K or V
  static constexpr int kQTiles = kPair ? 2 : 1;
  static constexpr int kRows = kQTiles * kTile;                   // query rows of an item
  // barriers and the staging area (split: the exchange of both chains' statistics) before the tiles
  static constexpr uint32_t kHead = 1024 + (kPair ? kStagingBytes : 2048u);
  static constexpr int kFit = (int)((232448 - kHead) / kTileBytes) - kQTiles;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr uint32_t kSmem = kHead + (kQTiles + kStages) * kTileBytes;
};

template <typename T, int D, bool kPair>
__global__ void __launch_bounds__(Layout<D, kPair>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap q_map,
                           const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = Layout<D, kPair>;
  constexpr int kTiles = L::kQTiles, kRows = L::kRows, kStages = L::kStages, kThreads = L::kThreads;
  constexpr uint32_t kTileBytes = L::kTileBytes, kPanel = kTile * 128;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle goes by address bits up to 9
  const uint32_t sb = smem_u32(smem);
  auto full = [&](int s) { return sb + 8u * s; };
  auto empty = [&](int s) { return sb + 80u + 8u * s; };
  auto q_full = [&](int t) { return sb + 160u + 8u * t; };
  auto q_empty = [&](int t) { return sb + 176u + 8u * t; };
  // of a chain and one of its two score buffers
  auto s_full = [&](int chain, int half) { return sb + 192u + 16u * chain + 8u * half; };
  auto p_full = [&](int chain, int half) { return sb + 224u + 16u * chain + 8u * half; };
  auto o_done = [&](int chain, int half) { return sb + 256u + 16u * chain + 8u * half; };
  const uint32_t drained = sb + 288u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 296);
  int* gone = reinterpret_cast<int*>(smem + 300);
  auto raw = [&](int s) { return sb + 304u + 8u * s; };  // pair form: in place of full(s) for veiled values
  // the numbers of the last items with values that were not finite; the value
  // warp is at most half a ring of items ahead of the softmax warps
  constexpr int kItems = 8;
  static_assert(kStages / 2 + 2 < kItems);
  volatile int* left_out = reinterpret_cast<int*>(smem + 384);
  uint8_t* staging = smem + 1024;                          // [8][32 rows][128 bytes]: of the softmax warps
  float2* exchange = reinterpret_cast<float2*>(staging);   // [2][128]: both chains' (m, sum)
  const uint32_t q_at = sb + L::kHead, ring = q_at + L::kQTiles * kTileBytes;
  uint8_t* ring_smem = smem + L::kHead + L::kQTiles * kTileBytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const moe_attn_args_t& a = p.a;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
      if (kPair) mbar_init(raw(s), 1);
    }
    for (int i = 0; i < kItems; ++i) left_out[i] = -1;
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      for (int half = 0; half < 2; ++half) {
        mbar_init(s_full(t, half), 1);
        mbar_init(p_full(t, half), 4);
        mbar_init(o_done(t, half), 1);
      }
    }
    mbar_init(drained, 1);
    fence_mbar_init();
    *gone = 0;
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), 512);
  if (warp == kCopyWarp && lane == 0) {
    tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const Waiter wait{gone, p.status};
  // A tile of an item's veiled values, by a warp, before the products read them.
  auto clean = [&](int item, Veil veil, int u, int stage) {
    const bool found = clean_values<T, D>(ring_smem + stage * kTileBytes, max(0, veil.lo - u * kTile),
                                          veil.hi - u * kTile);
    fence_proxy_async_smem();
    if (__any_sync(0xffffffffu, found) && lane == 0) left_out[item % kItems] = item;
    __syncwarp();
  };
  pdl_wait();
  pdl_launch_dependents();

  // ---- the plan, from the cost of each sequence (of one key/value head); few
  // sequences: every warp makes it by itself and goes on without the others
  Plan plan;
  const bool wide = a.max_q_len > 4 * kTiles * p.tokens;  // sequences of many items: a warp each
  if (a.batch <= 32 && !wide && p.fits) {
    int sum = 0;
    if (lane < a.batch) {
      const Seq s = load_seq(p, lane);
      if (s.bad && blockIdx.x == 0) atomicOr(p.status, kAttnBadLength);
      for (int i = 0; i * kTiles * p.tokens < s.n; ++i) sum += units_of<kTiles>(p, s, i) + kItemCost<kTiles>;
    }
    plan = make_plan<kTiles, false>(p, 1, sum, [&](int) { return sum; });
  } else {
    int* cost = reinterpret_cast<int*>(ring_smem);  // the ring is not in use yet
    for (int b = wide ? warp : tid; b < a.batch; b += wide ? kThreads / 32 : kThreads) {
      const Seq s = load_seq(p, b);
      if (s.bad && blockIdx.x == 0) atomicOr(p.status, kAttnBadLength);
      int sum = 0;
      for (int i = wide ? lane : 0; i * kTiles * p.tokens < s.n; i += wide ? 32 : 1)
        sum += units_of<kTiles>(p, s, i) + kItemCost<kTiles>;
      if (wide) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      }
      if (!wide || lane == 0) cost[b] = sum;
    }
    __syncthreads();
    const int per = (a.batch + 31) / 32;
    long long sum = 0;
    for (int b = lane * per; b < min(a.batch, (lane + 1) * per); ++b) sum += cost[b];
    plan = make_plan<kTiles, true>(p, per, sum, [&](int b) { return cost[b]; });
    fence_proxy_async_smem();  // the costs' place becomes the ring
    __syncthreads();
  }
  if (p.by_item) {
    // items that are not cut say so where they begin; these have no items
    if (blockIdx.x == 0)
      for (int i = tid; i < a.batch * p.n_kv_heads; i += kThreads)
        if (load_seq(p, i / p.n_kv_heads).n == 0) p.cuts[i].parts = 0;
  } else if (tid == 0) {
    p.cuts[blockIdx.x].parts = 0;
  }

  if (warp < kMmaWarp) {
    Walk<kTiles> walk(p, plan);
    Item it{};
    // ---- softmax: chain 0 in warps 0-3, chain 1 in warps 4-7, a row per thread
    const int chain = warp >> 2, r = tid & 127;
    const int q_tile = kPair ? chain : 0;
    const uint32_t lane_at = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
    const uint32_t s_at = tmem + lane_at + chain * kTile, o_at = tmem + lane_at + 2 * kTile + chain * D;
    const float c = a.scale * 1.4426950408889634f;  // exponents in base 2
    const float rescale = kRescaleLog2 / c;
    int tiles[2] = {0, 0};  // tiles of positions of the even and the odd chain before this item
    const int row_token = r / p.group, row_head = r - row_token * p.group;
    for (int item = 0; walk.next(it); ++item) {
      const int token0 = (it.tile * kTiles + q_tile) * p.tokens;  // the tile's first, in the chunk
      const int token = token0 + row_token, head = it.h * p.group + row_head;
      const bool valid = row_token < p.tokens && token < it.s.n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      // positions below `plain` are seen, from `end` on hidden, between them
      // the tree's bits decide
      const unsigned long long bits = a.tree_mask && valid ? (unsigned long long)a.tree_mask[it.s.q0 + token] : 0ull;
      const int end = !valid ? 0 : a.tree_mask ? it.s.kv : min(it.s.kv, max(0, it.s.base + token + 1));
      const int plain = a.tree_mask ? max(0, min(it.s.base, end)) : end;
      const int warp_plain = __reduce_min_sync(0xffffffffu, plain);
      float m = -INFINITY, l = 0.f;
      int done = 0;  // tiles of this chain in this item
      // One step: 64 positions, straight through with or without masking (a
      // branch around the masking alone would hold the scores twice).
      auto softmax_step = [&](int half, int first_pos, auto masked_type) {
        constexpr bool masked = decltype(masked_type)::value;
        uint32_t s[kHalf];
        tmem_ld32(s_at + kHalf * half, s);
        tmem_ld32(s_at + kHalf * half + 32, s + 32);
        tmem_wait_ld();
        if (masked) {
          // a bit for each column: those below `plain`, and a tree's
          const int left = plain - first_pos, sh = it.s.base - first_pos;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t seen = below(left - 32 * w);
            if (a.tree_mask) {
              const int k = 32 * w - sh;
              const unsigned long long part = k >= 64 || k <= -32 ? 0ull : k >= 0 ? bits >> k : bits << -k;
              seen |= (uint32_t)part & below(end - first_pos - 32 * w);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1)) s[32 * w + i] = 0xff800000u;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kHalf; i += 2) max3(top[(i / 2) & 3], s[i], s[i + 1]);
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        float shrink = 1.f;
        if (high > m + rescale || m == -INFINITY) {
          if (m != -INFINITY) shrink = exp2_approx((m - high) * c);
          m = high;
        }
        if ((done > 0 || half > 0) && __any_sync(0xffffffffu, shrink != 1.f)) {
          // the products so far have to be in before their sums shrink: the
          // last step's, for these scores came after the ones before
          wait(o_done(chain, half ^ 1), (tiles[0] * (1 - chain) + tiles[1] * chain + done - (half ^ 1)) & 1);
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t o[16];
            tmem_ld16(o_at + 16 * i, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * shrink);
            tmem_st16(o_at + 16 * i, o);
          }
          l *= shrink;
        }
        const float off = m == -INFINITY ? 0.f : m * c;
        const uint64_t c2 = pair_of(c, c), off2 = pair_of(-off, -off);
        uint64_t sum[2] = {0ull, 0ull};  // two pairs of fp32 zeros
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t packed[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint64_t z = fma2(pair_of(s[32 * i + 2 * k], s[32 * i + 2 * k + 1]), c2, off2);
            const float x = exp2_approx(low_of(z)), y = exp2_approx(high_of(z));
            sum[k & 1] = add2(sum[k & 1], pair_of(x, y));
            packed[k] = pack<T>(x, y);
          }
          tmem_st16(s_at + kHalf * half + 16 * i, packed);
        }
        sum[0] = add2(sum[0], sum[1]);
        l += low_of(sum[0]) + high_of(sum[0]);
        tmem_wait_st();
      };
      for (int u = kPair ? it.u0 : it.u0 + chain; u < it.u1; u += kPair ? 1 : 2) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int first_pos = u * kTile + half * kHalf;
          wait(s_full(chain, half), (tiles[0] * (1 - chain) + tiles[1] * chain + done) & 1);
          tc_fence_after();
          if (warp_valid) {
            if (warp_plain < first_pos + kHalf)
              softmax_step(half, first_pos, std::true_type{});
            else
              softmax_step(half, first_pos, std::false_type{});
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(chain, half));
        }
        ++done;
      }
      // ---- the end of the item
      const int n = it.u1 - it.u0;
      // both chains' tiles in this item
      const int count0 = kPair ? n : (n + 1) / 2, count1 = kPair ? n : n / 2;
      const bool cut = n < it.units;
      const int slot = 2 * blockIdx.x + (it.u0 == 0 ? 1 : 0);
      const int local = kPair ? chain * kTile + r : r;  // row of the item
      float f0 = 1.f, f1 = 0.f;
      bool seen0 = true, seen1 = true;
      if (!kPair) {
        // each chain's warps then write half of the columns
        exchange[chain * kTile + r] = make_float2(m, l);
        named_sync(1, 256);
        const float2 even = exchange[r], odd = exchange[kTile + r];
        named_sync(1, 256);  // before it is written over
        m = fmaxf(even.x, odd.x);
        seen0 = !nothing_seen(even), seen1 = !nothing_seen(odd);
        f0 = even.x == -INFINITY ? 0.f : exp2_approx((even.x - m) * c);
        f1 = odd.x == -INFINITY ? 0.f : exp2_approx((odd.x - m) * c);
        l = even.y * f0 + odd.y * f1;
      }
      tiles[0] += count0;
      tiles[1] += count1;
      // the last step's products (which come after all the others)
      if (!kPair || chain == 0) wait(o_done(0, 1), (tiles[0] - 1) & 1);
      if (kPair ? chain == 1 : count1 > 0) wait(o_done(1, 1), (tiles[1] - 1) & 1);
      tc_fence_after();
      if (warp_valid) {
        const float norm = cut ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
        constexpr int kBlocks = kPair ? D / 32 : D / 64;  // 32-column blocks of this warp
        const int block0 = kPair ? 0 : chain * kBlocks;
        const uint32_t even_at = tmem + lane_at + 2 * kTile + (kPair ? chain * D : 0);
        // Rows are 256 bytes or more apart, so a warp's lanes would write 32
        // places at a time: by way of shared memory eight lanes write 128 bytes
        // of a row.  The split form has few rows and rather another stage.
        uint8_t* mine = staging + warp * 4096;
        auto put = [&](int chunk, uint4 v) {
          *reinterpret_cast<uint4*>(mine + lane * 128 + (chunk ^ (lane & 7)) * 16) = v;
        };
        auto flush = [&](char* to) {  // this lane's 128 bytes, nullptr: none
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = i * 4 + lane / 8;
            const auto at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), row);
            char* dst = reinterpret_cast<char*>(at);
            const uint4 v = *reinterpret_cast<const uint4*>(mine + row * 128 + ((lane & 7) ^ (row & 7)) * 16);
            if (dst) *reinterpret_cast<uint4*>(dst + (lane & 7) * 16) = v;
          }
          __syncwarp();
        };
        char* out = reinterpret_cast<char*>(static_cast<T*>(a.out) + (long long)(it.s.q0 + token) * a.out_token_stride +
                                            head * a.out_head_stride);
        char* part = reinterpret_cast<char*>(p.part_o + ((long long)slot * kRows + local) * D);
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
          uint32_t o[32];
          tmem_ld32(even_at + 32 * (block0 + i), o);
          tmem_wait_ld();
          if (!kPair && count1 > 0) {
            uint32_t o1[32];
            tmem_ld32(even_at + D + 32 * (block0 + i), o1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              o[k] = __float_as_uint((seen0 ? __uint_as_float(o[k]) * f0 : 0.f) +
                                     (seen1 ? __uint_as_float(o1[k]) * f1 : 0.f));
          }
          if (cut) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 v = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
              if (kPair)
                put(k, v);
              else if (valid)
                *reinterpret_cast<uint4*>(part + 128 * (block0 + i) + 16 * k) = v;
            }
            if (kPair) flush(valid ? part + 128 * (block0 + i) : nullptr);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 v;
              uint32_t* w = &v.x;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack<T>(__uint_as_float(o[8 * k + 2 * j]) * norm, __uint_as_float(o[8 * k + 2 * j + 1]) * norm);
              if (kPair)
                put((i & 1) * 4 + k, v);
              else if (valid)
                *reinterpret_cast<uint4*>(out + 64 * (block0 + i) + 16 * k) = v;
            }
            if (kPair && (i & 1)) flush(valid ? out + 64 * (block0 + i - 1) : nullptr);
          }
        }
        if (valid && (kPair || chain == 0)) {
          if (cut)
            p.part_ml[(long long)slot * kRows + local] = make_float2(m, l);
          else if (a.lse)
            a.lse[(long long)(it.s.q0 + token) * (p.group * p.n_kv_heads) + head] =
                l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (left_out[item % kItems] == item)
        add_not_finite<T, D, kPair>(p, it.b, it.h, it.tile, it.u0, it.u1, cut, slot, chain, r);
      if (it.u0 == 0 && tid == 0) {
        const int at = p.by_item ? it.b * p.n_kv_heads + it.h : blockIdx.x;
        if (cut) {
          // this share ends inside the tile: which share holds its last unit
          const int last = plan.start + (plan.todo - walk.todo) - n + it.units - 1;
          const int e = (unsigned)last / (unsigned)plan.share;
          p.cuts[at] = Cut{e - (int)blockIdx.x / p.spread + 1, (int)blockIdx.x, it.b, it.h, it.tile};
        } else if (p.by_item) {
          p.cuts[at].parts = 0;
        }
      }
      if (!kPair) named_sync(1, 256);  // both chains' sums are read before the next item's
    }
  } else {
    if (warp == kCopyWarp) {
      Walk<kTiles> walk(p, plan);
      Item it{};
      // ---- copies: per 128 positions one box per page and 64 columns, a lane each
      constexpr int kHalves = D / 64;
      const int box_rows = min(a.page_size, kTile), per_tile = kTile / box_rows;
      const int pages_log2 = 31 - __clz(a.page_size);
      const int box = lane / kHalves, half = lane % kHalves;
      int filled = 0;
      // The table's entries come 32 at a time, an entry per lane, and a window
      // ahead of their use: `even` and `odd` hold the windows of those numbers.
      int even = 0, odd = 0, have = 0;
      auto fetch = [&](int window) {
        const int i = window * 32 + lane;
        const bool used = (long long)i * a.page_size < it.s.kv;
        const int page = used ? a.block_table[(long long)it.b * a.table_stride + i] : -1;
        if (window & 1)
          odd = page;
        else
          even = page;
        have = window;
      };
      auto start_item = [&]() {
        fetch((it.u0 * kTile >> pages_log2) / 32);
        fetch(have + 1);
      };
      int veiled = 0;  // the item's first tile of positions that not every row sees
      auto load = [&](const CUtensorMap* map, int u) {
        const int stage = filled % kStages, round = filled / kStages;
        const int pos = u * kTile + box * box_rows, i = pos >> pages_log2, window = (u * kTile >> pages_log2) / 32;
        int page = __shfl_sync(0xffffffffu, window & 1 ? odd : even, i & 31);
        const bool mine = box < per_tile && pos < it.s.kv;
        if (mine && (unsigned)page >= (unsigned)a.n_pages) {
          atomicOr(p.status, kAttnBadPage);
          page = a.n_pages;  // outside the tensor: reads as zeros
        }
        if (round > 0) wait(empty(stage), (round - 1) & 1);
        const unsigned boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bar = kPair && map == &v_map && u >= veiled ? raw(stage) : full(stage);
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * box_rows * 128u);
        __syncwarp();
        if (mine)
          tma_load_3d(ring + stage * kTileBytes + half * kPanel + box * box_rows * 128, map, it.h * D + half * 64,
                      pos & (a.page_size - 1), page, bar);
        ++filled;
        return window;
      };
      // values come last of a position's copies: what is before their window is done with
      auto load_values = [&](int u) {
        const int window = load(&v_map, u);
        if (window == have) fetch(window + 1);
      };
      while (walk.next(it)) {
        const int n = it.u1 - it.u0;
        start_item();
        if (kPair) veiled = veil_of<kTiles>(p, it.s, it.tile).lo / kTile;
        if (kPair) {
          for (int j = 0; j < n; ++j) {
            load(&k_map, it.u0 + j);
            load_values(it.u0 + j);
          }
        } else {
          load(&k_map, it.u0);
          if (n > 1) load(&k_map, it.u0 + 1);
          for (int j = 0; j < n; ++j) {
            load_values(it.u0 + j);
            if (j + 2 < n) load(&k_map, it.u0 + j + 2);
          }
        }
      }
      // no copy is in flight when the CTA ends, also after a wait has given up
      for (int f = max(0, filled - kStages); f < filled; ++f) {
        unsigned long long waited;
        mbar_wait(full(f % kStages), (f / kStages) & 1, &waited);
      }
    } else if (warp == kQueryWarp) {
      // ---- queries, of a tile as one box of its tokens, the heads of a group
      // and 64 columns.  Past the sequence's last token it reads what follows,
      // which no row that counts sees.
      Walk<kTiles> walk(p, plan);
      Item it{};
      int round = 0;
      for (; walk.next(it); ++round) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (round > 0) wait(q_empty(t), (round - 1) & 1);
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full(t), p.tokens * p.group * D * 2);
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
              tma_load_3d(q_at + t * kTileBytes + half * kPanel, &q_map, half * 64, it.h * p.group,
                          it.s.q0 + (it.tile * kTiles + t) * p.tokens, q_full(t));
          }
          __syncwarp();
        }
      }
      // no copy is in flight when the CTA ends, also after a wait has given up
      unsigned long long waited;
      if (round > 0)
        for (int t = 0; t < kTiles; ++t) mbar_wait(q_full(t), (round - 1) & 1, &waited);
    } else if (kPair && warp == kValueWarp) {
      // ---- veiled values, ahead of the products that read them: an item's
      // tokens veil one to three tiles, for which the MMA warp would stop.
      // Their copies arrive at a barrier of their own, and this warp at the
      // stage's.
      Walk<kTiles> walk(p, plan);
      Item it{};
      int before = 0;           // tiles of keys and values of the items before this one
      uint32_t raw_parity = 0;  // a bit per stage: of its next veiled values
      for (int item = 0; walk.next(it); ++item) {
        const Veil veil = veil_of<kTiles>(p, it.s, it.tile);
        for (int u = max(it.u0, veil.lo / kTile); u < it.u1; ++u) {
          const int stage = (before + 2 * (u - it.u0) + 1) % kStages;  // keys and values in turn
          wait(raw(stage), (raw_parity >> stage) & 1);
          raw_parity ^= 1u << stage;
          clean(item, veil, u, stage);
          if (lane == 0) mbar_arrive(full(stage));
        }
        before += 2 * (it.u1 - it.u0);
      }
      // no copy is in flight when the CTA ends, also after a wait has given up
      unsigned long long waited;
      for (int s = 0; s < kStages; ++s) mbar_wait(raw(s), (~raw_parity >> s) & 1, &waited);
    } else if (warp == kMmaWarp) {
      Walk<kTiles> walk(p, plan);
      Item it{};
      // ---- products, issued by one lane
      constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
      constexpr uint32_t kDescS = mma_desc(kBf16, false, kTile, kPair ? kHalf : kTile);
      constexpr uint32_t kDescO = mma_desc(kBf16, true, kTile, D);
      int taken = 0, q_round = 0, item = 0;
      Veil veil{};
      uint32_t p_parity = 0;  // bit 2 chain + half: of the next probabilities
      auto next_stage = [&]() {
        const int stage = taken % kStages;
        wait(full(stage), (taken / kStages) & 1);
        ++taken;
        return stage;
      };
      // S of 64 of a stage's positions, into the chain's buffer of that half; in
      // the split form (half = 0) of all 128, into both
      auto scores = [&](int chain, int half, int q_tile, int stage) {
        if (elected()) {
          const uint64_t qd = smem_desc(q_at + q_tile * kTileBytes, 16, 1024);
          const uint64_t kd = smem_desc(ring + stage * kTileBytes + half * kHalf * 128, 16, 1024);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * kPanel + (k % 4) * 32) / 16;
            mma_ss(tmem + chain * kTile + half * kHalf, qd + off, kd + off, kDescS, k > 0);
          }
          mma_commit(s_full(chain, half));
          if (!kPair) mma_commit(s_full(chain, 1));
        }
      };
      auto products = [&](int chain, int half, int stage, bool add) {
        wait(p_full(chain, half), (p_parity >> (2 * chain + half)) & 1);
        p_parity ^= 1u << (2 * chain + half);
        tc_fence_after();
        if (elected()) {
          const uint64_t vd = smem_desc(ring + stage * kTileBytes + half * kHalf * 128, kPanel, 1024);
#pragma unroll
          for (int k = 0; k < kHalf / 16; ++k)
            mma_ts(tmem + 2 * kTile + chain * D, tmem + chain * kTile + half * kHalf + k * 8, vd + k * 128, kDescO,
                   add || k > 0);
          mma_commit(o_done(chain, half));
        }
      };
      auto release = [&](int stage) {
        if (elected()) mma_commit(empty(stage));
      };
      // the item's scores are all issued: its queries make room for the next
      auto release_queries = [&]() {
        if (elected()) {
          mma_commit(q_empty(0));
          if (kPair) mma_commit(q_empty(1));
        }
      };
      // the split form's few rows veil few positions: another warp for them comes
      // later than this one (chain of 6: 14.1 us, with a warp 14.7)
      auto value_stage = [&](int u) {
        const int stage = next_stage();
        if (!kPair && (u + 1) * kTile > veil.lo) clean(item, veil, u, stage);
        return stage;
      };
      while (uniform((int)walk.next(it))) {
        const int n = uniform(it.u1 - it.u0);
        veil = veil_of<kTiles>(p, it.s, it.tile);
        veil.lo = uniform(veil.lo), veil.hi = uniform(veil.hi);
        wait(q_full(0), q_round & 1);
        if (kPair) wait(q_full(1), q_round & 1);
        int ks[2], vs[2];
        // scores go two steps ahead of the products: a chain's softmax finds the
        // next scores ready while the MMAs of its last step are still to come
        if (kPair) {
          ks[0] = next_stage();
          tc_fence_after();
          for (int step = 0; step < 4; ++step) scores(step & 1, step >> 1, step & 1, ks[0]);
          release(ks[0]);
          if (n == 1) release_queries();
          for (int j = 0; j < n; ++j) {
#pragma unroll
            for (int step = 0; step < 4; ++step) {
              const int chain = step & 1, half = step >> 1;
              if (step == 0) vs[0] = value_stage(it.u0 + j);
              products(chain, half, vs[0], j > 0 || half > 0);
              if (j + 1 < n) {
                if (step == 0) ks[0] = next_stage();
                scores(chain, half, chain, ks[0]);
              }
            }
            release(vs[0]);
            if (j + 1 < n) release(ks[0]);
            if (j + 2 == n) release_queries();
          }
        } else {
          for (int i = 0; i < min(n, 2); ++i) {
            ks[0] = next_stage();
            tc_fence_after();
            scores(i, 0, 0, ks[0]);
            release(ks[0]);
          }
          if (n <= 2) release_queries();
          for (int i0 = 0; i0 < n; i0 += 2) {
#pragma unroll
            for (int step = 0; step < 4; ++step) {
              const int chain = step >> 1, half = step & 1, i = i0 + chain;
              if (i >= n) continue;
              if (half == 0) vs[chain] = value_stage(it.u0 + i);
              products(chain, half, vs[chain], i0 > 0 || half > 0);
              if (half == 0) continue;
              release(vs[chain]);
              if (i + 2 < n) {
                ks[0] = next_stage();
                scores(chain, 0, 0, ks[0]);
                release(ks[0]);
              }
              if (i + 3 == n) release_queries();
            }
          }
        }
        ++q_round;
        ++item;
      }
      if (elected()) mma_commit(drained);
      unsigned long long waited;
      mbar_wait(drained, 0, &waited);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_free(tmem, 512);
}

// Joins the tiles that shares have cut: out = sum_i O_i 2^(c (m_i - m)) / sum_i
// l_i 2^(c (m_i - m)) in the order of the shares.  Block (i, y): of cut i, 4
// rows at a time.  What it costs is the latency of its reads, so all of a
// row's statistics are read at once, by the lanes of a warp, and then its
// parts by four threads per column, whose sums are added in order.
//
// Cuts by item are few and wait for nothing but these reads, so a thread may
// have many under way (128 registers: 13.3 us for 6 tokens over 8192, with 64
// registers 14.4) as long as all blocks run at once; of the blocks by CTA two
// or more share an SM (ragged chunks: 9 us less than with 128 registers).
template <typename T, int D, int kRows, bool kByItem>
__global__ void __launch_bounds__(kJoinRows * kJoinGroups * D / 4, kByItem ? 128 / D * 2 - 1 : 256 / D)
    join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kColumns = D / 4;
  __shared__ float factor[kJoinRows][kMaxParts];
  __shared__ float4 sums[kJoinGroups - 1][kJoinRows][kColumns];
  __shared__ float2 total[kJoinRows];  // (1 / sum, log-sum)
  const moe_attn_args_t& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int column = tid % kColumns, row = tid / kColumns % kJoinRows, part = tid / (kColumns * kJoinRows);
  // the lengths are no output of the kernel before, which starts this one only
  // after it has waited for what came before itself
  Seq s;
  if (kByItem) s = load_seq(p, blockIdx.x / p.n_kv_heads);
  pdl_wait();
  pdl_launch_dependents();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.parts == 0) return;
  if (!kByItem) s = load_seq(p, cut.b);
  // rows of the item in use: of the pair's second tile from 128 on
  auto token_of = [&](int row) {
    const int in_tile = row % kTile / p.group;
    return in_tile < p.tokens ? (cut.tile * (kRows / kTile) + row / kTile) * p.tokens + in_tile : s.n;
  };
  const float c = a.scale * 1.4426950408889634f;
  auto write = [&](int row, int token, int column, float4 o, float norm, float lse) {
    const int head = cut.h * p.group + row % kTile % p.group;
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (long long)(s.q0 + token) * a.out_token_stride +
                              head * a.out_head_stride + column * 4) =
        make_uint2(pack<T>(o.x * norm, o.y * norm), pack<T>(o.z * norm, o.w * norm));
    if (a.lse && column == 0) a.lse[(long long)(s.q0 + token) * (p.group * p.n_kv_heads) + head] = lse;
  };
  auto slot = [&](int i) { return 2ll * (cut.c + i * p.spread) + (i == 0 ? 1 : 0); };
  auto factor_of = [&](float part_m, float m) { return part_m == -INFINITY ? 0.f : exp2_approx((part_m - m) * c); };
  // Few parts (tiles of long chunks, cut once or twice): a thread reads all of
  // its column's at once.
  if (cut.parts <= kFewParts) {
    constexpr int kAtOnce = kJoinRows * kJoinGroups;
    for (int r = blockIdx.y * kAtOnce + tid / kColumns; r < kRows; r += gridDim.y * kAtOnce) {
      const int token = token_of(r);
      if (token >= s.n) continue;
      float2 ml[kFewParts];
      float4 v[kFewParts];
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        if (i < cut.parts) {
          ml[i] = p.part_ml[slot(i) * kRows + r];
          v[i] = reinterpret_cast<const float4*>(p.part_o)[(slot(i) * kRows + r) * kColumns + column];
        }
      }
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) m = fmaxf(m, ml[i].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kFewParts; ++i) {
        if (nothing_seen(ml[i])) continue;
        const float f = factor_of(ml[i].x, m);
        l = fmaf(ml[i].y, f, l);
        o.x = fmaf(v[i].x, f, o.x);
        o.y = fmaf(v[i].y, f, o.y);
        o.z = fmaf(v[i].z, f, o.z);
        o.w = fmaf(v[i].w, f, o.w);
      }
      write(r, token, column, o, l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l),
            l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f);
    }
    return;
  }
  for (int r0 = blockIdx.y * kJoinRows; r0 < kRows; r0 += gridDim.y * kJoinRows) {
    if (token_of(r0) >= s.n) continue;  // nor does a later row of the four have a token
    const int token = token_of(r0 + row);
    const bool mine = token < s.n;
    // the first parts' sums are on their way while the factors are worked out
    constexpr int kAhead = 8;
    const int per = (cut.parts + kJoinGroups - 1) / kJoinGroups;
    const int first = part * per, end = min(cut.parts, first + per);
    auto sums_of = [&](int i) {
      return reinterpret_cast<const float4*>(p.part_o)[(slot(i) * kRows + r0 + row) * kColumns + column];
    };
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (mine && first + i < end) ahead[i] = sums_of(first + i);
    if (warp < kJoinRows && token_of(r0 + warp) < s.n) {
      float m = -INFINITY, l = 0.f;
      for (int i = lane; i < cut.parts; i += 32) m = fmaxf(m, p.part_ml[slot(i) * kRows + r0 + warp].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      for (int i = lane; i < cut.parts; i += 32) {
        const float2 ml = p.part_ml[slot(i) * kRows + r0 + warp];
        const float f = factor_of(ml.x, m);
        factor[warp][i] = nothing_seen(ml) ? -1.f : f;
        l += ml.y * f;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (lane == 0)
        total[warp] = make_float2(l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l),
                                  l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f);
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (mine) {
      auto add = [&](int i, float4 v) {
        const float f = factor[row][i];
        if (f < 0.f) return;
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (first + i < end) add(first + i, ahead[i]);
#pragma unroll 4
      for (int i = first + kAhead; i < end; ++i) add(i, sums_of(i));
      if (part > 0) sums[part - 1][row][column] = o;
    }
    __syncthreads();
    if (mine && part == 0) {
#pragma unroll
      for (int q = 0; q < kJoinGroups - 1; ++q) {
        const float4 v = sums[q][row][column];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      write(r0 + row, token, column, o, total[row].x, total[row].y);
    }
    __syncthreads();  // before the next rows' factors are written
  }
}

using MapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

MapEncode map_encode() {
  static const MapEncode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess)
      f = nullptr;
    return reinterpret_cast<MapEncode>(f);
  }();
  return fn;
}

struct Maps {
  CUtensorMap q, k, v;
};

using MapReplace = CUresult (*)(CUtensorMap*, void*);

MapReplace map_replace() {
  static const MapReplace fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapReplaceAddress", &f, 12000, cudaEnableDefault, &r) != cudaSuccess)
      f = nullptr;
    return reinterpret_cast<MapReplace>(f);
  }();
  return fn;
}

// What a map says apart from its address, and the map: encoding one takes some
// microseconds of the host, giving one another address a fraction of that.
struct Shape {
  int dtype, columns, d1, d2, rows, slabs;
  int64_t stride1, stride2;
  bool operator==(const Shape& o) const {
    return dtype == o.dtype && columns == o.columns && d1 == o.d1 && d2 == o.d2 && rows == o.rows &&
           slabs == o.slabs && stride1 == o.stride1 && stride2 == o.stride2;
  }
};
// A three-dimensional map of 16-bit elements, innermost contiguous, whose boxes
// are 64 columns of `rows` by `slabs`.
int encode_map(CUtensorMap* map, const Shape& s, const void* base, const char* what) {
  const MapEncode encode = map_encode();
  if (!encode) return fail(MOE_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {(cuuint64_t)s.columns, (cuuint64_t)s.d1, (cuuint64_t)s.d2};
  const cuuint64_t strides[2] = {(cuuint64_t)s.stride1 * 2, (cuuint64_t)s.stride2 * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)s.rows, (cuuint32_t)s.slabs};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r =
      encode(map, s.dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS
             ? MOE_OK
             : fail(MOE_ERR_INVALID_ARG, "no tensor map for the strides of %s (driver error %d)", what, (int)r);
}

struct KnownMap {
  Shape shape{};
  CUtensorMap map;
};

int map_for(KnownMap& known, const Shape& s, const void* base, CUtensorMap* map, const char* what) {
  if (!(known.shape == s)) {
    const int rc = encode_map(&known.map, s, base, what);
    if (rc != MOE_OK) {
      known.shape = Shape{};
      return rc;
    }
    known.shape = s;
  }
  *map = known.map;
  const MapReplace replace = map_replace();
  const CUresult r = replace ? replace(map, const_cast<void*>(base)) : CUDA_ERROR_NOT_FOUND;
  return r == CUDA_SUCCESS
             ? MOE_OK
             : fail(MOE_ERR_CUDA, "no tensor map at the address of %s (driver error %d)", what, (int)r);
}

}  // namespace
}  // namespace wse

using namespace wse;

struct moe_attn {
  int n_heads = 0, n_kv_heads = 0, head_dim = 0, n_sms = 0, dev = 0;
  int* status = nullptr;
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  Cut* cuts = nullptr;
  KnownMap q_map, k_map, v_map;
};

namespace {

void free_attn(moe_attn* h) {
  cudaFree(h->status);
  cudaFree(h->part_o);
  cudaFree(h->part_ml);
  cudaFree(h->cuts);
  delete h;
}

template <typename T, int D, bool kPair>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(paged_attention_kernel<T, D, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Layout<D, kPair>::kSmem);
}
template <typename T, int D>
cudaError_t allow_smem_both() {
  const cudaError_t e = allow_smem<T, D, true>();
  return e != cudaSuccess ? e : allow_smem<T, D, false>();
}

template <typename T, int D, bool kPair>
int launch_attn(const moe_attn* h, const AttnParams& p, const Maps& maps, moe_stream_t stream) {
  using L = Layout<D, kPair>;
  const int grid = h->n_sms / p.spread * p.spread;
  const int rc = launch_pdl(paged_attention_kernel<T, D, kPair>, dim3(grid), dim3(L::kThreads), L::kSmem, stream,
                            1, p, maps.q, maps.k, maps.v);
  if (rc != MOE_OK) return rc;
  const dim3 threads(kJoinRows * kJoinGroups * D / 4);
  // cuts by item: as many blocks as their rows have use for; else most of the
  // blocks find no cut
  const int rows = kPair ? L::kRows : std::max(1, std::min(p.a.max_q_len, p.tokens)) * p.group;
  if (p.by_item)
    return launch_pdl(join_kernel<T, D, L::kRows, true>,
                      dim3(p.a.batch * p.n_kv_heads, (rows + kJoinRows - 1) / kJoinRows), threads, 0, stream, 1, p);
  return launch_pdl(join_kernel<T, D, L::kRows, false>, dim3(grid, 16), threads, 0, stream, 1, p);
}

template <typename T, int D>
int launch_attn(const moe_attn* h, const AttnParams& p, const Maps& maps, moe_stream_t stream) {
  // one tile of rows per sequence and key/value head: the split form
  return p.a.max_q_len > p.tokens ? launch_attn<T, D, true>(h, p, maps, stream)
                                  : launch_attn<T, D, false>(h, p, maps, stream);
}

}  // namespace

extern "C" {

moe_attn_t* moe_attn_create(int n_heads, int n_kv_heads, int head_dim) {
  if (n_kv_heads >= 1 && n_heads / n_kv_heads > kTile) {
    fail(MOE_ERR_UNSUPPORTED, "%d query heads share a key/value head: at most %d can", n_heads / n_kv_heads, kTile);
    return nullptr;
  }
  if (n_kv_heads < 1 || n_heads < 1 || n_heads % n_kv_heads || n_heads > 65536) {
    fail(MOE_ERR_INVALID_ARG, "n_heads = %d must be a multiple of n_kv_heads = %d", n_heads, n_kv_heads);
    return nullptr;
  }
  if (head_dim != 64 && head_dim != 128) {
    fail(MOE_ERR_UNSUPPORTED, "head_dim = %d: must be 64 or 128", head_dim);
    return nullptr;
  }
  if (check_device() != MOE_OK) return nullptr;
  auto* h = new (std::nothrow) moe_attn;
  if (!h) {
    fail(MOE_ERR_OOM, "attention handle: out of memory");
    return nullptr;
  }
  h->n_heads = n_heads;
  h->n_kv_heads = n_kv_heads;
  h->head_dim = head_dim;
  cudaError_t e = cudaGetDevice(&h->dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->n_sms, cudaDevAttrMultiProcessorCount, h->dev);
  h->n_sms = std::min(h->n_sms, kMaxParts);
  if (e == cudaSuccess)
    e = head_dim == 64 ? allow_smem_both<__nv_bfloat16, 64>() : allow_smem_both<__nv_bfloat16, 128>();
  if (e == cudaSuccess) e = head_dim == 64 ? allow_smem_both<__half, 64>() : allow_smem_both<__half, 128>();
  const size_t rows = (size_t)h->n_sms * 2 * (2 * kTile);  // two partial tiles per CTA, of a pair's rows
  if (e == cudaSuccess) e = cudaMalloc(&h->status, sizeof(int));
  if (e == cudaSuccess) e = cudaMalloc(&h->part_o, rows * head_dim * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&h->part_ml, rows * sizeof(float2));
  if (e == cudaSuccess) e = cudaMalloc(&h->cuts, h->n_sms * sizeof(Cut));
  if (e == cudaSuccess) e = cudaMemset(h->status, 0, sizeof(int));
  if (e != cudaSuccess) {
    fail(e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA, "attention workspace: %s", cudaGetErrorString(e));
    cudaGetLastError();
    free_attn(h);
    return nullptr;
  }
  return h;
}

int moe_attn_forward(moe_attn_t* h, const moe_attn_args_t* a, moe_stream_t stream) {
  if (!h || !a) return fail(MOE_ERR_INVALID_ARG, "null handle or arguments");
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_FP16)
    return fail(MOE_ERR_INVALID_ARG, "dtype = %d: must be MOE_DTYPE_BF16 or MOE_DTYPE_FP16", a->dtype);
  if (a->batch < 0 || a->n_tokens < 0 || a->max_q_len < 0 || a->table_stride < 0 || a->table_pages < 0)
    return fail(MOE_ERR_INVALID_ARG, "batch, n_tokens, max_q_len, table_stride and table_pages must be 0 or more");
  if (!(a->scale > 0.f) || !(a->scale < INFINITY))
    return fail(MOE_ERR_INVALID_ARG, "scale must be positive and finite");
  if (a->page_size != 16 && a->page_size != 32 && a->page_size != 64 && a->page_size != 128 && a->page_size != 256)
    return fail(MOE_ERR_UNSUPPORTED, "page_size = %d: must be 16, 32, 64, 128 or 256", a->page_size);
  if (a->tree_mask && a->max_q_len > 64)
    return fail(MOE_ERR_UNSUPPORTED, "max_q_len = %d: a tree mask has 64 bits", a->max_q_len);
  if (a->batch == 0 || a->n_tokens == 0) return MOE_OK;
  if (a->n_pages < 1) return fail(MOE_ERR_INVALID_ARG, "n_pages = %d < 1", a->n_pages);
  if (!a->q || !a->k_cache || !a->v_cache || !a->out || !aligned(a->q, 16) || !aligned(a->k_cache, 16) ||
      !aligned(a->v_cache, 16) || !aligned(a->out, 16))
    return fail(MOE_ERR_INVALID_ARG, "q, out and the caches must be non-null and 16-byte aligned");
  const int table_pages = a->table_pages > 0 ? a->table_pages : a->table_stride;
  if ((!a->block_table && table_pages > 0) || !a->q_starts || !a->kv_lens || !aligned(a->block_table, 4) ||
      !aligned(a->q_starts, 4) || !aligned(a->kv_lens, 4) || !aligned(a->tree_mask, 8) || !aligned(a->lse, 4))
    return fail(MOE_ERR_INVALID_ARG, "block_table, q_starts and kv_lens must be non-null, and all aligned");
  if ((a->q_token_stride | a->q_head_stride | a->out_token_stride | a->out_head_stride | a->k_page_stride |
       a->k_row_stride | a->v_page_stride | a->v_row_stride) & 7)
    return fail(MOE_ERR_INVALID_ARG, "every stride must be a multiple of 8 elements (16 bytes)");
  if (a->n_tokens > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "n_tokens = %d is too many", a->n_tokens);
  if (a->batch > kMaxBatch) return fail(MOE_ERR_UNSUPPORTED, "batch = %d exceeds %d", a->batch, kMaxBatch);
  const int group = h->n_heads / h->n_kv_heads, columns = h->n_kv_heads * h->head_dim;
  const int tokens = kTile / group, box_rows = std::min(a->page_size, kTile);
  const double item_tokens = (a->max_q_len > tokens ? 2. : 1.) * tokens;
  const double item_cost = std::min(1073741824., (double)table_pages * a->page_size) / kTile + 1 + kItemCost<2>;
  if ((a->n_tokens / item_tokens + a->batch) * h->n_kv_heads * item_cost > kMaxUnits)
    return fail(MOE_ERR_UNSUPPORTED, "too much work for one call: split the tokens");
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev != h->dev)
    return fail(MOE_ERR_INVALID_ARG, "the handle belongs to device %d, the current device is %d", h->dev, dev);
  const bool fits = a->batch * std::ceil(a->max_q_len / item_tokens) * h->n_kv_heads * item_cost <= kMaxUnits;
  Maps maps;
  int rc = map_for(h->q_map, {a->dtype, h->head_dim, h->n_heads, a->n_tokens, group, tokens, a->q_head_stride,
                              a->q_token_stride},
                   a->q, &maps.q, "q");
  if (rc == MOE_OK)
    rc = map_for(h->k_map, {a->dtype, columns, a->page_size, a->n_pages, box_rows, 1, a->k_row_stride,
                            a->k_page_stride},
                 a->k_cache, &maps.k, "k_cache");
  if (rc == MOE_OK)
    rc = map_for(h->v_map, {a->dtype, columns, a->page_size, a->n_pages, box_rows, 1, a->v_row_stride,
                            a->v_page_stride},
                 a->v_cache, &maps.v, "v_cache");
  if (rc != MOE_OK) return rc;
  int spread = 1;
  while (spread < kMaxSpread && h->n_kv_heads % (2 * spread) == 0) spread *= 2;
  const bool one_item = a->max_q_len <= (a->max_q_len > tokens ? 2 : 1) * tokens;
  AttnParams p{*a,       h->n_kv_heads, group,      tokens,  spread,
               h->status, h->part_o,     h->part_ml, h->cuts, one_item && a->batch * h->n_kv_heads <= h->n_sms,
               fits};
  p.a.table_pages = table_pages;
  if (a->dtype == MOE_DTYPE_BF16)
    return h->head_dim == 64 ? launch_attn<__nv_bfloat16, 64>(h, p, maps, stream)
                             : launch_attn<__nv_bfloat16, 128>(h, p, maps, stream);
  return h->head_dim == 64 ? launch_attn<__half, 64>(h, p, maps, stream)
                           : launch_attn<__half, 128>(h, p, maps, stream);
}

int moe_attn_get_status(moe_attn_t* h) {
  if (!h) return fail(MOE_ERR_INVALID_ARG, "null handle");
  int st = 0, current = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&current)) != cudaSuccess || (e = cudaSetDevice(h->dev)) != cudaSuccess)
    return fail_cuda(e, "the handle's device");
  if ((e = cudaDeviceSynchronize()) == cudaSuccess &&
      (e = cudaMemcpy(&st, h->status, sizeof st, cudaMemcpyDeviceToHost)) == cudaSuccess)
    e = cudaMemset(h->status, 0, sizeof st);
  cudaSetDevice(current);
  if (e != cudaSuccess) return fail_cuda(e, "attention status");
  if (st & kAttnTimeout) return fail(MOE_ERR_DEVICE_TIMEOUT, "a bounded wait of the attention kernel ran out");
  if (st)
    return fail(MOE_ERR_INVALID_ARG, "%s%s", st & kAttnBadPage ? "a block table names a page outside the cache; " : "",
                st & kAttnBadLength ? "a length does not fit the block table or max_q_len" : "");
  return MOE_OK;
}

void moe_attn_destroy(moe_attn_t* h) {
  if (!h) return;
  int current = 0;
  cudaGetDevice(&current);
  cudaSetDevice(h->dev);
  cudaDeviceSynchronize();
  free_attn(h);
  cudaSetDevice(current);
}

}  // extern "C"
