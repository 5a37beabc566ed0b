// attention_work.cuh -- what the attention kernels share: how the work is listed,
// split over the CTAs and walked, waits with a limit, and the joining of tiles
// that shares have cut.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "host_util.cuh"
#include "tcgen05.cuh"

namespace wse {

// A tile that was cut at the end of CTA c's share: joined from the partial sums
// of CTAs c, c + spread, .., `parts` of them (0: no such tile).
struct Cut {
  int parts, c, b, h, tile;
};
constexpr double kMaxUnits = 2e9;          // of a call: they are counted in 32 bits
constexpr int kMaxParts = 1024;            // CTAs, which is at least the shares of one tile

// What an item costs besides its units, in units: its queries, the first scores
// and the last sums, which nothing overlaps.  In the 16-bit kernel's pair form as
// much as two units: ragged chunks of 900 to 1500 tokens over 1500 to 6000 take
// 145 us with 0, 124 with 1, 119 with 2, 120 with 3.  In its split form, whose
// copies run ahead, nothing to speak of (decode batch 130 us with 0 and 131 with
// 1 or 2).
template <int kTiles>
constexpr int kItemCost = kTiles == 2 ? 2 : 0;
// ... in the lists of a batch behind a prefix: 128 tokens behind 16,384 take 78.6 us
// with 2, 77.5 with 3, 76.1 with 4, 64 of them 44.9, 45.8 and 45.8; 8 behind 8,192
// 17.9 to 18.0 with each
constexpr int kSharedItemCost = 3;
// ... over codes, whose items end with the warps' joining: 32 sequences of 2,000 to
// 32,768 positions 73.5 us with 2, 73.2 with 3, 73.1 with 4 (79 with 0), a chain of
// 6 over 8,192 15.9, 15.6 and 15.8; behind a prefix 128 tokens 112, 109 and 108, 8
// tokens 20.1, 20.3 and 21.2
constexpr int kCodeItemCost = 3;

struct AttnParams {
  static constexpr bool kShared = false;
  static constexpr bool kAhead = false;  // a walk reads a sequence's lengths while it is at the one before
  template <int kTiles>
  static constexpr int kCost = kItemCost<kTiles>;
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
  __device__ __forceinline__ int sequences() const { return a.batch; }
  __device__ __forceinline__ int longest() const { return a.max_q_len; }
  __device__ __forceinline__ const int32_t* table_row(int b) const {
    return a.block_table + (long long)b * a.table_stride;
  }
};

// A batch whose sequences begin with the same `prefix` positions (whole pages,
// the first prefix_pages of the table's first row).  The work list has one more
// sequence, number 0: all tokens of the batch over the prefix, which all of them
// see; sequence b + 1 is the batch's b-th without it.  Every token then has two
// results, unnormalised sums with their (m, sum of p), which shared_join_kernel
// joins: where a share cut the tile in the parts, else in its place by token.
struct SharedParams : AttnParams {
  static constexpr bool kShared = true;
  static constexpr bool kAhead = true;
  template <int kTiles>
  static constexpr int kCost = kSharedItemCost;
  enum Lists { kBoth, kPrefixOnly, kOwnOnly };
  Lists lists;                  // those that this launch works on
  int prefix, prefix_pages;
  int prefix_items, own_items;  // items of each key/value head: of the prefix, and of a sequence
  float* whole_o;               // [prefix, own][n_tokens][heads][D]
  float2* whole_ml;             // [prefix, own][n_tokens][heads]
  // `cuts` has an entry for every item: of the prefix by head and item, then of
  // the sequences by number, head and item; 1 part: not cut
  __device__ __forceinline__ int sequences() const { return lists == kPrefixOnly ? 1 : a.batch + 1; }
  __device__ __forceinline__ int longest() const {
    return lists == kOwnOnly ? a.max_q_len : max(a.max_q_len, a.n_tokens);
  }
  __device__ __forceinline__ const int32_t* table_row(int b) const {
    return b == 0 ? a.block_table : a.block_table + (long long)(b - 1) * a.table_stride + prefix_pages;
  }
  __device__ __forceinline__ int item_number(int b, int h, int item) const {
    return b == 0 ? h * prefix_items + item
                  : n_kv_heads * prefix_items + ((b - 1) * n_kv_heads + h) * own_items + item;
  }
  // of a row's result over the prefix (b = 0) or its own positions
  __device__ __forceinline__ long long whole_row(int b, int token, int head) const {
    return ((long long)(b == 0 ? 0 : a.n_tokens) + token) * (n_kv_heads * group) + head;
  }
};

// How the items of one list were cut into tiles, and what their results say.
struct JoinSide {
  int tokens, tiles;       // of a tile, of an item
  const float* part_o;
  const float2* part_ml;
  float c;                 // a maximum times c is an exponent in base 2
};
struct JoinParams {
  SharedParams p;
  JoinSide before, own;    // of the prefix and of the sequences' own positions
};

namespace {

enum : int { kAttnBadPage = 1, kAttnBadLength = 2, kAttnTimeout = 4 };

constexpr int kTile = 128;                 // query rows of a tile, and positions
constexpr int kMaxBatch = 4096;
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

// One sequence as the kernel takes it: lengths that do not fit are cut.
struct Seq {
  int q0, n, kv, base;  // first new token, their count, positions, those before the chunk
  bool bad;
};
// What memory says of a sequence.
struct Lengths {
  int q0, q1, kv;
};
__device__ __forceinline__ Lengths lengths_of(const AttnParams& p, int b) {
  return {p.a.q_starts[b], p.a.q_starts[b + 1], p.a.kv_lens[b]};
}
__device__ __forceinline__ Lengths lengths_of(const SharedParams& p, int b) {
  if (b == 0) return {p.a.q_starts[0], p.a.q_starts[p.a.batch], 0};
  return {p.a.q_starts[b - 1], p.a.q_starts[b], p.a.kv_lens[b - 1]};
}
__device__ __forceinline__ Seq seq_of(const AttnParams& p, int, const Lengths& n) {
  const moe_attn_args_t& a = p.a;
  Seq s;
  const int q0 = n.q0, q1 = n.q1, kv = n.kv;
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
__device__ __forceinline__ Seq seq_of(const SharedParams& p, int b, const Lengths& n) {
  const moe_attn_args_t& a = p.a;
  Seq s;
  if (b == 0) {
    s.q0 = max(0, min(n.q0, a.n_tokens));
    s.n = p.lists == SharedParams::kOwnOnly ? 0 : max(0, min(n.q1, a.n_tokens) - s.q0);
    s.kv = s.base = p.prefix;
    s.bad = false;
    return s;
  }
  const int q0 = n.q0, q1 = n.q1, kv = n.kv;
  const long long room = min(1ll << 30, (long long)(a.table_pages - p.prefix_pages) * a.page_size);
  s.q0 = max(0, min(q0, a.n_tokens));
  s.n = max(0, min(max(0, min(q1, a.n_tokens)) - s.q0, a.max_q_len));
  const long long own = (long long)kv - p.prefix, base = own - ((long long)q1 - q0);
  s.kv = (int)max(0ll, min(own, room));
  // the new tokens come after the prefix
  s.bad = s.q0 != q0 || (long long)s.n != (long long)q1 - q0 || s.kv != own || base < 0;
  s.base = (int)max(-(1ll << 30), min(base, (1ll << 30) - 1));
  return s;
}
template <typename P>
__device__ __forceinline__ Seq load_seq(const P& p, int b) {
  return seq_of(p, b, lengths_of(p, b));
}
// 128-position tiles that item i of a sequence visits (at least one, which
// writes the zeros of rows that see nothing).  kTiles: query tiles of an item.
template <int kTiles, typename P>
__device__ __forceinline__ int units_of(const P& p, const Seq& s, int i) {
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

template <int kTiles, typename P>
struct Walk {
  const P& p;
  int b, h, tile, at, todo;
  Seq s;
  int loaded;
  Lengths ahead;  // of the sequence after `loaded`
  __device__ Walk(const P& p_, const Plan& plan)
      : p(p_), b(plan.b), h(plan.h), tile(plan.tile), at(plan.at), todo(plan.todo), s(plan.s), loaded(plan.b) {
    if (P::kAhead) read_ahead();
  }
  __device__ void read_ahead() {
    if (todo > 0 && loaded + 1 < p.sequences()) ahead = lengths_of(p, loaded + 1);
  }
  __device__ bool next(Item& it) {
    if (todo <= 0) return false;
    for (;;) {
      if (loaded != b) {
        if (P::kAhead) {  // b is the next one: sequences are walked one by one
          s = seq_of(p, b, ahead);
          loaded = b;
          read_ahead();
        } else {
          s = load_seq(p, b);
          loaded = b;
        }
      }
      if (tile * kTiles * p.tokens < s.n) break;
      tile = 0;
      if (s.n > 0 && ++h < p.n_kv_heads / p.spread) continue;
      h = 0;
      ++b;
    }
    it.b = b, it.h = h * p.spread + (int)blockIdx.x % p.spread, it.tile = tile, it.s = s;
    it.units = units_of<kTiles>(p, s, tile);
    const int to = min(it.units + P::template kCost<kTiles>, at + todo);
    todo -= to - at;
    it.u0 = max(0, at - P::template kCost<kTiles>);
    it.u1 = max(0, to - P::template kCost<kTiles>);
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
template <int kTiles, typename P>
__device__ __forceinline__ Veil veil_of(const P& p, const Seq& s, int item) {
  if (p.a.tree_mask) return {max(0, min(s.base, s.kv)), s.kv};
  const int first = item * kTiles * p.tokens, last = min(s.n, first + kTiles * p.tokens) - 1;
  const int lo = max(0, min(s.base + first + 1, s.kv));
  return {lo, max(lo, min(s.base + last + 1, s.kv))};
}

// Where this CTA's share begins, found by each warp for itself: lane l has the
// sequences l * per, .., whose costs (one head's units) cost(b) gives and sum
// to `lane_sum`; seq_at(b): sequence b, the same in every lane.
template <int kTiles, bool kChecked, typename P, typename Cost, typename SeqAt>
__device__ __forceinline__ Plan make_plan(const P& p, int per, long long lane_sum, Cost cost, SeqAt seq_at) {
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
  plan.s = seq_at(plan.b);
  plan.h = (unsigned)rest / (unsigned)own;
  rest -= plan.h * own;
  for (int tile = lane;; tile += 32) {  // 32 items at a time
    const int u = tile * kTiles * p.tokens < plan.s.n ? units_of<kTiles>(p, plan.s, tile) + P::template kCost<kTiles> : 0;
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

// The same for a CTA of kThreads, all of which call it; few sequences: every
// warp makes the plan by itself and goes on without the others.  `cost`: shared
// memory for a number per sequence, which bulk copies may write afterwards.
template <int kTiles, int kThreads, typename P>
__device__ __forceinline__ Plan plan_of(const P& p, int* cost) {
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const bool wide = p.longest() > 4 * kTiles * p.tokens;  // sequences of many items: a warp each
  if (p.sequences() <= 32 && !wide && p.fits) {
    int sum = 0;
    Seq s{};
    if (lane < p.sequences()) {
      s = load_seq(p, lane);
      if (s.bad && blockIdx.x == 0) atomicOr(p.status, kAttnBadLength);
      for (int i = 0; i * kTiles * p.tokens < s.n; ++i) sum += units_of<kTiles>(p, s, i) + P::template kCost<kTiles>;
    }
    return make_plan<kTiles, false>(p, 1, sum, [&](int) { return sum; }, [&](int b) {
      if (kTiles == 2) return load_seq(p, b);  // chunks: 4 us slower with the shuffles, ragged ones of 121
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, b); };
      return Seq{of(s.q0), of(s.n), of(s.kv), of(s.base), false};
    });
  }
  for (int b = wide ? warp : tid; b < p.sequences(); b += wide ? kThreads / 32 : kThreads) {
    const Seq s = load_seq(p, b);
    if (s.bad && blockIdx.x == 0) atomicOr(p.status, kAttnBadLength);
    int sum = 0;
    for (int i = wide ? lane : 0; i * kTiles * p.tokens < s.n; i += wide ? 32 : 1)
      sum += units_of<kTiles>(p, s, i) + P::template kCost<kTiles>;
    if (wide) {
#pragma unroll
      for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    }
    if (!wide || lane == 0) cost[b] = sum;
  }
  __syncthreads();
  const int per = (p.sequences() + 31) / 32;
  long long sum = 0;
  for (int b = lane * per; b < min(p.sequences(), (lane + 1) * per); ++b) sum += cost[b];
  const Plan plan = make_plan<kTiles, true>(p, per, sum, [&](int b) { return cost[b]; },
                                           [&](int b) { return load_seq(p, b); });
  fence_proxy_async_smem();  // the costs' place becomes the ring
  __syncthreads();
  return plan;
}

// Before the items: what says of the cuts' entries that nothing was cut there.
template <int kThreads>
__device__ __forceinline__ void clear_cuts(const AttnParams& p) {
  if (p.by_item) {
    // items that are not cut say so where they begin; these have no items
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < p.a.batch * p.n_kv_heads; i += kThreads)
        if (load_seq(p, i / p.n_kv_heads).n == 0) p.cuts[i].parts = 0;
  } else if (threadIdx.x == 0) {
    p.cuts[blockIdx.x].parts = 0;
  }
}
template <int kThreads>
__device__ __forceinline__ void clear_cuts(const SharedParams&) {}  // every item says it itself

// By one thread at the end of each item that this share began (u0 = 0), `todo`
// being what the walk had left past it: whether, and between which shares, it is
// cut.
template <typename P>
__device__ __forceinline__ void note_cut(const P& p, const Plan& plan, int todo, const Item& it) {
  const int n = it.u1 - it.u0;
  // which share holds its last unit
  const int last = plan.start + (plan.todo - todo) - n + it.units - 1;
  const int e = (unsigned)last / (unsigned)plan.share;
  if constexpr (P::kShared) {
    p.cuts[p.item_number(it.b, it.h, it.tile)] =
        Cut{n < it.units ? e - (int)blockIdx.x / p.spread + 1 : 1, (int)blockIdx.x, it.b, it.h, it.tile};
  } else {
    const int at = p.by_item ? it.b * p.n_kv_heads + it.h : blockIdx.x;
    if (n < it.units)
      p.cuts[at] = Cut{e - (int)blockIdx.x / p.spread + 1, (int)blockIdx.x, it.b, it.h, it.tile};
    else if (p.by_item)
      p.cuts[at].parts = 0;
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

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
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

}  // namespace
}  // namespace wse
