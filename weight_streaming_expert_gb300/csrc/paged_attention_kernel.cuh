// paged_attention_kernel.cuh -- the kernel of paged_attention.cu, which explains
// it; its instances for batches with a shared prefix are in shared_attention.cu.
#pragma once

#include <type_traits>

#include "attention_work.cuh"

namespace wse {
namespace {

constexpr int kHalf = 64;                  // positions of a softmax step
// Two softmax warpgroups, then a warp each for MMAs, copies and queries, and in
// the pair form one for veiled values.
constexpr int kMmaWarp = 8, kCopyWarp = 9, kQueryWarp = 10, kValueWarp = 11;
constexpr int kMaxStages = 10;
constexpr uint32_t kStagingBytes = 8 * 4096;  // 32 rows of 128 bytes for each softmax warp

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

// Adds the infinities and NaN that clean_values has taken out of an item's
// tiles u0 .. u1 - 1 to the rows that see them: whatever its weight, an infinity
// is the sum's then.  For row r of the chain's columns, whose 16-bit output or
// fp32 part (in place `slot`) is in memory already.  Hardly ever called.
template <typename T, int D, bool kPair, typename P>
__device__ __noinline__ void add_not_finite(const P& p, int b, int h, int tile, int u0, int u1, bool cut,
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
  if constexpr (P::kShared) {
    if (!cut) part = p.whole_o + p.whole_row(b, (int)row, head) * D + column0;
  }
  for (int pos = max(veil.lo, u0 * kTile); pos < min(veil.hi, u1 * kTile); ++pos) {
    const int other = pos - s.base;  // the chunk's token at that position
    if (a.tree_mask ? other >= 64 || (other >= 0 && !((a.tree_mask[row] >> other) & 1)) : other > token) continue;
    const int page = p.table_row(b)[pos / a.page_size];
    if ((unsigned)page >= (unsigned)a.n_pages) continue;
    const T* v = static_cast<const T*>(a.v_cache) + page * a.v_page_stride + pos % a.page_size * a.v_row_stride +
                 h * D + column0;
    for (int column = 0; column < kColumns; column += 8) {
      if (!not_finite<T>(*reinterpret_cast<const uint4*>(v + column))) continue;
      for (int i = column; i < column + 8; ++i) {
        const float x = (float)v[i];
        if (fabsf(x) < INFINITY) continue;
        if (P::kShared || cut)
          part[i] += x;
        else
          out[i] = (T)((float)out[i] + x);
      }
    }
  }
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

// P: AttnParams, or SharedParams, whose items all leave unnormalised sums.
template <typename T, int D, bool kPair, typename P>
__global__ void __launch_bounds__(Layout<D, kPair>::kThreads, 1)
    paged_attention_kernel(const __grid_constant__ P p, const __grid_constant__ CUtensorMap q_map,
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

  // the plan, from the cost of each sequence (of one key/value head)
  const Plan plan = plan_of<kTiles, kThreads>(p, reinterpret_cast<int*>(ring_smem));  // the ring is not in use yet
  clear_cuts<kThreads>(p);

  if (warp < kMmaWarp) {
    Walk<kTiles, P> walk(p, plan);
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
        const bool raw = P::kShared || cut;  // unnormalised sums
        const float norm = raw ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
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
        float* sums = p.part_o + ((long long)slot * kRows + local) * D;
        float2* ml = p.part_ml + (long long)slot * kRows + local;
        if constexpr (P::kShared) {
          if (!cut) {
            const long long row = p.whole_row(it.b, it.s.q0 + token, head);
            sums = p.whole_o + row * D;
            ml = p.whole_ml + row;
          }
        }
        char* part = reinterpret_cast<char*>(sums);
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
          if (raw) {
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
          if (raw)
            *ml = make_float2(m, l);
          else if (a.lse)
            a.lse[(long long)(it.s.q0 + token) * (p.group * p.n_kv_heads) + head] =
                l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (left_out[item % kItems] == item)
        add_not_finite<T, D, kPair>(p, it.b, it.h, it.tile, it.u0, it.u1, cut, slot, chain, r);
      if (it.u0 == 0 && tid == 0) note_cut(p, plan, walk.todo, it);
      if (!kPair) named_sync(1, 256);  // both chains' sums are read before the next item's
    }
  } else {
    if (warp == kCopyWarp) {
      Walk<kTiles, P> walk(p, plan);
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
        const int page = used ? p.table_row(it.b)[i] : -1;
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
      Walk<kTiles, P> walk(p, plan);
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
      Walk<kTiles, P> walk(p, plan);
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
      Walk<kTiles, P> walk(p, plan);
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

}  // namespace
}  // namespace wse
