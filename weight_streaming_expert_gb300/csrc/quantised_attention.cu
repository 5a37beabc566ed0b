// quantised_attention.cu -- attention of few rows over the quantised cache
// (include/attention.h): decoded tokens, verified chains and trees, and all
// tokens of a batch over a shared prefix.
//
// With code k_jd 2^(e_j) for key j and v_jd 2^(f_j) for its value, everything in
// powers of two (c = scale log2 e):
//   w_j = c 2^(e_j) q.k_j + f_j,   M = max_j w_j,   p_j = 2^(w_j - M),
//   out = sum_j p_j v_j / sum_j p_j 2^(-f_j).
// The values' scales thus go into the probabilities, and codes into the products
// as they are.  Any M gives the same quotient; M follows the maximum up when it
// has grown by more than 8, so a p_j is at most 2^8 and the largest about 1:
// what fp16 rounds away of the others is 2^-11 of each, or 2^-25 of the largest.
//
// Reading the cache is the bound of few rows, at 22 bytes a clock and SM, so a code may cost
// few instructions and little shared memory traffic: a warp takes 16 positions
// from where the copies put them straight into the registers that the warp-wide
// MMA wants (m16n8k16, fp16), converted two at a time, and never writes them back.
// (As 16-bit tiles in shared memory for tcgen05 each code would cost 7 bytes of
// the 128 that shared memory moves in a clock: 150 of them.)
//   S^T = K Q^T   A: 16 positions by 16 columns, a lane's 16 bytes of a row being
//                 the same columns of the queries, which it holds as B;
//   O^T = V^T P^T A: 16 columns by 16 positions, bytes of two rows interleaved by
//                 byte permutes; B: the probabilities, transposed in 8 x 8 blocks.
// Which position is a fragment's row g is free, and chosen so that eight lanes
// read eight different 16-byte columns of the swizzled tile (position_of).
// Q enters as fp16 with a power of two for each row: bf16's eight bits fit.
//
// A tile is 8, 16, 32 or 64 rows (whole tokens with the heads that share a
// key/value head).  Up to 16 rows eight warps share out the 128 positions of a
// unit; of 32 (64) rows each group of four (two) warps takes 16 and converts the
// unit's codes for itself, as O of more rows does not fit a warp's registers.
// Each warp has its own M, sums and O, which are joined at an item's end through
// shared memory, in the order of the warps.
//
// One GB300 (copy 6693 GB/s), 32 single tokens of 32/4 heads of 128 over 2,000 to
// 32,768 positions: 73 us, 5.7 TB/s, of which 10 us are the call's start and end
// (a tile of 8 rows; 16 rows 91 us, 32 rows 131, 64 rows 175: the conversions'
// instructions and their latency, where 16-bit caches take 124 to 137 at any of
// these rows).  6 tokens over 8,192: 15.5 us.
#include <algorithm>

#include "attention_handle.cuh"
#include "e4m3.cuh"

namespace wse {
namespace {

struct CodeParams : AttnParams {
  static constexpr bool kAhead = true;
  template <int kTiles>
  static constexpr int kCost = kCodeItemCost;
};
static_assert(kCodeItemCost <= kSharedItemCost, "the host's limit of a batch behind a prefix counts the latter");
struct SharedCodeParams : SharedParams {
  static constexpr bool kAhead = true;
  template <int kTiles>
  static constexpr int kCost = kCodeItemCost;
};

constexpr int kWarps = 8, kCopyWarps = 4, kCodeThreads = (kWarps + kCopyWarps) * 32;

// Registers of a thread: the copying warps give most of theirs to the others,
// which hold two blocks of positions at a time (16 rows: 110 us with one and 200
// bytes spilled, 89 with two when that was built, 91 now).  The shares add up to what the block is launched
// with, which launch() makes sure of.
constexpr int kLaunchRegisters = 168, kWorkRegisters = 224, kCopyRegisters = 56;
static_assert(kWarps * kWorkRegisters + kCopyWarps * kCopyRegisters == (kWarps + kCopyWarps) * kLaunchRegisters);

template <int D>
struct CodeLayout {
  static constexpr uint32_t kCodeTile = kTile * D;            // codes of keys or values of a unit
  static constexpr uint32_t kStage = 2 * kCodeTile;
  static constexpr uint32_t kScales = 2 * kTile;              // scale bytes of a unit
  static constexpr uint32_t kJoin = kWarps * 8 * (D + 4) * 4;  // [warp][8 rows][D + 4] fp32
  static constexpr uint32_t kMarks = kMaxCodeRows * D / 8;     // a bit for each output that a NaN makes one
  static constexpr uint32_t kStats = kWarps * 16 * 8;          // [warp][16 rows] (M, sum)
  static constexpr uint32_t kHead = 1024;                      // barriers
  static constexpr int kFit = (int)((232448 - kHead - kJoin - kMarks - kStats) / (kStage + kScales));
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  // the ring begins on a multiple of 1024 bytes, as the swizzle wants
  static constexpr uint32_t kRing = kHead;
  static constexpr uint32_t kScaleAt = kRing + kStages * kStage;
  static constexpr uint32_t kJoinAt = kScaleAt + kStages * kScales;
  static constexpr uint32_t kMarksAt = kJoinAt + kJoin;
  static constexpr uint32_t kStatsAt = kMarksAt + kMarks;
  static constexpr uint32_t kSmem = kStatsAt + kStats;
};

// The position, of eight, that is row (or pair of columns) g of a fragment: the
// lanes that read at the same time then read different banks.
template <int D>
__device__ __forceinline__ int position_of(int g) {
  if (D == 128) return (g & 1) * 4 + (g >> 1);
  return (g & 4) + ((g & 1) ? 3 - (g >> 1 & 1) : (g >> 1 & 1));
}
// Where 16-byte column c of row r of a tile lies, as the copies write it: with the
// 128-byte swizzle (128-byte rows) or the 64-byte one (64-byte rows).
template <int D>
__device__ __forceinline__ uint32_t place_of(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4);
}

// 16 bytes to shared memory, both sides aligned to them, without waiting; zeros
// without a look at `src` where it is not there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
// Arrives on `bar` once this thread's copies so far are in.
__device__ __forceinline__ void arrive_with_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// An 8 x 8 block of 16-bit elements, a row's two in each lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// D += A (16 x 16) B (16 x 8); unlike mma_f16 free to move among other work.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes that are NaN: the top bit of each such byte.
__device__ __forceinline__ uint32_t nan_codes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// What a row of an item sees.
template <typename P>
__device__ __forceinline__ bool row_sees(const P& p, const Item& it, int row, int pos) {
  const int token = it.tile * p.tokens + row / p.group, other = pos - it.s.base;
  if (row / p.group >= p.tokens || token >= it.s.n || pos >= it.s.kv) return false;
  if (!p.a.tree_mask) return other <= token;
  return other < 0 || (other < 64 && ((unsigned long long)p.a.tree_mask[it.s.q0 + token] >> other & 1));
}

// Notes the columns from `column` on whose codes at `pos` are NaN (a bit of
// `bad` for each byte) for those of the `rows` rows from `row0` that see them.
template <typename P>
__device__ __noinline__ void note_nan(const P& p, Item it, uint32_t* marks, volatile int* marked, uint32_t bad,
                                      int row0, int rows, int pos, int column, int D) {
  for (int row = row0; row < row0 + rows; ++row) {
    if (!row_sees(p, it, row, pos)) continue;
    for (int k = 0; k < 4; ++k) {
      const int bit = row * D + column + k;
      if (bad >> (8 * k + 7) & 1) atomicOr(marks + bit / 32, 1u << (bit & 31));
    }
    *marked = 1;
  }
}

// kN: 8-row blocks of a warp; kG: groups of warps with rows of their own.  c:
// scale * log2 e.
template <int D, int kN, int kG, typename P>
__global__ void __launch_bounds__(kCodeThreads, 1)
    quantised_attention_kernel(const __grid_constant__ P p, const __grid_constant__ moe_cache_scales_t scales,
                               const float c, const __grid_constant__ CUtensorMap k_map,
                               const __grid_constant__ CUtensorMap v_map) {
  using L = CodeLayout<D>;
  constexpr int kStages = L::kStages;
  constexpr int kTogether = kWarps / kG;          // warps that share out the positions
  constexpr int kB = 2;                           // blocks of 16 positions of a warp's step
  constexpr int kPiece = 16 * kB, kPieces = kTile / kPiece;
  constexpr int kSteps = D / 16;                  // MMAs of a score, and 16-column blocks of an output
  constexpr int kChunks = D / 64;                 // 16-byte columns of a key row in a lane
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  auto full = [&](int s) { return sb + 8u * s; };
  auto empty = [&](int s) { return sb + 64u + 8u * s; };
  int* gone = reinterpret_cast<int*>(smem + 128);
  volatile int* marked = reinterpret_cast<int*>(smem + 132);  // an item's values hold NaN that some rows see
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const moe_attn_args_t& a = p.a;
  uint32_t* marks = reinterpret_cast<uint32_t*>(smem + L::kMarksAt);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), kCopyWarps * 5);  // of each its codes, and four lanes' scales
      mbar_init(empty(s), kWarps);
    }
    fence_mbar_init();
    *gone = 0;
    *marked = 0;
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
  }
  for (int i = tid; i < (int)L::kMarks / 4; i += kCodeThreads) marks[i] = 0u;
  __syncthreads();
  const Waiter wait{gone, p.status};
  pdl_wait();
  pdl_launch_dependents();
  const Plan plan = plan_of<1, kCodeThreads>(p, reinterpret_cast<int*>(smem + L::kRing));
  clear_cuts<kCodeThreads>(p);
  Walk<1, P> walk(p, plan);
  Item it{};

  if (warp >= kWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegisters));
    // ---- copies, by four warps: keys and values, and the first and last pages of
    // a unit.  The codes with TMA, a lane per page: the lanes' copies are issued one
    // after the other, 90 clocks each, so one warp alone would need 1500 for a unit's
    // 16 boxes of 16 rows, as long as memory does (pages of 16: 104 us, with four 79).  The
    // scales 16 bytes a lane.
    const int values = (warp - kWarps) >> 1, half = (warp - kWarps) & 1;
    const int box_rows = min(a.page_size, kTile), per_unit = kTile / box_rows, page_log2 = 31 - __clz(a.page_size);
    const bool codes = lane < 4;
    const int place = 4 * half + (lane & 3), step = codes ? box_rows : 16;
    const CUtensorMap* const map = values ? &v_map : &k_map;
    const char* const scale = static_cast<const char*>(values ? scales.v_scale : scales.k_scale);
    const long long scale_page = values ? scales.v_page_stride : scales.k_page_stride;
    const long long scale_head = values ? scales.v_head_stride : scales.k_head_stride;
    int filled = 0;
    while (walk.next(it)) {
      // The table's entries come 32 at a time, an entry per lane, and a window
      // ahead of their use: `even` and `odd` hold the windows of those numbers.
      const int32_t* row = p.table_row(it.b);
      int even = 0, odd = 0, have = 0;
      auto fetch = [&](int window) {
        const int i = window * 32 + lane;
        const int page = (long long)i * a.page_size < it.s.kv ? row[i] : -1;
        if (window & 1)
          odd = page;
        else
          even = page;
        have = window;
      };
      fetch((it.u0 * kTile >> page_log2) / 32);
      fetch(have + 1);
      for (int u = it.u0; u < it.u1; ++u) {
        const int pos = u * kTile + place * step, window = (u * kTile >> page_log2) / 32;
        const int page = __shfl_sync(0xffffffffu, window & 1 ? odd : even, (pos >> page_log2) & 31);
        const bool mine = lane < 8 && pos < it.s.kv && (!codes || place < per_unit);
        const bool there = (unsigned)page < (unsigned)a.n_pages;
        if (mine && !there) atomicOr(p.status, kAttnBadPage);
        const int stage = filled % kStages, round = filled / kStages;
        if (round > 0) wait(empty(stage), (round - 1) & 1);
        const unsigned boxes = __popc(__ballot_sync(0xffffffffu, mine && codes));
        if (lane == 0) mbar_arrive_expect_tx(full(stage), boxes * D * box_rows);
        __syncwarp();
        // a page that is not there: codes of zero with the least scale, so that they
        // weigh as zeros do and do not push M up with a scale that lay there before
        if (mine && !codes)
          copy16(sb + L::kScaleAt + stage * L::kScales + values * kTile + place * 16,
                 scale + (there ? page * scale_page + it.h * scale_head + (pos & (a.page_size - 1)) : 0), there);
        if (lane >= 4 && lane < 8) arrive_with_copies(full(stage));
        if (mine && codes)  // a page that is not there lies outside the tensor and reads as zeros
          tma_load_3d(sb + L::kRing + stage * L::kStage + values * L::kCodeTile + place * box_rows * D, map, it.h * D,
                      pos & (a.page_size - 1), there ? page : a.n_pages, full(stage));
        ++filled;
        if (((u + 1) * kTile >> page_log2) / 32 == have) fetch(have + 1);
      }
    }
    // no copy is in flight when the CTA ends, also after a wait has given up
    for (int f = max(0, filled - kStages); f < filled; ++f) {
      unsigned long long waited;
      mbar_wait(full(f % kStages), (f / kStages) & 1, &waited);
    }
    return;
  }

  // ---- scores, probabilities and sums
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWorkRegisters));
  const int g = lane >> 2, t = lane & 3;
  const int rows_at = warp / kTogether * (8 * kN), part = warp % kTogether;  // this warp's first row
  float* join = reinterpret_cast<float*>(smem + L::kJoinAt);
  float2* stats = reinterpret_cast<float2*>(smem + L::kStatsAt);
  int taken = 0;
  // this lane's columns of the queries of rows 8 i + g, as B
  uint32_t q[kN][kSteps][2];
  auto load_queries = [&] {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = rows_at + 8 * i + g, in_tile = r / p.group, token = it.tile * p.tokens + in_tile;
      const bool valid = in_tile < p.tokens && token < it.s.n;
      const uint16_t* from = static_cast<const uint16_t*>(a.q) + (long long)(it.s.q0 + token) * a.q_token_stride +
                             (long long)(it.h * p.group + r - in_tile * p.group) * a.q_head_stride + 16 * t;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        uint4 v[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (valid) {
          v[0] = *reinterpret_cast<const uint4*>(from + 64 * k);
          v[1] = *reinterpret_cast<const uint4*>(from + 64 * k + 8);
        }
        q[i][4 * k][0] = v[0].x, q[i][4 * k][1] = v[0].y, q[i][4 * k + 1][0] = v[0].z, q[i][4 * k + 1][1] = v[0].w;
        q[i][4 * k + 2][0] = v[1].x, q[i][4 * k + 2][1] = v[1].y, q[i][4 * k + 3][0] = v[1].z, q[i][4 * k + 3][1] = v[1].w;
      }
    }
  };
  bool more = walk.next(it);
  if (more) load_queries();
  while (more) {
    const Veil veil = veil_of<1>(p, it.s, it.tile);
    float factor[kN][2];  // what their row's power of two leaves to the scores of rows 8 i + 2 t and + 1
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      int e = 0;
      if (a.dtype == MOE_DTYPE_BF16) {
        float largest = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            largest = fmaxf(largest, fmaxf(finite_size(bf16lo(q[i][s][k])), finite_size(bf16hi(q[i][s][k]))));
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
        largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
        // the largest in [2^13, 2^14): no power of two below 2^-24, fp16's last, unless 2^-38 of it
        if (largest > 0.f) e = max((int)(__float_as_uint(largest) >> 23) - 127 - 13, -100);
        const float down = power_of_two(-e);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int k = 0; k < 2; ++k) q[i][s][k] = pack<__half>(bf16lo(q[i][s][k]) * down, bf16hi(q[i][s][k]) * down);
      }
      const float up = c * power_of_two(e);  // of row 8 i + g, in lanes 4 g ..
      factor[i][0] = __shfl_sync(0xffffffffu, up, 8 * t);
      factor[i][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
    }
    float M[kN][2], l[kN][2], o[kN][kSteps][4];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) M[i][k] = -INFINITY, l[i][k] = 0.f;
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][j][k] = 0.f;
    }

    for (int u = it.u0; u < it.u1; ++u) {
      const int stage = taken % kStages;
      wait(full(stage), (taken / kStages) & 1);
      ++taken;
      const uint8_t* keys = smem + L::kRing + stage * L::kStage;
      const uint8_t* values = keys + L::kCodeTile;
      const uint8_t* scale_at = smem + L::kScaleAt + stage * L::kScales;
      // this warp's steps of the unit; with more warps than steps units go to halves
      // of the warps in turn
      int piece = part;
      if (kTogether > kPieces) piece = part / kPieces == ((u - it.u0) & 1) ? part % kPieces : kPieces;
#pragma unroll 1
      for (; piece < kPieces; piece += kTogether) {
        const int first = u * kTile + piece * kPiece;  // position
        if (first >= veil.hi) break;                    // none of these rows sees more
        // ---- scores of positions at(h) and at(h) + 8
        auto at = [&](int h) { return piece * kPiece + 16 * h + position_of<D>(g); };
        float s[kB][kN][4];
#pragma unroll
        for (int h = 0; h < kB; ++h) {
#pragma unroll
          for (int i = 0; i < kN; ++i) s[h][i][0] = s[h][i][1] = s[h][i][2] = s[h][i][3] = 0.f;
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint4 low = *reinterpret_cast<const uint4*>(keys + place_of<D>(at(h), t + 4 * k));
            const uint4 high = *reinterpret_cast<const uint4*>(keys + place_of<D>(at(h) + 8, t + 4 * k));
            const uint32_t lw[4] = {low.x, low.y, low.z, low.w}, hw[4] = {high.x, high.y, high.z, high.w};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2(lw[w], a0, a2);
              e4m3x4_to_f16x2(hw[w], a1, a3);
#pragma unroll
              for (int i = 0; i < kN; ++i) mma(s[h][i], a0, a1, a2, a3, q[i][4 * k + w][0], q[i][4 * k + w][1]);
            }
          }
        }
        const bool veiled = first + kPiece > veil.lo;
        // the four positions that are this lane's columns of the probabilities, and of
        // their values D / 8 bytes at its g
        auto row_of = [&](int h, int r) {
          return piece * kPiece + 16 * h + position_of<D>(2 * t + (r & 1)) + 8 * (r >> 1);
        };
        constexpr int kWords = D / 32;
        uint32_t v[kB][4][kWords];
#pragma unroll
        for (int h = 0; h < kB; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (D == 128) {
              const uint4 x =
                  *reinterpret_cast<const uint4*>(values + place_of<D>(row_of(h, r), (g & 1) * 4 + (g >> 1)));
              v[h][r][0] = x.x, v[h][r][1] = x.y, v[h][r][kWords - 2] = x.z, v[h][r][kWords - 1] = x.w;
            } else {
              const uint2 x =
                  *reinterpret_cast<const uint2*>(values + place_of<D>(row_of(h, r), g >> 1) + (g & 1) * 8);
              v[h][r][0] = x.x, v[h][r][1] = x.y;
            }
          }
        float undo[kB][2];
        float over = -INFINITY;  // by how much the largest exceeds its row's M
#pragma unroll
        for (int h = 0; h < kB; ++h) {
          // the exponents of the two positions
          const float ke[2] = {power_of_two(exponent_of(scale_at[at(h)])), power_of_two(exponent_of(scale_at[at(h) + 8]))};
          const int f0 = exponent_of(scale_at[kTile + at(h)]), f1 = exponent_of(scale_at[kTile + at(h) + 8]);
          const float fe[2] = {(float)f0, (float)f1};
          undo[h][0] = power_of_two(-f0), undo[h][1] = power_of_two(-f1);
#pragma unroll
          for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[h][i][k] = fmaf(s[h][i][k] * factor[i][k & 1], ke[k >> 1], fe[k >> 1]);
        }
        if (veiled) {
          // a hidden position's probability is 0, but 0 * NaN is NaN: past the last
          // position that any row sees values may be anything and become 0, before it
          // NaN do and are noted for the rows that see them
#pragma unroll
          for (int h = 0; h < kB; ++h) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int pos = u * kTile + at(h) + 8 * (k >> 1);
                if (!row_sees(p, it, rows_at + 8 * i + 2 * t + (k & 1), pos)) s[h][i][k] = -INFINITY;
              }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int pos = u * kTile + row_of(h, r);
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
                if (pos >= veil.hi) v[h][r][w] = 0u;
                const uint32_t bad = nan_codes(v[h][r][w]);
                if (!bad) continue;
                v[h][r][w] &= ~((bad >> 7) * 0xffu);
                note_nan(p, it, marks, marked, bad, rows_at, 8 * kN, pos,
                         (D == 128 ? 16 * ((g & 1) * 4 + (g >> 1)) : 8 * g) + 4 * w, D);
              }
            }
          }
        }
#pragma unroll
        for (int h = 0; h < kB; ++h)
#pragma unroll
          for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) over = fmaxf(over, fmaxf(s[h][i][k], s[h][i][k + 2]) - M[i][k]);
        if (__any_sync(0xffffffffu, over > kRescaleLog2)) {
#pragma unroll
          for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float top = M[i][k];
#pragma unroll
              for (int h = 0; h < kB; ++h) top = fmaxf(top, fmaxf(s[h][i][k], s[h][i][k + 2]));
#pragma unroll
              for (int m = 4; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
              const float shrink = M[i][k] == -INFINITY ? 1.f : exp2_approx(M[i][k] - top);  // or nothing to shrink yet
              M[i][k] = top;
              l[i][k] *= shrink;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                o[i][j][k] *= shrink;
                o[i][j][k + 2] *= shrink;
              }
            }
        }
        uint32_t b[kB][kN][2];
#pragma unroll
        for (int h = 0; h < kB; ++h)
#pragma unroll
          for (int i = 0; i < kN; ++i) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[k] = exp2_approx(s[h][i][k] - (M[i][k & 1] == -INFINITY ? 0.f : M[i][k & 1]));
              l[i][k & 1] = fmaf(x[k], undo[h][k >> 1], l[i][k & 1]);
            }
            b[h][i][0] = transposed(pack<__half>(x[0], x[1]));
            b[h][i][1] = transposed(pack<__half>(x[2], x[3]));
          }
#pragma unroll
        for (int h = 0; h < kB; ++h)
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
#pragma unroll
            for (int pair = 0; pair < 2; ++pair) {  // bytes 2 pair and 2 pair + 1 of the word: columns' block 2 w + pair
              const uint32_t x = __byte_perm(v[h][0][w], v[h][1][w], pair == 0 ? 0x5140 : 0x7362);
              const uint32_t y = __byte_perm(v[h][2][w], v[h][3][w], pair == 0 ? 0x5140 : 0x7362);
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x2(x, a0, a1);
              e4m3x4_to_f16x2(y, a2, a3);
#pragma unroll
              for (int i = 0; i < kN; ++i) mma(o[i][2 * w + pair], a0, a1, a2, a3, b[h][i][0], b[h][i][1]);
            }
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(stage));
    }

    // ---- the end of the item: the warps that share its rows join their sums,
    // while the next item's queries are on their way
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) l[i][k] += __shfl_xor_sync(0xffffffffu, l[i][k], m);
        if (g == 0) stats[warp * (8 * kN) + 8 * i + 2 * t + k] = make_float2(M[i][k], l[i][k]);
      }
    const Item done = it;
    const int todo = walk.todo;
    bool has_marks = false;
    const bool cut = done.u1 - done.u0 < done.units, raw = P::kShared || cut;
    const int slot = 2 * blockIdx.x + (done.u0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* to = join + (warp * 8 + 2 * t + k) * (D + 4) + (D == 128 ? 16 * ((g & 1) * 4 + (g >> 1)) : 8 * g);
#pragma unroll
        for (int j = 0; j < kSteps; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(o[i][j][k], o[i][j][k + 2], o[i][j + 1][k], o[i][j + 1][k + 2]);
      }
      if (kN == 1) {  // of 16 rows their registers would be too many
        more = walk.next(it);
        if (more) load_queries();
      }
      named_sync(1, kWarps * 32);
      has_marks = *marked != 0;
      // a thread for four columns of a row of each group
#pragma unroll 1
      for (int unit = tid; unit < kG * 8 * D / 4; unit += kWarps * 32) {
        const int column = unit % (D / 4) * 4, in_block = unit / (D / 4) % 8, group = unit / (D / 4) / 8;
        const int r = group * (8 * kN) + 8 * i + in_block, in_tile = r / p.group;
        const int token = done.tile * p.tokens + in_tile;
        if (in_tile >= p.tokens || token >= done.s.n) continue;
        const int row = group * kTogether * (8 * kN) + 8 * i + in_block;  // of the first of its warps
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kTogether; ++w) m = fmaxf(m, stats[row + w * (8 * kN)].x);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kTogether; ++w) {
          const float2 ml = stats[row + w * (8 * kN)];
          const float4 v = *reinterpret_cast<const float4*>(join + ((group * kTogether + w) * 8 + in_block) * (D + 4) + column);
          if (nothing_seen(ml)) continue;
          const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
          sum = fmaf(ml.y, f, sum);
          x.x = fmaf(v.x, f, x.x);
          x.y = fmaf(v.y, f, x.y);
          x.z = fmaf(v.z, f, x.z);
          x.w = fmaf(v.w, f, x.w);
        }
        if (has_marks) {
          const uint32_t bits = marks[(r * D + column) / 32] >> (column & 31);
          const float nan = __uint_as_float(0x7fffffffu);
          if (bits & 1) x.x = nan;
          if (bits & 2) x.y = nan;
          if (bits & 4) x.z = nan;
          if (bits & 8) x.w = nan;
        }
        const int head = done.h * p.group + r - in_tile * p.group;
        const long long t_row = done.s.q0 + token;
        if (raw) {
          float* to = p.part_o + ((long long)slot * kTile + r) * D;
          float2* to_ml = p.part_ml + (long long)slot * kTile + r;
          if constexpr (P::kShared) {
            if (!cut) {
              const long long whole = p.whole_row(done.b, (int)t_row, head);
              to = p.whole_o + whole * D;
              to_ml = p.whole_ml + whole;
            }
          }
          *reinterpret_cast<float4*>(to + column) = x;
          if (column == 0) *to_ml = make_float2(m, sum);
        } else {
          const float norm = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
          uint2 y;
          if (a.dtype == MOE_DTYPE_BF16)
            y = make_uint2(pack<__nv_bfloat16>(x.x * norm, x.y * norm), pack<__nv_bfloat16>(x.z * norm, x.w * norm));
          else
            y = make_uint2(pack<__half>(x.x * norm, x.y * norm), pack<__half>(x.z * norm, x.w * norm));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + t_row * a.out_token_stride + head * a.out_head_stride +
                                    column) = y;
          if (a.lse && column == 0)
            a.lse[t_row * (p.group * p.n_kv_heads) + head] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
        }
      }
      named_sync(1, kWarps * 32);  // before the next block's sums, or the next item's
    }
    if (done.u0 == 0 && tid == 0) note_cut(p, plan, todo, done);
    if (has_marks) {
      for (int k = tid; k < (int)L::kMarks / 4; k += kWarps * 32) marks[k] = 0u;
      if (tid == 0) *marked = 0;
      named_sync(1, kWarps * 32);
    }
    if (kN > 1) {
      more = walk.next(it);
      if (more) load_queries();
    }
  }
}

template <int D, int kN, int kG, typename P>
cudaError_t allow() {
  return cudaFuncSetAttribute(quantised_attention_kernel<D, kN, kG, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)CodeLayout<D>::kSmem);
}
template <int D, typename P>
cudaError_t allow_rows() {
  cudaError_t e = allow<D, 1, 1, P>();
  if (e == cudaSuccess) e = allow<D, 2, 1, P>();
  if (e == cudaSuccess) e = allow<D, 2, 2, P>();
  return e == cudaSuccess ? allow<D, 2, 4, P>() : e;
}

template <int D, int kN, int kG, typename P>
int launch(const moe_attn& h, const P& p, const moe_cache_scales_t& s, const Maps& maps, moe_stream_t stream) {
  // with fewer registers than the shares of its warps a block would wait for them for ever
  static const int registers = [] {
    cudaFuncAttributes f{};
    return cudaFuncGetAttributes(&f, quantised_attention_kernel<D, kN, kG, P>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (registers != kLaunchRegisters)
    return fail(MOE_ERR_CUDA, "the kernel has %d registers, not %d", registers, kLaunchRegisters);
  const float c = p.a.scale * 1.4426950408889634f;
  return launch_pdl(quantised_attention_kernel<D, kN, kG, P>, dim3(h.n_sms / p.spread * p.spread), dim3(kCodeThreads),
                    CodeLayout<D>::kSmem, stream, 1, p, s, c, maps.k, maps.v);
}
template <int D, typename P>
int launch_rows(const moe_attn& h, const P& p, const moe_cache_scales_t& s, const Maps& maps, moe_stream_t stream) {
  const int rows = code_rows(p.tokens * p.group);
  return rows == 8    ? launch<D, 1, 1>(h, p, s, maps, stream)
         : rows == 16 ? launch<D, 2, 1>(h, p, s, maps, stream)
         : rows == 32 ? launch<D, 2, 2>(h, p, s, maps, stream)
                      : launch<D, 2, 4>(h, p, s, maps, stream);
}

template <typename T, int D>
int launch_code_join(const moe_attn& h, const AttnParams& p, moe_stream_t stream) {
  const dim3 threads(kJoinRows * kJoinGroups * D / 4);
  const int rows = std::max(1, std::min(p.a.max_q_len, p.tokens)) * p.group;
  if (p.by_item)
    return launch_pdl(join_kernel<T, D, kTile, true>,
                      dim3(p.a.batch * p.n_kv_heads, (rows + kJoinRows - 1) / kJoinRows), threads, 0, stream, 1, p);
  return launch_pdl(join_kernel<T, D, kTile, false>, dim3(h.n_sms / p.spread * p.spread, (rows + kJoinRows - 1) / kJoinRows),
                    threads, 0, stream, 1, p);
}

// ---- pages in 16 bits, for chunks of many rows -------------------------------------------------------------------------

struct UnpackArgs {
  const uint8_t* cache[2];
  int64_t page_stride[2], row_stride[2];
  const uint8_t* scale[2];
  int64_t scale_page[2], scale_head[2];
  uint16_t* out[2];
  const int32_t* block_table;
  const int32_t* kv_lens;
  int32_t* table;
  int* status;
  int table_stride, page_size, n_pages, n_kv_heads, head_dim;
  int out_stride, prefix_pages, own_pages;
  bool prefix, bf16;
};

constexpr int kUnpackThreads = 256;
// Most CTAs of a call, in waves of them: 32 chunks of 9 tokens of 32/4 heads over
// 2,000 to 32,768 positions in a table of that width take 460 us with 2, 415 with 4,
// 409 with 8, and with one for each page of it 436; over up to 2,000 in a table of
// 18,000 63, 64, 69 and 116.
constexpr int kUnpackWaves = 4;

// Page `page` of the cache in 16 bits as page `to`, by a CTA.
__device__ __forceinline__ void unpack_page(const UnpackArgs& a, int z, int page, long long to) {
  const bool there = (unsigned)page < (unsigned)a.n_pages;
  const int tid = threadIdx.x;
  if (!there && tid == 0) atomicOr(a.status, kAttnBadPage);
  const int per_head = a.head_dim / 16, per_row = a.n_kv_heads * per_head, units = a.page_size * per_row;
  const uint8_t* from = a.cache[z] + (there ? page : 0) * a.page_stride[z];
  const uint8_t* scale = a.scale[z] + (there ? page : 0) * a.scale_page[z];
  uint16_t* out = a.out[z] + to * units * 16;
  for (int u = tid; u < units; u += kUnpackThreads) {
    const int row = u / per_row, in_row = u - row * per_row, head = in_row / per_head;
    uint4 codes = make_uint4(0u, 0u, 0u, 0u);
    uint32_t byte = kScaleBias;
    if (there) {
      codes = *reinterpret_cast<const uint4*>(from + row * a.row_stride[z] + in_row * 16);
      byte = scale[head * a.scale_head[z] + row];
    }
    uint32_t v[8];
    expand_e4m3(codes, power_of_two(exponent_of(byte)), a.bf16, v);
    uint4* dst = reinterpret_cast<uint4*>(out + (long long)u * 16);
    dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
    dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// CTA (x, z): a page of the prefix, then `ctas` for each sequence, which take its
// pages in turn, as many as the length found here says; z: keys or values.  Of a
// prompt's hundreds of pages it is the latency of length, entry and codes (6 MB:
// 11 us under a profiler, DRAM 9 %), of the decode batch's 0.4 GB memory (about 260
// us, 4.7 TB/s read and written).
__global__ void __launch_bounds__(kUnpackThreads) unpack_kernel(const __grid_constant__ UnpackArgs a, int ctas) {
  const int from_prefix = a.prefix ? a.prefix_pages : 0, x = (int)blockIdx.x, z = blockIdx.y;
  const bool prefix = x < from_prefix;
  const int b = prefix ? 0 : (x - from_prefix) / ctas, skip = prefix ? 0 : a.prefix_pages;
  int i = prefix ? x : x - from_prefix - b * ctas;
  pdl_wait();
  pdl_launch_dependents();
  const int32_t* row = a.block_table + (long long)b * a.table_stride + skip;
  // of the sequence's own pages those that begin before its end
  const int pages = prefix ? a.prefix_pages : a.own_pages, len = prefix ? 0x7fffffff : a.kv_lens[b];
  for (; i < pages && (prefix || ((long long)skip + i) * a.page_size < len); i += prefix ? pages : ctas) {
    const long long to = prefix ? i : (long long)a.prefix_pages + (long long)b * a.own_pages + i;
    if (z == 0 && threadIdx.x == 0) a.table[(long long)b * a.out_stride + skip + i] = (int)to;
    unpack_page(a, z, row[i], to);
  }
}

}  // namespace

int code_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : kMaxCodeRows; }

cudaError_t allow_quantised(int head_dim) {
  const cudaError_t e = head_dim == 64 ? allow_rows<64, CodeParams>() : allow_rows<128, CodeParams>();
  return e != cudaSuccess   ? e
         : head_dim == 64 ? allow_rows<64, SharedCodeParams>()
                            : allow_rows<128, SharedCodeParams>();
}

int launch_quantised(const moe_attn& h, const AttnParams& p, const moe_cache_scales_t& s, const Maps& maps,
                     moe_stream_t stream) {
  const CodeParams c{p};
  const int rc = h.head_dim == 64 ? launch_rows<64>(h, c, s, maps, stream) : launch_rows<128>(h, c, s, maps, stream);
  if (rc != MOE_OK) return rc;
  AttnParams joined = p;
  joined.a.scale = kUnitScale;
  if (p.a.dtype == MOE_DTYPE_BF16)
    return h.head_dim == 64 ? launch_code_join<__nv_bfloat16, 64>(h, joined, stream)
                            : launch_code_join<__nv_bfloat16, 128>(h, joined, stream);
  return h.head_dim == 64 ? launch_code_join<__half, 64>(h, joined, stream)
                          : launch_code_join<__half, 128>(h, joined, stream);
}

int launch_quantised(const moe_attn& h, const SharedParams& p, const moe_cache_scales_t& s, const Maps& maps,
                     moe_stream_t stream) {
  const SharedCodeParams c{p};
  return h.head_dim == 64 ? launch_rows<64>(h, c, s, maps, stream) : launch_rows<128>(h, c, s, maps, stream);
}

int launch_unpack(const moe_attn& h, const moe_attn_args_t& a, const moe_cache_scales_t& s, const Unpacked& to, bool prefix,
                  int batch, moe_stream_t stream) {
  // a CTA for each page that the table has room for, unless they are too many: the
  // table may be much wider than its sequences are long
  const int most = kUnpackWaves * h.n_sms * (2048 / kUnpackThreads) / 2;
  const int ctas = std::min(to.own_pages, std::max(1, most / std::max(1, batch)));
  const long long grid = (prefix ? to.prefix_pages : 0) + (long long)batch * ctas;
  if (grid == 0) return MOE_OK;
  const UnpackArgs u{{static_cast<const uint8_t*>(a.k_cache), static_cast<const uint8_t*>(a.v_cache)},
                     {a.k_page_stride, a.v_page_stride},
                     {a.k_row_stride, a.v_row_stride},
                     {static_cast<const uint8_t*>(s.k_scale), static_cast<const uint8_t*>(s.v_scale)},
                     {s.k_page_stride, s.v_page_stride},
                     {s.k_head_stride, s.v_head_stride},
                     {static_cast<uint16_t*>(to.k), static_cast<uint16_t*>(to.v)},
                     a.block_table, a.kv_lens, to.table, h.status, a.table_stride, a.page_size, a.n_pages, h.n_kv_heads,
                     h.head_dim, to.table_stride, to.prefix_pages, to.own_pages, prefix, a.dtype == MOE_DTYPE_BF16};
  return launch_pdl(unpack_kernel, dim3((unsigned)grid, 2), dim3(kUnpackThreads), 0, stream, 1, u, std::max(1, ctas));
}

}  // namespace wse
