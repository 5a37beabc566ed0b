// shared_attention.cu -- attention of a batch whose sequences begin with the same
// pages (include/attention.h): the kernel of paged_attention.cu over a work list
// with one more sequence, all tokens of the batch over the prefix, and the
// joining of every token's two results.
//
//   out = (O_1 2^(c (m_1 - m)) + O_2 2^(c (m_2 - m))) / (l_1 .. + l_2 ..),
// m = max(m_1, m_2), for the unnormalised sums O, l over the prefix and over the
// sequence's own positions: the same as one softmax over both.
//
// One list and one launch for both: prefix and own tiles fill the SMs together,
// and a share's cut may fall anywhere.  A tile that no share cuts leaves its sums
// in fp32 by token, 4 D bytes a row written and read back once, which is little
// beside the positions (128 single tokens of 32/4 heads of 128 behind 16,384: 8 of
// 215 MB) and keeps the output's rounding the only one.
//
// What bounds it: of few tokens the latencies of a short call and of joining the
// prefix's many parts (8 tokens of 20/4 heads behind 8,192 positions: 18 us); of
// large batches the products over the prefix and the short own items, 3 to 4 us
// each that nothing overlaps (128 tokens behind 16,384 with up to 2,000 of their
// own: 77 us, where each sequence read the prefix for itself 13 times the bytes).
#include <algorithm>

#include "attention_handle.cuh"
#include "paged_attention_kernel.cuh"

namespace wse {
namespace {

// Parts of an item that a warp joins by itself (4, 8 or 16: no call measured tells
// them apart); more of them, too, where the rows are many: beyond this many waves of
// joining CTAs (24 tokens of 20/4 heads behind 8,192: 25.1 us with 2, 26.8 with 1;
// 64 of 32/4 behind 16,384: 45.7 with 1 or 2, 57 with 8).
constexpr int kFewJoined = 8, kJoinWaves = 2;

// Where the results of the rows of one of a sequence's own items lie.
template <int D>
struct JoinItem {
  const JoinParams& j;
  const SharedParams& p;
  int b, h, item, first_token, tokens;  // the batch's first token, and how many there are from it
  Seq s;
  Cut own;
  __device__ JoinItem(const JoinParams& j_) : j(j_), p(j_.p) {
    item = blockIdx.x % p.own_items;
    h = blockIdx.x / p.own_items % p.n_kv_heads;
    b = blockIdx.x / p.own_items / p.n_kv_heads + 1;
    // the lengths are no output of the kernel before, which starts this one only
    // after it has waited for what came before itself
    s = load_seq(p, b);
    first_token = max(0, min(p.a.q_starts[0], p.a.n_tokens));
    tokens = max(0, min(p.a.q_starts[p.a.batch], p.a.n_tokens) - first_token);
  }
  __device__ int rows() const { return j.own.tiles * kTile; }
  __device__ bool empty() const { return item * j.own.tiles * j.own.tokens >= s.n; }
  __device__ void load() { own = p.cuts[p.item_number(b, h, item)]; }
  // row r's token in the sequence; s.n: none
  __device__ int token_of(int r) const {
    const int in_tile = r % kTile / p.group;
    return in_tile < j.own.tokens ? (item * j.own.tiles + r / kTile) * j.own.tokens + in_tile : s.n;
  }
  struct Row {
    int token, head, first;  // first: parts of the prefix, before the own ones
    int row, before_row, parts;
    long long before, own;   // the whole results' places
    Cut prefix;
  };
  __device__ Row row_of(int r) const {
    Row x{};
    x.token = token_of(r);
    if (x.token >= s.n) return x;
    const int in_group = r % kTile % p.group, t = s.q0 + x.token, from = t - first_token;
    const int per = j.before.tiles * j.before.tokens, place = from % per;
    x.row = r;
    x.head = h * p.group + in_group;
    // starts that descend may name tokens that the prefix's list does not hold
    x.prefix = (unsigned)from < (unsigned)tokens ? p.cuts[p.item_number(0, h, from / per)] : Cut{};
    x.before_row = place / j.before.tokens * kTile + place % j.before.tokens * p.group + in_group;
    x.before = p.whole_row(0, t, x.head);
    x.own = p.whole_row(b, t, x.head);
    x.first = x.prefix.parts;
    x.parts = x.first + own.parts;
    return x;
  }
  __device__ long long slot(const Cut& cut, int i) const { return 2ll * (cut.c + i * p.spread) + (i == 0 ? 1 : 0); }
  __device__ long long place_of(const JoinSide& side, const Cut& cut, int i, int row) const {
    return slot(cut, i) * (side.tiles * kTile) + row;
  }
  // part i's maximum as an exponent in base 2, and its sum
  __device__ float2 ml_of(const Row& x, int i) const {
    const bool before = i < x.first;
    const float2 ml =
        before ? (x.first == 1 ? p.whole_ml[x.before] : j.before.part_ml[place_of(j.before, x.prefix, i, x.before_row)])
               : (own.parts == 1 ? p.whole_ml[x.own] : j.own.part_ml[place_of(j.own, own, i - x.first, x.row)]);
    return make_float2(ml.x * (before ? j.before.c : j.own.c), ml.y);
  }
  __device__ float4 sums_of(const Row& x, int i, int column) const {
    const float* at =
        i < x.first
            ? (x.first == 1 ? p.whole_o + x.before * D : j.before.part_o + place_of(j.before, x.prefix, i, x.before_row) * D)
            : (own.parts == 1 ? p.whole_o + x.own * D : j.own.part_o + place_of(j.own, own, i - x.first, x.row) * D);
    return reinterpret_cast<const float4*>(at)[column];
  }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
// (1 / sum, log-sum) of a row.
__device__ __forceinline__ float2 total_of(float m, float l) {
  return make_float2(l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l),
                     l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f);
}
__device__ __forceinline__ void add_scaled(float4& o, float4 v, float f) {
  o.x = fmaf(v.x, f, o.x);
  o.y = fmaf(v.y, f, o.y);
  o.z = fmaf(v.z, f, o.z);
  o.w = fmaf(v.w, f, o.w);
}
template <typename T>
__device__ __forceinline__ void write_row(const SharedParams& p, long long t, int head, int column, float4 o, float2 total) {
  const moe_attn_args_t& a = p.a;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + t * a.out_token_stride + head * a.out_head_stride + column * 4) =
      make_uint2(pack<T>(o.x * total.x, o.y * total.x), pack<T>(o.z * total.x, o.w * total.x));
  if (a.lse && column == 0) a.lse[t * (p.group * p.n_kv_heads) + head] = total.y;
}

// Joins a token's results.  Block (i, y): item i of the sequences' own, 4 rows at
// a time; the parts of a row, of the prefix and then of its own positions, are
// read and added in that order, so the same call gives the same bits every time.
//
// Where few tokens share the prefix it is cut into many parts (8 tokens of 20
// heads: 30 for each), whose latency is what counts: four threads for each column
// take a quarter of them each.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinRows * kJoinGroups * D / 4)
    join_many_parts_kernel(const __grid_constant__ JoinParams j) {
  constexpr int kColumns = D / 4;
  __shared__ float factor[kJoinRows][2 * kMaxParts];
  __shared__ float4 sums[kJoinGroups - 1][kJoinRows][kColumns];
  __shared__ float2 total[kJoinRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int column = tid % kColumns, row = tid / kColumns % kJoinRows, group = tid / (kColumns * kJoinRows);
  JoinItem<D> it(j);
  pdl_wait();
  pdl_launch_dependents();
  if (it.empty()) return;
  it.load();
  for (int r0 = blockIdx.y * kJoinRows; r0 < it.rows(); r0 += gridDim.y * kJoinRows) {
    if (it.token_of(r0) >= it.s.n) continue;  // nor does a later row of the four have a token
    const auto mine = it.row_of(r0 + row);
    const bool valid = mine.token < it.s.n;
    // the first parts' sums are on their way while the factors are worked out
    constexpr int kAhead = 4;
    const int share = valid ? (mine.parts + kJoinGroups - 1) / kJoinGroups : 0;
    const int first = group * share, end = valid ? min(mine.parts, first + share) : 0;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (first + i < end) ahead[i] = it.sums_of(mine, first + i, column);
    if (warp < kJoinRows) {
      const auto x = it.row_of(r0 + warp);
      if (x.token < it.s.n) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < x.parts; i += 32) m = fmaxf(m, it.ml_of(x, i).x);
        m = warp_max(m);
        for (int i = lane; i < x.parts; i += 32) {
          const float2 ml = it.ml_of(x, i);
          const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
          factor[warp][i] = nothing_seen(ml) ? -1.f : f;
          l += ml.y * f;
        }
        l = warp_sum(l);
        if (lane == 0) total[warp] = total_of(m, l);
      }
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, float4 v) {
      const float f = factor[row][i];
      if (!(f < 0.f)) add_scaled(o, v, f);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (first + i < end) add(first + i, ahead[i]);
#pragma unroll 4
    for (int i = first + kAhead; i < end; ++i) add(i, it.sums_of(mine, i, column));
    if (group > 0) sums[group - 1][row][column] = o;
    __syncthreads();
    if (valid && group == 0) {
#pragma unroll
      for (int q = 0; q < kJoinGroups - 1; ++q) add_scaled(o, sums[q][row][column], 1.f);
      write_row<T>(j.p, it.s.q0 + mine.token, mine.head, column, o, total[row]);
    }
    __syncthreads();  // before the next rows' factors are written
  }
}

// The same for many tokens, whose results have few parts: a warp for each row,
// and nothing shared (128 single tokens behind 16,384: 81 us, with the kernel above 111).
template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinRows) join_few_parts_kernel(const __grid_constant__ JoinParams j) {
  constexpr int kColumns = D / 4, kSide = 32 / kColumns;  // parts side by side
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, column = lane % kColumns, side = lane / kColumns;
  JoinItem<D> it(j);
  pdl_wait();
  pdl_launch_dependents();
  if (it.empty()) return;
  it.load();
  for (int r = blockIdx.y * kJoinRows + warp; r < it.rows(); r += gridDim.y * kJoinRows) {
    const auto x = it.row_of(r);
    if (x.token >= it.s.n) continue;
    float2 ml = lane < x.parts ? it.ml_of(x, lane) : make_float2(-INFINITY, 0.f);
    float m = ml.x;
    for (int i = lane + 32; i < x.parts; i += 32) m = fmaxf(m, it.ml_of(x, i).x);
    m = warp_max(m);
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < x.parts; i0 += 32) {
      if (i0 > 0) ml = i0 + lane < x.parts ? it.ml_of(x, i0 + lane) : make_float2(-INFINITY, 0.f);
      const float f = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - m);
      l += ml.y * f;
      const float used = nothing_seen(ml) ? -1.f : f;
      const int n = min(32, x.parts - i0);
#pragma unroll 4
      for (int i = 0; i < n; i += kSide) {
        const float g = __shfl_sync(0xffffffffu, used, (i + side) & 31);
        if (i + side < n && !(g < 0.f)) add_scaled(o, it.sums_of(x, i0 + i + side, column), g);
      }
    }
    if (kSide == 2) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, 16);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, 16);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
    }
    l = warp_sum(l);
    if (side == 0) write_row<T>(j.p, it.s.q0 + x.token, x.head, column, o, total_of(m, l));
  }
}

template <typename T, int D, bool kPair>
cudaError_t allow() {
  return cudaFuncSetAttribute(paged_attention_kernel<T, D, kPair, SharedParams>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D, kPair>::kSmem);
}
template <int D>
cudaError_t allow_all() {
  cudaError_t e = allow<__nv_bfloat16, D, true>();
  if (e == cudaSuccess) e = allow<__nv_bfloat16, D, false>();
  if (e == cudaSuccess) e = allow<__half, D, true>();
  return e == cudaSuccess ? allow<__half, D, false>() : e;
}

template <typename T, int D, bool kPair>
int launch(const moe_attn& h, const SharedParams& p, const Maps& maps, moe_stream_t stream) {
  using L = Layout<D, kPair>;
  return launch_pdl(paged_attention_kernel<T, D, kPair, SharedParams>, dim3(h.n_sms / p.spread * p.spread),
                    dim3(L::kThreads), L::kSmem, stream, 1, p, maps.q, maps.k, maps.v);
}
template <typename T, int D>
int launch(const moe_attn& h, const SharedParams& p, bool pair, const Maps& maps, moe_stream_t stream) {
  return pair ? launch<T, D, true>(h, p, maps, stream) : launch<T, D, false>(h, p, maps, stream);
}

template <typename T, int D>
int launch_join(const moe_attn& h, const JoinParams& j, moe_stream_t stream) {
  const SharedParams& p = j.p;
  // as many blocks as the rows of an item have use for
  const int rows = j.own.tiles == 2 ? 2 * kTile : std::max(1, std::min(p.a.max_q_len, j.own.tokens)) * p.group;
  const dim3 grid((unsigned)(p.a.batch * p.n_kv_heads * p.own_items), (unsigned)((rows + kJoinRows - 1) / kJoinRows));
  // about as many parts has an item of the prefix if the CTAs do nothing else
  const int parts = h.n_sms / p.spread / p.prefix_items;
  return parts > kFewJoined && (long long)grid.x * grid.y <= kJoinWaves * h.n_sms
             ? launch_pdl(join_many_parts_kernel<T, D>, grid, dim3(kJoinRows * kJoinGroups * D / 4), 0, stream, 1, j)
             : launch_pdl(join_few_parts_kernel<T, D>, grid, dim3(32 * kJoinRows), 0, stream, 1, j);
}

}  // namespace

cudaError_t allow_shared(int head_dim) { return head_dim == 64 ? allow_all<64>() : allow_all<128>(); }

int launch_shared(const moe_attn& h, const SharedParams& p, bool pair, const Maps& maps, moe_stream_t stream) {
  if (p.a.dtype == MOE_DTYPE_BF16)
    return h.head_dim == 64 ? launch<__nv_bfloat16, 64>(h, p, pair, maps, stream)
                            : launch<__nv_bfloat16, 128>(h, p, pair, maps, stream);
  return h.head_dim == 64 ? launch<__half, 64>(h, p, pair, maps, stream) : launch<__half, 128>(h, p, pair, maps, stream);
}

int launch_shared_join(const moe_attn& h, const JoinParams& j, moe_stream_t stream) {
  if (j.p.a.dtype == MOE_DTYPE_BF16)
    return h.head_dim == 64 ? launch_join<__nv_bfloat16, 64>(h, j, stream) : launch_join<__nv_bfloat16, 128>(h, j, stream);
  return h.head_dim == 64 ? launch_join<__half, 64>(h, j, stream) : launch_join<__half, 128>(h, j, stream);
}

}  // namespace wse
