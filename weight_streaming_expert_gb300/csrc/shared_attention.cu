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
// beside the prefix (128 single tokens of 32 heads over 16,384 positions: 4.2 of
// 380 MB) and keeps the output's rounding the only one.
#include <algorithm>

#include "attention_handle.cuh"
#include "paged_attention_kernel.cuh"

namespace wse {
namespace {

// Joins a token's results.  Block (i, y): item i of the sequences' own, 4 rows at
// a time; the parts of a row, of the prefix and then of its own positions, are
// read and added in that order by four threads for each column as in
// join_kernel, so the same call gives the same bits every time.
template <typename T, int D, int kTiles>
__global__ void __launch_bounds__(kJoinRows * kJoinGroups * D / 4)
    shared_join_kernel(const __grid_constant__ SharedParams p) {
  constexpr int kColumns = D / 4, kRows = kTiles * kTile;
  __shared__ float factor[kJoinRows][2 * kMaxParts];
  __shared__ float4 sums[kJoinGroups - 1][kJoinRows][kColumns];
  __shared__ float2 total[kJoinRows];  // (1 / sum, log-sum)
  const moe_attn_args_t& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int column = tid % kColumns, row = tid / kColumns % kJoinRows, group = tid / (kColumns * kJoinRows);
  const int item = blockIdx.x % p.own_items, h = blockIdx.x / p.own_items % p.n_kv_heads;
  const int b = blockIdx.x / p.own_items / p.n_kv_heads + 1;
  // the lengths are no output of the kernel before, which starts this one only
  // after it has waited for what came before itself
  const Seq s = load_seq(p, b);
  const int per = kTiles * p.tokens;
  pdl_wait();
  pdl_launch_dependents();
  if (item * per >= s.n) return;
  const Cut own = p.cuts[p.item_number(b, h, item)];
  const float c = a.scale * 1.4426950408889634f;

  // row r of the item: its token in the sequence (s.n: none), and where its
  // results lie
  auto token_of = [&](int r) {
    const int in_tile = r % kTile / p.group;
    return in_tile < p.tokens ? item * per + r / kTile * p.tokens + in_tile : s.n;
  };
  struct Row {
    int token, head, first;  // first: parts of the prefix
    long long before, own;   // the whole results' places
    int before_row, parts;
    Cut prefix;
  };
  auto row_of = [&](int r) {
    Row x{};
    x.token = token_of(r);
    if (x.token >= s.n) return x;
    const int t = s.q0 + x.token, place = t % per;
    x.head = h * p.group + r % kTile % p.group;
    x.prefix = p.cuts[p.item_number(0, h, t / per)];
    x.before_row = place / p.tokens * kTile + place % p.tokens * p.group + r % kTile % p.group;
    x.before = p.whole_row(0, t, x.head);
    x.own = p.whole_row(b, t, x.head);
    x.first = x.prefix.parts;
    x.parts = x.first + own.parts;
    return x;
  };
  auto slot = [&](const Cut& cut, int i) { return 2ll * (cut.c + i * p.spread) + (i == 0 ? 1 : 0); };
  auto ml_of = [&](const Row& x, int r, int i) {
    if (i < x.first) return x.first == 1 ? p.whole_ml[x.before] : p.part_ml[slot(x.prefix, i) * kRows + x.before_row];
    return own.parts == 1 ? p.whole_ml[x.own] : p.part_ml[slot(own, i - x.first) * kRows + r];
  };
  auto sums_of = [&](const Row& x, int r, int i) {
    const float* at = i < x.first
                          ? (x.first == 1 ? p.whole_o + x.before * D
                                          : p.part_o + (slot(x.prefix, i) * kRows + x.before_row) * D)
                          : (own.parts == 1 ? p.whole_o + x.own * D
                                            : p.part_o + (slot(own, i - x.first) * kRows + r) * D);
    return reinterpret_cast<const float4*>(at)[column];
  };

  for (int r0 = blockIdx.y * kJoinRows; r0 < kRows; r0 += gridDim.y * kJoinRows) {
    if (token_of(r0) >= s.n) continue;  // nor does a later row of the four have a token
    const Row mine = row_of(r0 + row);
    const bool valid = mine.token < s.n;
    // the first parts' sums are on their way while the factors are worked out
    constexpr int kAhead = 4;
    const int share = valid ? (mine.parts + kJoinGroups - 1) / kJoinGroups : 0;
    const int first = group * share, end = valid ? min(mine.parts, first + share) : 0;
    float4 ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (first + i < end) ahead[i] = sums_of(mine, r0 + row, first + i);
    if (warp < kJoinRows) {
      const int r = r0 + warp;
      const Row x = row_of(r);
      if (x.token < s.n) {
        float m = -INFINITY, l = 0.f;
        for (int i = lane; i < x.parts; i += 32) m = fmaxf(m, ml_of(x, r, i).x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        for (int i = lane; i < x.parts; i += 32) {
          const float2 ml = ml_of(x, r, i);
          const float f = ml.x == -INFINITY ? 0.f : exp2_approx((ml.x - m) * c);
          factor[warp][i] = nothing_seen(ml) ? -1.f : f;
          l += ml.y * f;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0)
          total[warp] = make_float2(l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l),
                                    l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.6931471805599453f);
      }
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
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
    for (int i = first + kAhead; i < end; ++i) add(i, sums_of(mine, r0 + row, i));
    if (group > 0) sums[group - 1][row][column] = o;
    __syncthreads();
    if (valid && group == 0) {
#pragma unroll
      for (int q = 0; q < kJoinGroups - 1; ++q) {
        const float4 v = sums[q][row][column];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      const float norm = total[row].x;
      const long long t = s.q0 + mine.token;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + t * a.out_token_stride + mine.head * a.out_head_stride +
                                column * 4) =
          make_uint2(pack<T>(o.x * norm, o.y * norm), pack<T>(o.z * norm, o.w * norm));
      if (a.lse && column == 0) a.lse[t * (p.group * p.n_kv_heads) + mine.head] = total[row].y;
    }
    __syncthreads();  // before the next rows' factors are written
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
int launch(const moe_attn& h, const SharedParams& p, const Maps& maps, moe_stream_t stream) {
  return shared_in_pairs(p.a.n_tokens, p.a.max_q_len, p.tokens) ? launch<T, D, true>(h, p, maps, stream)
                                                                : launch<T, D, false>(h, p, maps, stream);
}

template <typename T, int D>
int launch_join(const SharedParams& p, bool pair, moe_stream_t stream) {
  // as many blocks as the rows of an item have use for
  const int rows = pair ? 2 * kTile : std::max(1, std::min(p.a.max_q_len, p.tokens)) * p.group;
  const dim3 grid((unsigned)(p.a.batch * p.n_kv_heads * p.own_items), (unsigned)((rows + kJoinRows - 1) / kJoinRows));
  return launch_pdl(pair ? shared_join_kernel<T, D, 2> : shared_join_kernel<T, D, 1>, grid,
                    dim3(kJoinRows * kJoinGroups * D / 4), 0, stream, 1, p);
}

}  // namespace

// Whether tiles go in pairs: own chunks of more than a tile do as without a
// prefix, and where many tiles of tokens share the prefix each pair reads it once.
bool shared_in_pairs(int n_tokens, int max_q_len, int tokens) {
  return max_q_len > tokens || n_tokens >= 8 * tokens;
}

cudaError_t allow_shared(int head_dim) { return head_dim == 64 ? allow_all<64>() : allow_all<128>(); }

int launch_shared(const moe_attn& h, const SharedParams& p, const Maps& maps, moe_stream_t stream) {
  if (p.a.dtype == MOE_DTYPE_BF16)
    return h.head_dim == 64 ? launch<__nv_bfloat16, 64>(h, p, maps, stream)
                            : launch<__nv_bfloat16, 128>(h, p, maps, stream);
  return h.head_dim == 64 ? launch<__half, 64>(h, p, maps, stream) : launch<__half, 128>(h, p, maps, stream);
}

int launch_shared_join(const moe_attn& h, const SharedParams& p, bool pair, moe_stream_t stream) {
  if (p.a.dtype == MOE_DTYPE_BF16)
    return h.head_dim == 64 ? launch_join<__nv_bfloat16, 64>(p, pair, stream)
                            : launch_join<__nv_bfloat16, 128>(p, pair, stream);
  return h.head_dim == 64 ? launch_join<__half, 64>(p, pair, stream) : launch_join<__half, 128>(p, pair, stream);
}

}  // namespace wse
