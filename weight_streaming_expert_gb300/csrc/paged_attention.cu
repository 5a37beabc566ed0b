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
#include <algorithm>
#include <cmath>
#include <new>

#include "attention_handle.cuh"
#include "paged_attention_kernel.cuh"

namespace wse {
namespace {

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

// A three-dimensional map, innermost contiguous, whose boxes are a head's or half
// a head's columns of `rows` by `slabs`: 64 of 16 bits, or a head's bytes.
int encode_map(CUtensorMap* map, const Shape& s, const void* base, const char* what) {
  const MapEncode encode = map_encode();
  if (!encode) return fail(MOE_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t dims[3] = {(cuuint64_t)s.columns, (cuuint64_t)s.d1, (cuuint64_t)s.d2};
  const bool codes = s.dtype == kCodes;
  const cuuint64_t strides[2] = {(cuuint64_t)s.stride1 * (codes ? 1 : 2), (cuuint64_t)s.stride2 * (codes ? 1 : 2)};
  const cuuint32_t box[3] = {(cuuint32_t)s.box, (cuuint32_t)s.rows, (cuuint32_t)s.slabs};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r =
      encode(map,
             codes                       ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : s.dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             3, const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             codes && s.box == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS
             ? MOE_OK
             : fail(MOE_ERR_INVALID_ARG, "no tensor map for the strides of %s (driver error %d)", what, (int)r);
}

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
  return cudaFuncSetAttribute(paged_attention_kernel<T, D, kPair, AttnParams>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  const int rc = launch_pdl(paged_attention_kernel<T, D, kPair, AttnParams>, dim3(grid), dim3(L::kThreads), L::kSmem, stream,
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

// What both entries refuse; every stride of the caches a multiple of
// `cache_step` elements.  *none: nothing to compute.
int check_call(const moe_attn* h, const moe_attn_args_t* a, int cache_step, bool* none) {
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
  *none = a->batch == 0 || a->n_tokens == 0;
  if (*none) return MOE_OK;
  if (a->n_pages < 1) return fail(MOE_ERR_INVALID_ARG, "n_pages = %d < 1", a->n_pages);
  if (!a->q || !a->k_cache || !a->v_cache || !a->out || !aligned(a->q, 16) || !aligned(a->k_cache, 16) ||
      !aligned(a->v_cache, 16) || !aligned(a->out, 16))
    return fail(MOE_ERR_INVALID_ARG, "q, out and the caches must be non-null and 16-byte aligned");
  const int table_pages = a->table_pages > 0 ? a->table_pages : a->table_stride;
  if ((!a->block_table && table_pages > 0) || !a->q_starts || !a->kv_lens || !aligned(a->block_table, 4) ||
      !aligned(a->q_starts, 4) || !aligned(a->kv_lens, 4) || !aligned(a->tree_mask, 8) || !aligned(a->lse, 4))
    return fail(MOE_ERR_INVALID_ARG, "block_table, q_starts and kv_lens must be non-null, and all aligned");
  if (((a->q_token_stride | a->q_head_stride | a->out_token_stride | a->out_head_stride) & 7) ||
      ((a->k_page_stride | a->k_row_stride | a->v_page_stride | a->v_row_stride) & (cache_step - 1)))
    return fail(MOE_ERR_INVALID_ARG, "every stride must be a multiple of %d elements (16 bytes)", cache_step);
  if (a->n_tokens > (1 << 30)) return fail(MOE_ERR_UNSUPPORTED, "n_tokens = %d is too many", a->n_tokens);
  if (a->batch > kMaxBatch) return fail(MOE_ERR_UNSUPPORTED, "batch = %d exceeds %d", a->batch, kMaxBatch);
  return MOE_OK;
}

int check_current(const moe_attn& h) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail_cuda(e, "cudaGetDevice");
  if (dev != h.dev)
    return fail(MOE_ERR_INVALID_ARG, "the handle belongs to device %d, the current device is %d", h.dev, dev);
  return MOE_OK;
}

constexpr int kMaxPrefix = 1 << 30;  // positions: a token's number added to them stays in 32 bits

int too_much() { return fail(MOE_ERR_UNSUPPORTED, "too much work for one call: split the tokens"); }

// Units of a key/value head's longest possible item, with the `besides` that its
// list counts for each.
double item_cost(const moe_attn_args_t& a, int pages, int besides) {
  return std::min(1073741824., (double)pages * a.page_size) / kTile + 1 + besides;
}

// A call's parameters for tiles of `tokens` tokens, items of `tiles`.
int fill_params(const moe_attn& h, const moe_attn_args_t& a, int tokens, int tiles, int besides, AttnParams* p) {
  const double item_tokens = (double)tiles * tokens, cost = item_cost(a, a.table_pages, besides);
  if ((a.n_tokens / item_tokens + a.batch) * h.n_kv_heads * cost > kMaxUnits) return too_much();
  const int rc = check_current(h);
  if (rc != MOE_OK) return rc;
  int spread = 1;
  while (spread < kMaxSpread && h.n_kv_heads % (2 * spread) == 0) spread *= 2;
  const bool one_item = a.max_q_len <= tiles * tokens;
  *p = AttnParams{a,        h.n_kv_heads, h.n_heads / h.n_kv_heads, tokens, spread,
                  h.status, h.part_o,     h.part_ml,                h.cuts, one_item && a.batch * h.n_kv_heads <= h.n_sms,
                  a.batch * std::ceil(a.max_q_len / item_tokens) * h.n_kv_heads * cost <= kMaxUnits};
  return MOE_OK;
}

// Maps of the queries (boxes of `tokens` tokens) and a 16-bit cache.
int maps_16(moe_attn* h, const moe_attn_args_t& a, int tokens, Maps* maps) {
  const int group = h->n_heads / h->n_kv_heads, columns = h->n_kv_heads * h->head_dim;
  const int box_rows = std::min(a.page_size, kTile);
  int rc = map_for(h->q_map, {a.dtype, h->head_dim, h->n_heads, a.n_tokens, 64, group, tokens, a.q_head_stride,
                              a.q_token_stride},
                   a.q, &maps->q, "q");
  if (rc == MOE_OK)
    rc = map_for(h->k_map, {a.dtype, columns, a.page_size, a.n_pages, 64, box_rows, 1, a.k_row_stride, a.k_page_stride},
                 a.k_cache, &maps->k, "k_cache");
  if (rc == MOE_OK)
    rc = map_for(h->v_map, {a.dtype, columns, a.page_size, a.n_pages, 64, box_rows, 1, a.v_row_stride, a.v_page_stride},
                 a.v_cache, &maps->v, "v_cache");
  return rc;
}
int maps_codes(moe_attn* h, const moe_attn_args_t& a, Maps* maps) {
  const int columns = h->n_kv_heads * h->head_dim, box_rows = std::min(a.page_size, kTile);
  int rc = map_for(h->k8_map, {kCodes, columns, a.page_size, a.n_pages, h->head_dim, box_rows, 1, a.k_row_stride,
                               a.k_page_stride},
                   a.k_cache, &maps->k, "k_cache");
  if (rc == MOE_OK)
    rc = map_for(h->v8_map, {kCodes, columns, a.page_size, a.n_pages, h->head_dim, box_rows, 1, a.v_row_stride,
                             a.v_page_stride},
                 a.v_cache, &maps->v, "v_cache");
  return rc;
}

moe_attn_args_t with_pages(const moe_attn_args_t& a) {
  moe_attn_args_t r = a;
  r.table_pages = a.table_pages > 0 ? a.table_pages : a.table_stride;
  return r;
}

// What a call with options works on: its longest chunk goes into its tiles, lists
// and workspace, and none is longer than all tokens.
moe_attn_args_t with_bounds(const moe_attn_args_t& a) {
  moe_attn_args_t r = with_pages(a);
  r.max_q_len = std::min(a.max_q_len, a.n_tokens);
  return r;
}

int forward_16(moe_attn* h, const moe_attn_args_t& args, moe_stream_t stream) {
  const moe_attn_args_t a = with_pages(args);
  const int tokens = kTile / (h->n_heads / h->n_kv_heads);
  AttnParams p;
  Maps maps;
  int rc = fill_params(*h, a, tokens, a.max_q_len > tokens ? 2 : 1, kItemCost<2>, &p);
  if (rc == MOE_OK) rc = maps_16(h, a, tokens, &maps);
  if (rc != MOE_OK) return rc;
  if (a.dtype == MOE_DTYPE_BF16)
    return h->head_dim == 64 ? launch_attn<__nv_bfloat16, 64>(h, p, maps, stream)
                             : launch_attn<__nv_bfloat16, 128>(h, p, maps, stream);
  return h->head_dim == 64 ? launch_attn<__half, 64>(h, p, maps, stream)
                           : launch_attn<__half, 128>(h, p, maps, stream);
}

int forward_codes(moe_attn* h, const moe_attn_args_t& a, const moe_attn_opts_t& o, moe_stream_t stream) {
  const int group = h->n_heads / h->n_kv_heads, tokens = code_rows(std::max(1, a.max_q_len) * group) / group;
  AttnParams p;
  Maps maps;
  int rc = fill_params(*h, a, tokens, 1, kCodeItemCost, &p);
  if (rc == MOE_OK) rc = maps_codes(h, a, &maps);
  return rc != MOE_OK ? rc : launch_quantised(*h, p, *o.scales, maps, stream);
}

// Chunks of more rows than a tile over codes has: where a position's codes would
// be converted for every tile, they are converted once for all of them, into
// pages of 16 bits that the 16-bit kernel reads.  Up to there a tile is faster: 64
// rows of 32 sequences of 2,000 to 32,768 positions 175 us, unpacked 368, 32 rows
// 131 and 423; of one over 8,192 17.1 and 20.8.
bool in_chunks(const moe_attn& h, const moe_attn_args_t& a) {
  return std::max(1ll, (long long)a.max_q_len) * (h.n_heads / h.n_kv_heads) > kMaxCodeRows;
}
constexpr size_t kUnpackBytes = size_t{1} << 30;  // sequences beyond that take turns
// of a page in 16 bits, keys and values
size_t page_bytes(const moe_attn& h, const moe_attn_args_t& a) {
  return (size_t)a.page_size * h.n_kv_heads * h.head_dim * 4;
}
// of a sequence's pages behind a prefix in 16 bits, and its row of the table
size_t sequence_bytes(const moe_attn& h, const moe_attn_args_t& a, int prefix_pages) {
  return (a.table_pages - prefix_pages) * page_bytes(h, a) + (size_t)a.table_pages * 16;
}

// Tiles of tokens from which the prefix's list runs by itself (16 tiles behind
// 16,384 positions: 136 us in one list, 152 apart; 32 tiles 209 and 182).
constexpr int kApartTiles = 32;

// How a call with options is worked on, and what it keeps in the workspace.
struct Work {
  bool unpack;                 // every page goes through 16 bits
  // with a prefix:
  bool apart;                  // its list runs by itself, over 16 bits, and the sequences' own after it
  int tokens, tiles;           // of the prefix's tiles and items
  int own_tokens, own_tiles;
  int prefix_pages, prefix_items, own_items;
  size_t ml_at, cuts_at, parts_at, part_ml_at, prefix_at, sequences_at;  // the last two: unpacked pages
  size_t sequence, need, wanted;
};
Work work_of(const moe_attn& h, const moe_attn_args_t& a, const moe_attn_opts_t& o) {
  const int group = h.n_heads / h.n_kv_heads, tile = kTile / group, longest = std::max(1, a.max_q_len);
  Work w{};
  w.unpack = o.scales && in_chunks(h, a);
  w.prefix_pages = o.prefix_len / a.page_size;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at += (bytes + 15) / 16 * 16;
    return from;
  };
  if (o.prefix_len > 0) {
    if (o.scales && !w.unpack) {
      // one tile of codes takes all tokens, or the prefix goes to the 16-bit kernel
      w.apart = (long long)a.n_tokens * group > kMaxCodeRows;
      w.own_tokens = code_rows((w.apart ? longest : a.n_tokens) * group) / group;
      w.own_tiles = 1;
    } else {
      // many tiles of tokens: pairs of them over the prefix
      w.own_tiles = longest > tile ? 2 : 1;
      w.own_tokens = tile;
      w.apart = w.own_tiles == 1 && a.n_tokens >= kApartTiles * tile;
    }
    w.tokens = w.apart ? tile : w.own_tokens;
    w.tiles = w.apart ? (a.n_tokens > tile ? 2 : 1) : w.own_tiles;
    const int per = w.tokens * w.tiles, own_per = w.own_tokens * w.own_tiles;
    w.prefix_items = (a.n_tokens + per - 1) / per;
    w.own_items = (int)(((long long)longest + own_per - 1) / own_per);
    const size_t rows = 2 * (size_t)a.n_tokens * h.n_heads;
    const size_t items = (size_t)h.n_kv_heads * (w.prefix_items + (size_t)a.batch * w.own_items);
    take(rows * h.head_dim * sizeof(float));
    w.ml_at = take(rows * sizeof(float2));
    w.cuts_at = take(items * sizeof(Cut));
    if (w.apart) {
      const size_t parts = (size_t)h.n_sms * 2 * w.tiles * kTile;
      w.parts_at = take(parts * h.head_dim * sizeof(float));
      w.part_ml_at = take(parts * sizeof(float2));
    }
  }
  if (w.unpack || (o.scales && w.apart)) w.prefix_at = take(w.prefix_pages * (page_bytes(h, a) + 16));
  w.need = w.wanted = w.sequences_at = at;
  if (w.unpack) {
    w.sequence = sequence_bytes(h, a, w.prefix_pages);
    w.need += w.sequence;
    w.wanted += w.sequence * std::max<size_t>(1, std::min<size_t>(a.batch, kUnpackBytes / std::max<size_t>(w.sequence, 1)));
  }
  return w;
}

// The lists of a batch behind a prefix over 16-bit caches, or over codes the
// sequences' own list at least (`first`: the prefix's pages in 16 bits then).
int run_shared(moe_attn* h, const moe_attn_args_t& a, const moe_attn_opts_t& o, const Work& w, bool codes,
               const moe_attn_args_t& first, moe_stream_t stream) {
  char* at = static_cast<char*>(o.workspace);
  SharedParams p{};
  int rc = fill_params(*h, a, w.own_tokens, w.own_tiles, kSharedItemCost, &p);
  if (rc != MOE_OK) return rc;
  p.fits = true;
  p.by_item = false;
  p.lists = w.apart ? SharedParams::kOwnOnly : SharedParams::kBoth;
  p.prefix = o.prefix_len;
  p.prefix_pages = w.prefix_pages;
  p.prefix_items = w.prefix_items;
  p.own_items = w.own_items;
  p.whole_o = reinterpret_cast<float*>(at);
  p.whole_ml = reinterpret_cast<float2*>(at + w.ml_at);
  p.cuts = reinterpret_cast<Cut*>(at + w.cuts_at);
  const float c = a.scale * 1.4426950408889634f;
  JoinParams j{p, {}, {w.own_tokens, w.own_tiles, p.part_o, p.part_ml, codes ? 1.f : c}};
  j.before = j.own;
  Maps maps;
  if (w.apart) {
    SharedParams q = p;
    q.a = first;
    q.lists = SharedParams::kPrefixOnly;
    q.tokens = w.tokens;
    q.part_o = reinterpret_cast<float*>(at + w.parts_at);
    q.part_ml = reinterpret_cast<float2*>(at + w.part_ml_at);
    j.before = {w.tokens, w.tiles, q.part_o, q.part_ml, c};
    rc = maps_16(h, first, w.tokens, &maps);
    if (rc == MOE_OK) rc = launch_shared(*h, q, w.tiles == 2, maps, stream);
    if (rc != MOE_OK) return rc;
  }
  rc = codes ? maps_codes(h, a, &maps) : maps_16(h, a, w.own_tokens, &maps);
  if (rc == MOE_OK)
    rc = codes ? launch_quantised(*h, p, *o.scales, maps, stream) : launch_shared(*h, p, w.own_tiles == 2, maps, stream);
  return rc != MOE_OK ? rc : launch_shared_join(*h, j, stream);
}

// a's cache in 16-bit pages of the workspace, `pages` of them.
moe_attn_args_t over_pages(const moe_attn& h, const moe_attn_args_t& a, const Unpacked& u, long long pages) {
  const int64_t row = (int64_t)h.n_kv_heads * h.head_dim;
  moe_attn_args_t r = a;
  r.k_cache = u.k;
  r.v_cache = u.v;
  r.n_pages = (int)std::max(1ll, pages);
  r.k_row_stride = r.v_row_stride = row;
  r.k_page_stride = r.v_page_stride = a.page_size * row;
  r.block_table = u.table;
  r.table_stride = u.table_stride;
  return r;
}

int forward_with(moe_attn* h, const moe_attn_args_t& a, const moe_attn_opts_t& o, moe_stream_t stream) {
  const Work w = work_of(*h, a, o);
  if (o.prefix_len > 0) {
    const double units =
        ((double)w.prefix_items * ((double)o.prefix_len / kTile + 1 + kSharedItemCost) +
         (double)a.batch * w.own_items * item_cost(a, a.table_pages, kSharedItemCost)) * h->n_kv_heads;
    if (units > kMaxUnits) return too_much();
  }
  if (o.prefix_len == 0 && !w.unpack) return forward_codes(h, a, o, stream);
  AttnParams limits;  // before anything is launched
  const int tile = kTile / (h->n_heads / h->n_kv_heads);
  int rc = w.unpack ? fill_params(*h, a, tile, a.max_q_len > tile ? 2 : 1,
                                  o.prefix_len > 0 ? kSharedItemCost : kItemCost<2>, &limits)
                    : MOE_OK;
  if (rc == MOE_OK) rc = check_current(*h);
  if (rc != MOE_OK) return rc;
  char* at = static_cast<char*>(o.workspace);
  if (!w.unpack) {
    if (!o.scales || !w.apart) return run_shared(h, a, o, w, o.scales != nullptr, a, stream);
    // the prefix in 16 bits
    const size_t half = w.prefix_pages * page_bytes(*h, a) / 2;
    const Unpacked u{at + w.prefix_at, at + w.prefix_at + half, reinterpret_cast<int32_t*>(at + w.prefix_at + 2 * half),
                     w.prefix_pages, w.prefix_pages, 0};
    rc = launch_unpack(*h, a, *o.scales, u, true, 0, stream);
    return rc != MOE_OK ? rc : run_shared(h, a, o, w, true, over_pages(*h, a, u, w.prefix_pages), stream);
  }
  // rows without pages: nothing is unpacked, and one call does all
  const int at_once =
      w.sequence == 0 ? a.batch : (int)std::min<size_t>(a.batch, (o.workspace_bytes - w.sequences_at) / w.sequence);
  const int own_pages = a.table_pages - w.prefix_pages;
  const long long pages = w.prefix_pages + (long long)at_once * own_pages;
  if (pages > 0x7fffffffll) return too_much();
  const size_t half = pages * page_bytes(*h, a) / 2;
  char* k = at + w.prefix_at;
  const Unpacked u{k, k + half, reinterpret_cast<int32_t*>(k + 2 * half), a.table_pages, w.prefix_pages, own_pages};
  for (int b = 0; b < a.batch; b += at_once) {
    moe_attn_args_t part = a;
    part.batch = std::min(at_once, a.batch - b);
    part.q_starts = a.q_starts + b;
    part.kv_lens = a.kv_lens + b;
    part.block_table = a.block_table + (long long)b * a.table_stride;
    rc = launch_unpack(*h, part, *o.scales, u, b == 0 && o.prefix_len > 0, part.batch, stream);
    if (rc != MOE_OK) return rc;
    if (a.table_pages > 0) part = over_pages(*h, part, u, pages);
    rc = o.prefix_len > 0 ? run_shared(h, part, o, w, false, part, stream) : forward_16(h, part, stream);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
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
  if (e == cudaSuccess) e = allow_shared(head_dim);
  if (e == cudaSuccess) e = allow_quantised(head_dim);
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
  bool none = false;
  const int rc = check_call(h, a, 8, &none);
  return rc != MOE_OK || none ? rc : forward_16(h, *a, stream);
}

size_t moe_attn_workspace(const moe_attn_t* h, const moe_attn_args_t* a, const moe_attn_opts_t* o) {
  if (!h || !a || !o || a->batch <= 0 || a->n_tokens <= 0 || a->page_size <= 0 || o->prefix_len < 0 ||
      o->prefix_len > kMaxPrefix)
    return 0;
  const moe_attn_args_t all = with_bounds(*a);
  return o->prefix_len / a->page_size > all.table_pages ? 0 : work_of(*h, all, *o).wanted;
}

int moe_attn_forward_ex(moe_attn_t* h, const moe_attn_args_t* a, const moe_attn_opts_t* o, moe_stream_t stream) {
  if (!o || (!o->scales && o->prefix_len == 0)) return moe_attn_forward(h, a, stream);
  bool none = false;
  int rc = check_call(h, a, o->scales ? 16 : 8, &none);
  if (rc != MOE_OK) return rc;
  const moe_cache_scales_t* sc = o->scales;
  if (o->prefix_len < 0 || o->prefix_len % a->page_size)
    return fail(MOE_ERR_INVALID_ARG, "prefix_len = %d: must be whole pages of %d", o->prefix_len, a->page_size);
  if (o->prefix_len > kMaxPrefix)
    return fail(MOE_ERR_UNSUPPORTED, "prefix_len = %d exceeds %d", o->prefix_len, kMaxPrefix);
  const int table_pages = a->table_pages > 0 ? a->table_pages : a->table_stride;
  if (a->batch > 0 && o->prefix_len / a->page_size > table_pages)
    return fail(MOE_ERR_INVALID_ARG, "prefix_len = %d: a row of the table holds %d pages", o->prefix_len, table_pages);
  if (none) return MOE_OK;
  if (sc) {
    if (!sc->k_scale || !sc->v_scale || !aligned(sc->k_scale, 16) || !aligned(sc->v_scale, 16))
      return fail(MOE_ERR_INVALID_ARG, "the scales must be non-null and 16-byte aligned");
    if ((sc->k_page_stride | sc->k_head_stride | sc->v_page_stride | sc->v_head_stride) & 15)
      return fail(MOE_ERR_INVALID_ARG, "every stride of the scales must be a multiple of 16 bytes");
  }
  const moe_attn_args_t all = with_bounds(*a);
  const size_t need = work_of(*h, all, *o).need;
  if (need > 0 && (!o->workspace || !aligned(o->workspace, 16) || o->workspace_bytes < need))
    return fail(MOE_ERR_INVALID_ARG, "the workspace must be 16-byte aligned and hold %zu bytes", need);
  return forward_with(h, all, *o, stream);
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
