// attention_handle.cuh -- the handle of attention.h, and the launches of its
// kernels that lie in translation units of their own.
#pragma once

#include "attention_work.cuh"

namespace wse {

struct Maps {
  CUtensorMap q, k, v;
};

constexpr int kCodes = 2;  // in place of a MOE_DTYPE_*: bytes

// What a map says apart from its address, and the map: encoding one takes some
// microseconds of the host, giving one another address a fraction of that.
struct Shape {
  int dtype, columns, d1, d2, box, rows, slabs;
  int64_t stride1, stride2;
  bool operator==(const Shape& o) const {
    return dtype == o.dtype && columns == o.columns && d1 == o.d1 && d2 == o.d2 && box == o.box && rows == o.rows &&
           slabs == o.slabs && stride1 == o.stride1 && stride2 == o.stride2;
  }
};
struct KnownMap {
  Shape shape{};
  CUtensorMap map;
};

}  // namespace wse

struct moe_attn {
  int n_heads = 0, n_kv_heads = 0, head_dim = 0, n_sms = 0, dev = 0;
  int* status = nullptr;
  float* part_o = nullptr;
  float2* part_ml = nullptr;
  wse::Cut* cuts = nullptr;
  wse::KnownMap q_map, k_map, v_map, k8_map, v8_map;  // 8: of codes
};

namespace wse {

// shared_attention.cu: 16-bit caches behind a shared prefix, in tiles of kTile rows or pairs of them
cudaError_t allow_shared(int head_dim);
int launch_shared(const moe_attn& h, const SharedParams& p, bool pair, const Maps& maps, moe_stream_t stream);
// ... and the joining of every token's two results
int launch_shared_join(const moe_attn& h, const JoinParams& j, moe_stream_t stream);

// quantised_attention.cu, whose scores and maxima are exponents in base 2: what
// joins its results takes this scale
constexpr float kUnitScale = 0.6931471805599453f;
constexpr int kMaxCodeRows = 64;  // query rows of a tile over codes
int code_rows(int rows);          // of the tile that a call takes whose sequences have as many
cudaError_t allow_quantised(int head_dim);
int launch_quantised(const moe_attn& h, const AttnParams& p, const moe_cache_scales_t& s, const Maps& maps,
                     moe_stream_t stream);
int launch_quantised(const moe_attn& h, const SharedParams& p, const moe_cache_scales_t& s, const Maps& maps,
                     moe_stream_t stream);
// Pages in 16 bits, for what reads them often: those of a prefix (of the table's first row) as pages 0 .. prefix_pages -
// 1 of k and v, and behind them own_pages of each sequence.  `table` has a row of as many entries for each sequence, the
// prefix's in the first one alone.
struct Unpacked {
  void* k;
  void* v;
  int32_t* table;
  int table_stride, prefix_pages, own_pages;
};
// of the prefix, if `prefix`, and of `batch` sequences
int launch_unpack(const moe_attn& h, const moe_attn_args_t& a, const moe_cache_scales_t& s, const Unpacked& to, bool prefix,
                  int batch, moe_stream_t stream);

}  // namespace wse
