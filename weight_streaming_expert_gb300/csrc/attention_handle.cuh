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

// shared_attention.cu: 16-bit caches, all tokens over a shared prefix
cudaError_t allow_shared(int head_dim);
int launch_shared(const moe_attn& h, const SharedParams& p, const Maps& maps, moe_stream_t stream);
// ... and the joining of every token's two results, for tiles of kTile rows or pairs of them
int launch_shared_join(const moe_attn& h, const SharedParams& p, bool pair, moe_stream_t stream);
bool shared_in_pairs(int n_tokens, int max_q_len, int tokens);

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
// The pages of a->batch sequences in 16 bits, page i of sequence b as page b * table_pages + i of k_out and v_out, and
// that table.
int launch_unpack(const moe_attn& h, const moe_attn_args_t& a, const moe_cache_scales_t& s, void* k_out, void* v_out,
                  int32_t* table, moe_stream_t stream);

}  // namespace wse
