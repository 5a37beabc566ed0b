/*
 * attention.h -- C ABI of the attention half of a decode/verify step, the
 * part that stands before the routed-MoE layer of moe.h:
 *   - norms of queries and keys per head with the position rotation, in one
 *     pass that also writes keys and values into a paged cache;
 *   - attention of a chunk of new tokens over that cache, from one decoded
 *     token per sequence over a verified chain or tree of drafts to a
 *     prompt's chunk of thousands;
 *   - moving pages and rows of the cache (forks, copy on write, compaction,
 *     keeping the accepted rows of a verified tree).
 *
 * The paged cache is memory of the caller: per layer one array of keys and
 * one of values, [n_pages][page_size][n_kv_heads][head_dim], whose first two
 * strides may be larger than the shape's.  Position p of a sequence lies in
 * row p % page_size of page block_table[seq][p / page_size]; a slot is page *
 * page_size + row.  Elements are bf16 or fp16 (MOE_DTYPE_*), the same in
 * every argument of a call.
 *
 * Conventions (device/host pointers, status codes, moe_last_error(), one
 * handle per host thread and stream, sm_103a only) are those of moe.h.  Every
 * call is asynchronous on `stream`, allocates nothing, copies nothing to the
 * host, and can be captured into a CUDA graph.  The framework serves models:
 * none of these operators has a backward pass.
 */
#ifndef WSE_ATTENTION_H
#define WSE_ATTENTION_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_DTYPE_BF16 0
#define MOE_DTYPE_FP16 1

/*
 * moe_qk_norm_rope -- for each token t, head h, with x its D values:
 *   y = x / sqrt(mean(x^2) + eps) * weight          (no weight: y = x)
 *   the first rotary_dim values of y are rotated pair by pair: pair i by the
 *   angle 2 pi * frac(positions[t] * turns[i] / 2^64); the rest stay.
 * Queries go to q_out, keys to k_cache at slots[t], values unchanged to
 * v_cache at slots[t].  fp32 throughout, rounded once on writing.  The angle
 * is exact modulo a turn (integer arithmetic), so far positions lose nothing.
 */
typedef struct {
  int dtype;               /* MOE_DTYPE_* of q, k, v, weights, q_out and the caches */
  int n_tokens;            /* 0: no work */
  int n_heads, n_kv_heads; /* n_heads may be 0 (keys and values only), n_kv_heads too */
  int head_dim;            /* 64, 128 or 256 */
  int rotary_dim;          /* 0 or a multiple of 16, at most head_dim */
  int interleaved;         /* pairs (2i, 2i+1) instead of (i, i + rotary_dim/2) */
  float eps;
  const void* q;           /* device, token t head h at q + t*q_token_stride + h*q_head_stride elements, */
  const void* k;           /* the D values contiguous; bases and strides multiples of 16 bytes */
  const void* v;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  const void* q_weight;    /* device [head_dim], 16-byte aligned, or NULL: queries without norm */
  const void* k_weight;    /* the same for keys */
  const uint64_t* turns;   /* device [rotary_dim/2]: turns per position of pair i as a fraction of 2^64 */
  const int32_t* positions;/* device [n_tokens] (unused when rotary_dim is 0) */
  const int64_t* slots;    /* device [n_tokens]; a slot outside [0, n_pages*page_size) writes no key and value */
  void* q_out;             /* device, strided like q; may be q itself */
  int64_t q_out_token_stride, q_out_head_stride;
  void* k_cache;           /* device, one layer; may not overlap q, k, v */
  void* v_cache;
  int64_t k_page_stride, k_row_stride, v_page_stride, v_row_stride; /* elements */
  int n_pages, page_size;
} moe_qk_norm_rope_args_t;

int moe_qk_norm_rope(const moe_qk_norm_rope_args_t* a, moe_stream_t stream);

/*
 * Attention of new tokens over the paged cache.  Sequence b of the batch has
 * the new tokens q_starts[b] .. q_starts[b+1]-1 (n of them, any count) and
 * kv_lens[b] positions in the cache, the new tokens' own included as the last
 * n.  Token i of the chunk sees position j when
 *   j <= kv_len - n + i                              (no tree_mask), or
 *   j < kv_len - n, or bit j - (kv_len - n) of tree_mask[token] is set,
 * and j < kv_len.  out = sum_j softmax_j(scale * q.k_j) v_j over the seen
 * positions, query head h with key/value head h / (n_heads / n_kv_heads).  A
 * token that sees nothing gets zeros (and -inf as its log-sum).  Keys and values
 * that a token does not see may hold anything, infinities and NaN among them;
 * those that it sees show.
 * Scores, softmax statistics and sums are fp32; the probabilities are rounded
 * to the element type for the second product; out is rounded once.
 */
typedef struct moe_attn moe_attn_t; /* opaque; holds the workspace of split sequences */

/* On the current device, which has to be current in every forward.  n_heads a multiple of n_kv_heads (up to 128 times),
 * head_dim 64 or 128.  NULL on error. */
moe_attn_t* moe_attn_create(int n_heads, int n_kv_heads, int head_dim);

typedef struct {
  int dtype;
  int batch;               /* sequences; 0: no work */
  int n_tokens;            /* rows of q and out */
  int max_q_len;           /* at least the longest chunk; with tree_mask at most 64 */
  float scale;             /* > 0 */
  const void* q;           /* token t head h at q + t*q_token_stride + h*q_head_stride elements */
  int64_t q_token_stride, q_head_stride;
  const void* k_cache;
  const void* v_cache;
  int64_t k_page_stride, k_row_stride, v_page_stride, v_row_stride; /* elements */
  int n_pages, page_size;  /* page_size: 16, 32, 64, 128 or 256 */
  const int32_t* block_table; /* device, row b at block_table + b*table_stride; entries past a sequence's pages are not
                              read.  May be NULL where a row holds no pages */
  int table_stride;        /* from one row to the next; 0: the sequences share one row */
  const int32_t* q_starts; /* device [batch+1], ascending */
  const int32_t* kv_lens;  /* device [batch] */
  const int64_t* tree_mask;/* device [n_tokens] or NULL */
  void* out;
  int64_t out_token_stride, out_head_stride;
  float* lse;              /* NULL, or device [n_tokens][n_heads]: natural log of the sum of exp(scale q.k) */
  int table_pages;         /* pages a row of the table holds; 0: table_stride of them */
} moe_attn_args_t;

/*
 * Errors found on the device (a page outside the cache, whose positions then
 * count as zeros; a length beyond the table or 2^30, which is cut; a chunk
 * longer than max_q_len, whose tokens beyond it are not computed; chunks that
 * overlap, and where they make more work than the limit below nothing is
 * computed; a bounded wait that ran out) set the handle's sticky status word.
 *
 * MOE_ERR_UNSUPPORTED for a batch above 4096, and for more than 2e9 tiles of work, counted with as many positions as
 * a row of the table could hold (a tile: 128 positions of a key/value head for 2 * (128 / group) tokens, half as many
 * where max_q_len is no more than that): 2^20 tokens of 32/4 heads and tables of 2^20 positions are half of it.
 */
int moe_attn_forward(moe_attn_t* h, const moe_attn_args_t* a, moe_stream_t stream);

/* Synchronises the handle's device, then returns and clears the sticky status: MOE_OK, MOE_ERR_INVALID_ARG (bad pages
 * or lengths) or MOE_ERR_DEVICE_TIMEOUT; moe_last_error() names what was found. */
int moe_attn_get_status(moe_attn_t* h);

/* Frees the handle (NULL-safe); synchronises its device first. */
void moe_attn_destroy(moe_attn_t* h);

/*
 * moe_copy_pages -- page dst[i] := page src[i] in every layer of both pools.
 *   pools      device [n_layers][n_pages][page_bytes]: layer l page p at pool + l*layer_stride + p*page_stride
 *              bytes; bases, strides and page_bytes multiples of 16.
 *   src, dst   device int32 [n].  A pair with a page outside [0, n_pages) is left out.  No page may be in dst twice
 *              or in both lists (the copies run in any order).
 */
int moe_copy_pages(void* k_pool, void* v_pool, int n_layers, int64_t k_layer_stride, int64_t v_layer_stride,
                   int64_t k_page_stride, int64_t v_page_stride, int n_pages, int64_t page_bytes, const int32_t* src,
                   const int32_t* dst, int n, moe_stream_t stream);

/*
 * moe_copy_rows -- cache rows dst[i] := src[i] (slots) in every layer of both pools, as if all were read before any
 * is written: the accepted rows of a verified tree moving up to the end of their sequence.
 *   src, dst   device int64 [n], n <= MOE_COPY_ROWS_MAX.  A pair with a slot outside the pool is left out; no slot
 *              may be in dst twice.
 *   row_bytes  bytes of a row (n_kv_heads * head_dim * 2); bases, strides and row_bytes multiples of 16.
 */
#define MOE_COPY_ROWS_MAX 64
int moe_copy_rows(void* k_pool, void* v_pool, int n_layers, int64_t k_layer_stride, int64_t v_layer_stride,
                  int64_t k_page_stride, int64_t v_page_stride, int n_pages, int page_size, int64_t row_bytes,
                  const int64_t* src, const int64_t* dst, int n, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WSE_ATTENTION_H */
