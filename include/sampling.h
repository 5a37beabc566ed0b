/*
 * sampling.h -- C ABI of drawing each row's next token from its logits, with
 * temperature, top-k, top-p and min-p, from a given uniform number: the step
 * after the vocabulary projection of lm_head.h.  Between the two
 * moe_adjust_logits (at the end) applies penalties for repeated tokens, biases
 * and a grammar's mask to the logits.
 *
 * Row m, with l its logits (NaN counts as -inf) and l0 the largest:
 *   weight      w_i = floor(2^38 * exp((l_i - l0) / temperature)), the
 *               subtraction, division and exp in fp32.  Whole numbers: their
 *               sums do not depend on the order of addition, so the same
 *               inputs give the same token on any grid.
 *               What is infinitely far below l0 weighs nothing, at any
 *               temperature.
 *   temperature not above 0: greedy, the largest logit (probability 1).
 *   top_k       > 0: only the top_k largest logits stay.
 *   top_p       < 1: of those, by falling logit, each stays whose preceding
 *               weights sum to less than top_p times their total (the first
 *               always does).
 *   min_p       > 0: of those, each stays with w_i >= min_p * 2^38 (above 1
 *               counts as 1).
 *   The token is the lowest id whose running sum of the staying weights, by
 *   id, exceeds floor(u * total); its probability is w / total.
 * Equal logits go to the lower id first throughout.  A row without any logit
 * above -inf gives token -1 and probability 0.
 */
#ifndef WSE_SAMPLING_H
#define WSE_SAMPLING_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_SAMPLE_MAX_VOCAB 8388608

/*
 * moe_sample -- asynchronous on `stream`, allocates nothing.
 *   logits       device fp32, row m at logits + m*row_stride elements, 4-byte aligned, read only.
 *   rows, vocab  rows 0..65535 (0: no work), vocab 1..MOE_SAMPLE_MAX_VOCAB.
 *   u            device fp32 [rows], each in [0, 1).
 *   temperature, top_p, min_p   device fp32 [rows]; top_k device int32 [rows]; each may be NULL: 1, 1, 0, 0 (off).
 *   tokens       device int32 [rows].
 *   probs        NULL or device fp32 [rows].
 * MOE_ERR_INVALID_ARG for bad pointers or sizes, MOE_ERR_CUDA if the launch fails.
 */
int moe_sample(const float* logits, int64_t row_stride, int rows, int vocab, const float* u, const float* temperature,
               const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens, float* probs,
               moe_stream_t stream);

/*
 * moe_adjust_logits -- row m of logits, x its value for token v, becomes
 *   x / repetition if x > 0, else x * repetition, where v stands anywhere in
 *                    the row's part of the history (prompt and answer);
 *   x - frequency * (how often v stands in the answer);
 *   x - presence     where it does at all;
 *   x + bias         of the last entry for v in the row's part of the list;
 *   -inf             where v's bit of the row's mask is 0 (whatever x was),
 * each step in fp32 and rounded (the division to within its last bit, of logits
 * below 2^-125 its last two).  What is not given is left out; a NaN without a
 * mask's 0 stays one.  The same inputs give the same bits every time.
 * Asynchronous on `stream`, allocates nothing, can be captured into a graph.
 */
typedef struct {
  const float* logits;     /* device, row m at logits + m*row_stride elements, 4-byte aligned */
  int64_t row_stride;
  float* out;              /* the same shape; may be logits itself (then only what changes is written), else may not
                              overlap it */
  int64_t out_stride;
  int rows, vocab;         /* rows 0..65535 (0: no work), vocab 1..MOE_SAMPLE_MAX_VOCAB */
  const int32_t* history;  /* device [n_history]: tokens; those outside the vocabulary are ignored; may be NULL */
  int n_history;
  const int32_t* spans;    /* device [rows][3]: (begin, answer, end), the row's history is begin..end-1, its answer
                              answer..end-1; rows may share history; cut to 0..n_history.  Not NULL with history */
  const float* repetition; /* device [rows] or NULL */
  const float* presence;   /* device [rows] or NULL */
  const float* frequency;  /* device [rows] or NULL */
  const int32_t* bias_ids; /* device [n_biases], or NULL: tokens; those outside the vocabulary are ignored */
  const float* bias_values;
  int n_biases;
  const int32_t* bias_starts; /* device [rows + 1]: row m has entries bias_starts[m] .. bias_starts[m+1]-1, cut to
                              0..n_biases */
  const uint32_t* allowed; /* device, row m at allowed + m*allowed_stride words: bit v % 32 of word v / 32; or NULL */
  int64_t allowed_stride;  /* 0: the rows share one mask */
} moe_adjust_logits_args_t;

/* MOE_ERR_INVALID_ARG for bad pointers or sizes, MOE_ERR_CUDA if the launch fails. */
int moe_adjust_logits(const moe_adjust_logits_args_t* a, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* WSE_SAMPLING_H */
