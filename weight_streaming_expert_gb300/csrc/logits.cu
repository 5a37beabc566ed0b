// logits.cu -- penalties for repeated tokens, biases and grammar masks on
// logits before the draw (include/sampling.h).
//
// Per row and token: x / r or x * r for tokens of the history, - f * count - p
// for those of the answer, + bias, -inf where the mask says no.  A logit is
// read and written once (8 bytes, and 1/8 of mask).
//
// A CTA takes kSlice tokens of a row.  It asks for their logits first, then
// counts the row's history in a table in shared memory with a word per token
// (whole numbers: any order gives the same), and meanwhile the logits arrive.
// The history is read by each of a row's CTAs, from L2: 4,000 tokens are 16 KB
// against the 32 KB of logits that a CTA moves.  Of several biases for a token
// the last in the list holds: a second table takes the largest entry number.
//
// In place nothing is asked for ahead: only tokens that change are read, and
// those that the mask forbids only written, each by itself (64 rows as below with
// masks 30 us, without 27).
//
// 64 rows of 157,184 with histories up to 8,000, masks and biases: 28 us, 3 TB/s
// (memory needs 12.5; nothing to adjust: 14 us).  A CTA's life is three latencies,
// of the row's span, of its tokens and logits, and of the table, and the CTAs come
// in three waves; 64 % of the issue slots are taken, DRAM 19 %.  6 rows with a
// history of 4,000: 5.6 us.
#include "host_util.cuh"
#include "list_parts.h"
#include "sampling.h"

namespace wse {
namespace {

constexpr int kLogitThreads = 256;
constexpr int kLogitLoads = 4;                              // float4 of a thread
constexpr int kSlice = kLogitThreads * kLogitLoads * 4;     // tokens of a CTA
constexpr int kTokens = 8;                                  // of the history that a thread has in flight
constexpr int kResident = 5;                                // CTAs of an SM (64 rows: with 4 31 us, with 5 or 6 28)

// (begin, answer, end) of a row, cut to the history.
__device__ __forceinline__ Span span_of(const moe_adjust_logits_args_t& a, int row) {
  const int32_t* s = a.spans + 3ll * row;
  return cut_span(s[0], s[1], s[2], a.n_history);
}
// The row's entries of the list of biases, cut to it.
__device__ __forceinline__ Part part_of(const moe_adjust_logits_args_t& a, int row) {
  return cut_part(a.bias_starts[row], a.bias_starts[row + 1], a.n_biases);
}

// The slice's tokens are numbered from the 16-byte boundary at or before the
// row's first logit, so that a thread's four lie in one aligned load whatever
// the row's address: token = number - shift.  kInPlace: out is logits.
// kAligned: the output rows lie on the same remainder of 16 bytes.
template <bool kInPlace, bool kAligned>
__global__ void __launch_bounds__(kLogitThreads, kResident) adjust_logits_kernel(const __grid_constant__ moe_adjust_logits_args_t a) {
  // kSlice counts of the answer's tokens and a byte for each that the prompt has,
  // then kSlice bias numbers (each only where given)
  extern __shared__ uint4 table_words[];
  const int tid = threadIdx.x, row = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const float* in = a.logits + row * a.row_stride;
  float* out = a.out + row * a.out_stride;
  const int shift = (int)(reinterpret_cast<uintptr_t>(in) >> 2 & 3);
  const int first = (int)blockIdx.x * kSlice - shift;  // token number 0 of the slice
  const bool counts = a.history != nullptr, biases = a.bias_ids != nullptr;
  uint32_t* count_of = reinterpret_cast<uint32_t*>(table_words);
  uint8_t* seen_in_prompt = reinterpret_cast<uint8_t*>(count_of + kSlice);
  int* bias_of = reinterpret_cast<int*>(count_of) + (counts ? kSlice + kSlice / 4 : 0);
  const uint32_t* allowed = a.allowed ? a.allowed + row * a.allowed_stride : nullptr;

  // the thread's four tokens of load i; which of them the vocabulary holds, and
  // which of those the mask allows
  auto token_of = [&](int i) { return first + (i * kLogitThreads + tid) * 4; };
  auto inside_of = [&](int v) {
    if (v >= 0 && v + 3 < a.vocab) return 15u;
    uint32_t bits = 0;
    for (int k = 0; k < 4; ++k) bits |= (unsigned)(v + k) < (unsigned)a.vocab ? 1u << k : 0u;
    return bits;
  };
  auto bits_of = [&](int v, uint32_t inside) {
    if (!allowed || !inside) return inside;
    const int low = max(v, 0);
    const uint32_t word = allowed[low >> 5], next = allowed[min(v + 3, a.vocab - 1) >> 5];
    return __funnelshift_r(word, next, low & 31) << (low - v) & inside;
  };
  auto load4 = [&](int v, uint32_t wanted) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (inside_of(v) == 15u) {
      if (wanted) x = *reinterpret_cast<const float4*>(in + v);
    } else {
      if (wanted & 1) x.x = in[v];
      if (wanted & 2) x.y = in[v + 1];
      if (wanted & 4) x.z = in[v + 2];
      if (wanted & 8) x.w = in[v + 3];
    }
    return x;
  };

  uint32_t allow[kLogitLoads];
  float4 x[kLogitLoads];
#pragma unroll
  for (int i = 0; i < kLogitLoads; ++i) allow[i] = bits_of(token_of(i), inside_of(token_of(i)));
  if (!kInPlace) {
#pragma unroll
    for (int i = 0; i < kLogitLoads; ++i) x[i] = load4(token_of(i), allow[i]);
  }

  // what is not given changes nothing as these numbers
  const float rep = a.repetition ? a.repetition[row] : 1.f, presence = a.presence ? a.presence[row] : 0.f;
  const float frequency = a.frequency ? a.frequency[row] : 0.f;
  // what it is divided by, and the power of two that this leaves: of a repetition
  // whose reciprocal would be subnormal or infinite
  const float scale = fabsf(rep) < 0x1p-100f ? 0x1p60f : fabsf(rep) > 0x1p100f ? 0x1p-60f : 1.f;
  const float by = rep * scale, inverse = __frcp_rn(by);

  // ---- the tables
  if (counts || biases) {
    // the history's first tokens are on their way while the tables are cleared
    const Span span = counts ? span_of(a, row) : Span{0, 0, 0};
    int token[kTokens];
    const int32_t* next = a.history + span.begin + tid;
    int left = span.end - span.begin - tid;  // tokens from `next` on
    auto read_tokens = [&] {
#pragma unroll
      for (int k = 0; k < kTokens; ++k) token[k] = k * kLogitThreads < left ? next[k * kLogitThreads] : -1;
    };
    read_tokens();
    const int words = ((counts ? kSlice + kSlice / 4 : 0) + (biases ? kSlice : 0)) / 4;
    for (int i = tid; i < words; i += kLogitThreads) table_words[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const int lowest = max(first, 0), skipped = lowest - first;  // the slice's first token, and its place
    const unsigned here = (unsigned)max(0, min(first + kSlice, a.vocab) - lowest);  // a row's last slice may hold none
    int answer = span.answer - span.begin - tid;  // tokens from `next` on that are the prompt's
    while (left > 0) {
#pragma unroll
      for (int k = 0; k < kTokens; ++k) {
        const unsigned at = (unsigned)(token[k] - lowest);
        if (at >= here) continue;
        if (k * kLogitThreads >= answer)
          atomicAdd(count_of + skipped + at, 1u);
        else
          seen_in_prompt[skipped + at] = 1;  // by whichever thread
      }
      next += kTokens * kLogitThreads;
      left -= kTokens * kLogitThreads;
      answer -= kTokens * kLogitThreads;
      if (left > 0) read_tokens();
    }
    if (biases) {
      const Part part = part_of(a, row);
      const unsigned entries = (unsigned)(part.to - part.from);  // up to INT_MAX: the step past them stays in 32 bits
      for (unsigned i = tid; i < entries; i += kLogitThreads) {
        const unsigned at = (unsigned)(a.bias_ids[part.from + i] - lowest);
        if (at < here) atomicMax(bias_of + skipped + at, (int)i + 1);
      }
    }
    __syncthreads();
  }

  // ---- the logits
  // v / rep by the reciprocal and a correction from what the product leaves
  // (Markstein's division): a last bit off at most, or the last two of a v below
  // 2^-125, whose remainder loses bits
  auto divided = [&](float v) {
    const float q = __fmul_rn(v, inverse), rest = __fmaf_rn(-q, by, v);
    return __fmul_rn(fabsf(rest) < INFINITY ? __fmaf_rn(rest, inverse, q) : q, scale);  // not of infinities
  };
#pragma unroll
  for (int i = 0; i < kLogitLoads; ++i) {
    const int v = token_of(i), at = v - first;
    const uint32_t inside = inside_of(v);
    if (!inside) continue;
    uint32_t touched = 0;
    uint4 count = make_uint4(0u, 0u, 0u, 0u);
    uint32_t prompt = 0u;
    int4 bias = make_int4(0, 0, 0, 0);
    if (counts) {
      count = *reinterpret_cast<const uint4*>(count_of + at);
      prompt = *reinterpret_cast<const uint32_t*>(seen_in_prompt + at);
    }
    if (biases) bias = *reinterpret_cast<const int4*>(bias_of + at);
    const uint32_t c[4] = {count.x, count.y, count.z, count.w};
    const int b[4] = {bias.x, bias.y, bias.z, bias.w};
    const uint32_t any = count.x | count.y | count.z | count.w | prompt;
    const int biased = bias.x | bias.y | bias.z | bias.w;
    float p[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    if (kInPlace && (any || biased)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) touched |= c[k] || (prompt >> 8 * k & 1) || b[k] ? 1u << k : 0u;
      const float4 y = load4(v, touched & allow[i]);
      p[0] = y.x, p[1] = y.y, p[2] = y.z, p[3] = y.w;
    }
    if (any) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y = p[k] > 0.f ? divided(p[k]) : __fmul_rn(p[k], rep);
        p[k] = c[k] || (prompt >> 8 * k & 1) ? y : p[k];
        const float less = __fsub_rn(__fsub_rn(p[k], __fmul_rn(frequency, (float)c[k])), presence);
        p[k] = c[k] ? less : p[k];
      }
    }
    if (biased) {
      const float* values = a.bias_values + part_of(a, row).from - 1;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (b[k]) p[k] = __fadd_rn(p[k], values[b[k]]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!(allow[i] >> k & 1)) p[k] = -INFINITY;
    if (kInPlace) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((inside >> k & 1) && ((touched >> k & 1) || !(allow[i] >> k & 1))) out[v + k] = p[k];
    } else if (kAligned && inside == 15u) {
      *reinterpret_cast<float4*>(out + v) = make_float4(p[0], p[1], p[2], p[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (inside >> k & 1) out[v + k] = p[k];
    }
  }
}

}  // namespace
}  // namespace wse

using namespace wse;

extern "C" int moe_adjust_logits(const moe_adjust_logits_args_t* a, moe_stream_t stream) {
  if (!a) return fail(MOE_ERR_INVALID_ARG, "null arguments");
  if (a->rows < 0 || a->rows > 65535) return fail(MOE_ERR_INVALID_ARG, "rows = %d: must be in 0..65535", a->rows);
  if (a->vocab < 1 || a->vocab > MOE_SAMPLE_MAX_VOCAB)
    return fail(MOE_ERR_INVALID_ARG, "vocab = %d: must be in 1..%d", a->vocab, MOE_SAMPLE_MAX_VOCAB);
  if (a->n_history < 0 || a->n_biases < 0)
    return fail(MOE_ERR_INVALID_ARG, "n_history and n_biases must be 0 or more");
  if (a->rows == 0) return MOE_OK;
  if (!a->logits || !a->out || !aligned(a->logits, 4) || !aligned(a->out, 4))
    return fail(MOE_ERR_INVALID_ARG, "logits and out must be non-null and 4-byte aligned");
  if (a->history && !a->spans) return fail(MOE_ERR_INVALID_ARG, "a history needs spans");
  if (a->bias_ids && (!a->bias_values || !a->bias_starts))
    return fail(MOE_ERR_INVALID_ARG, "bias_ids need bias_values and bias_starts");
  if (!aligned(a->history, 4) || !aligned(a->spans, 4) || !aligned(a->repetition, 4) || !aligned(a->presence, 4) ||
      !aligned(a->frequency, 4) || !aligned(a->bias_ids, 4) || !aligned(a->bias_values, 4) ||
      !aligned(a->bias_starts, 4) || !aligned(a->allowed, 4))
    return fail(MOE_ERR_INVALID_ARG, "every array must be 4-byte aligned");
  if (a->rows > 1 && (a->row_stride < 0 || a->out_stride < a->vocab))
    return fail(MOE_ERR_INVALID_ARG, "row strides must be 0 or more, and out's rows may not overlap");
  if (a->allowed_stride < 0) return fail(MOE_ERR_INVALID_ARG, "allowed_stride must be 0 or more");
  const bool in_place = a->out == a->logits;
  if (in_place && a->rows > 1 && a->out_stride != a->row_stride)
    return fail(MOE_ERR_INVALID_ARG, "logits adjusted in place have one row stride");
  const int rc = check_device();
  if (rc != MOE_OK) return rc;
  // up to three numbers before the first token, see `shift`
  const unsigned slices = (unsigned)((a->vocab + 3 + kSlice - 1) / kSlice);
  const size_t smem = ((a->history ? 5u : 0u) + (a->bias_ids ? 4u : 0u)) * kSlice;
  const bool same = ((reinterpret_cast<uintptr_t>(a->logits) ^ reinterpret_cast<uintptr_t>(a->out)) & 15) == 0 &&
                    (a->rows == 1 || ((a->row_stride ^ a->out_stride) & 3) == 0);
  return launch_pdl(in_place ? adjust_logits_kernel<true, true>
                             : same ? adjust_logits_kernel<false, true> : adjust_logits_kernel<false, false>,
                    dim3(slices, (unsigned)a->rows), dim3(kLogitThreads), smem, stream, 1, *a);
}
