// list_parts.h -- parts of a list of n entries that a call's numbers name, cut
// to the list on both sides before anything is computed from them: any int is
// safe, and no difference or sum of the results with a thread's number leaves
// 32 bits.  Plain C++ for the host, too.
#pragma once

#ifdef __CUDACC__
#define WSE_BOTH __host__ __device__ __forceinline__
#else
#define WSE_BOTH inline
#endif

namespace wse {

WSE_BOTH int cut_to(int v, int low, int high) { return v < low ? low : v > high ? high : v; }

// A row's history begin..end-1, its answer from `answer` on: 0 <= begin <=
// answer <= end <= n.
struct Span {
  int begin, answer, end;
};
WSE_BOTH Span cut_span(int begin, int answer, int end, int n) {
  Span s;
  s.begin = cut_to(begin, 0, n);
  s.end = cut_to(end, s.begin, n);
  s.answer = cut_to(answer, s.begin, s.end);
  return s;
}

}  // namespace wse
