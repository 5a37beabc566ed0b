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

// A row's entries from..to-1 of a list: 0 <= from <= to <= n.
struct Part {
  int from, to;
};
WSE_BOTH Part cut_part(int from, int to, int n) {
  Part p;
  p.from = cut_to(from, 0, n);
  p.to = cut_to(to, p.from, n);
  return p;
}

}  // namespace wse
