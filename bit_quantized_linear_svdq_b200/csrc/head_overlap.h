// head_overlap.h -- whether two strided tensors of heads share memory.  Plain
// integer code, also compiled by the tests.
//
// A tensor of heads is tokens x heads runs of `bytes` contiguous bytes.  Two runs
// at A and B overlap where -bytes_a < A - B < bytes_b; over all tokens and heads
// of both, A - B is a difference plus multiples of the strides, so for each pair
// of heads (each difference of head numbers, where the head strides agree) the
// tokens need one division if the token strides agree, as in slices of one packed
// projection, and one a token otherwise.
#pragma once

#include <cstdint>

namespace svdq {

struct HeadRuns {
  long long at, token_stride, head_stride;      // address, bytes
  long long tokens, heads, bytes;               // each at least 1
};

// Some k in k0 .. k1 with lo < c + k s < hi.
inline bool step_between(long long c, long long s, long long k0, long long k1, long long lo, long long hi) {
  if (s == 0) return lo < c && c < hi;
  if (s < 0) {
    const long long t = -k1;
    k1 = -k0, k0 = t, s = -s;
  }
  const long long d = lo - c;                   // the first k past lo: floor(d / s) + 1
  long long k = (d >= 0 ? d / s : -((-d + s - 1) / s)) + 1;
  if (k < k0) k = k0;
  return k <= k1 && c + k * s < hi;
}

// Some i < n and j < m with lo < c + i s - j t < hi.
inline bool steps_between(long long c, long long s, long long n, long long t, long long m, long long lo, long long hi) {
  if (s == t) return step_between(c, s, -(m - 1), n - 1, lo, hi);
  if (m < n) {
    for (long long j = 0; j < m; ++j)
      if (step_between(c - j * t, s, 0, n - 1, lo, hi)) return true;
  } else {
    for (long long i = 0; i < n; ++i)
      if (step_between(c + i * s, -t, 0, m - 1, lo, hi)) return true;
  }
  return false;
}

// Heads, then tokens, that follow each other without a gap become one run.
inline HeadRuns merged(HeadRuns r) {
  if (r.heads == 1) r.head_stride = 0;
  if (r.tokens == 1) r.token_stride = 0;
  if (r.heads > 1 && r.head_stride == r.bytes) r.bytes *= r.heads, r.heads = 1, r.head_stride = 0;
  if (r.heads == 1 && r.tokens > 1 && r.token_stride == r.bytes) r.bytes *= r.tokens, r.tokens = 1, r.token_stride = 0;
  return r;
}

inline long long end_of(const HeadRuns& r) {
  return r.at + (r.tokens - 1) * r.token_stride + (r.heads - 1) * r.head_stride + r.bytes;
}

// (Strides of at least 0.)
inline bool runs_overlap(HeadRuns a, HeadRuns b) {
  if (a.at >= end_of(b) || b.at >= end_of(a)) return false;
  a = merged(a);
  b = merged(b);
  const long long c = a.at - b.at, lo = -a.bytes, hi = b.bytes;
  if (a.head_stride == b.head_stride) {
    for (long long h = -(b.heads - 1); h < a.heads; ++h)
      if (steps_between(c + h * a.head_stride, a.token_stride, a.tokens, b.token_stride, b.tokens, lo, hi)) return true;
    return false;
  }
  for (long long h = 0; h < a.heads; ++h)
    for (long long g = 0; g < b.heads; ++g)
      if (steps_between(c + h * a.head_stride - g * b.head_stride, a.token_stride, a.tokens, b.token_stride, b.tokens, lo, hi))
        return true;
  return false;
}

}  // namespace svdq
