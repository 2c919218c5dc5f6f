// The sequences of a batch, for the kernels of the operators around the
// recurrence.  Plain C++, so that the host can check them too.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define KDA_SEQS_FN __host__ __device__ __forceinline__
#else
#define KDA_SEQS_FN inline
#endif

namespace kda {

// Tokens [start, end) of a sequence.
struct Span {
  int start, end;
};

// The sequences of a batch, as ranges of its tokens: rows of T tokens, or
// packed ones between the offsets cu.  Whatever cu holds, a range stays inside
// the batch and has no negative length, and a walk (next) takes no token
// twice, so that wrong offsets give wrong results, no wild access, and no more
// work than right ones.
struct Seqs {
  const int32_t* cu;
  int n;
  int64_t T, tokens;

  KDA_SEQS_FN int64_t start(int s) const {
    if (!cu) return s * T;
    const int64_t c = cu[s];
    return c < 0 ? 0 : c > tokens ? tokens : c;
  }
  KDA_SEQS_FN int64_t end(int s) const {
    const int64_t lo = start(s), hi = start(s + 1);
    return hi > lo ? hi : lo;
  }
  // sequence s in a walk over consecutive sequences that has come to token *at
  KDA_SEQS_FN Span next(int s, int* at) const {
    const int lo = (int)start(s), hi = (int)start(s + 1), first = lo > *at ? lo : *at;
    *at = hi > first ? hi : first;
    return Span{first, *at};
  }
  // first sequence that starts at token t or later (n if none does)
  KDA_SEQS_FN int from(int64_t t) const {
    if (!cu) {
      if (T == 0) return t > 0 ? n : 0;
      const int64_t s = (t + T - 1) / T;
      return s < n ? (int)s : n;
    }
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) >= t)
        hi = mid;
      else
        lo = mid + 1;
    }
    return lo;
  }
};

}  // namespace kda
