// Bracket arithmetic of the 64-ary lower-bound search over cu_seqlens that
// the kernels run with one wave (64 lanes probing at once).  Kept apart, in
// 64-bit arithmetic, so that a CPU program can run the same steps with an
// emulated ballot: the bracket reaches 2^31 - 1 entries, where 32-bit sums
// of the probe offsets would wrap.
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define VDC_HD __host__ __device__
#else
#define VDC_HD
#endif

namespace vdc {

// Spacing of the 64 probes in the bracket [lo, hi) (lo < hi): probe q sits
// at lo + q * step, so the probes span the bracket.
VDC_HD inline int64_t search_step(int64_t lo, int64_t hi) { return (hi - lo + 63) >> 6; }

// Entry probed by lane q, or -1 when it lies at or past hi (no probe).
VDC_HD inline int64_t search_probe(int64_t lo, int64_t hi, int64_t step, int q) {
  const int64_t idx = lo + (int64_t)q * step;
  return idx < hi ? idx : -1;
}

// Narrows [lo, hi) given c, the number of leading probes (lanes 0 .. c-1)
// whose entry is below the value sought: the answer lies after probe c-1
// and at or before probe c.  The bracket shrinks at least 64-fold per round
// and stays inside the previous one.
VDC_HD inline void search_narrow(int64_t& lo, int64_t& hi, int64_t step, int c) {
  const int64_t nlo = c == 0 ? lo : lo + (int64_t)(c - 1) * step + 1;
  const int64_t nhi = lo + (int64_t)c * step;
  hi = nhi < hi ? nhi : hi;
  lo = nlo;
}

// The first index i in [0, n) with at(i) >= v (n if none), by one thread: 31 probes at
// most.  Contents in no order give some index in [0, n].
template <class At>
VDC_HD inline int64_t search_alone(const At& at, int64_t n, int64_t v) {
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo) / 2;
    if ((int64_t)at(mid) < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// The documents around token v of n entries of cu_seqlens, by one thread.
struct TokenDocs {
  int64_t ends;    // the document that ends before the token, or -1
  int64_t starts;  // the one that starts at it, or -1 (behind the last one, too)
  bool any;        // whether there is an entry at the token
};
template <class At>
VDC_HD inline TokenDocs token_docs(const At& at, int64_t n, int64_t v) {
  // Of the entries at one token the first follows the document that ends and the last
  // is that of the one that starts there; others are empty ones'.
  const int64_t first = search_alone(at, n, v);
  if (first == n || (int64_t)at(first) != v) return {-1, -1, false};
  const int64_t last = search_alone(at, n, v + 1) - 1;
  return {first - 1, last >= first && last < n - 1 ? last : -1, true};
}

}  // namespace vdc
