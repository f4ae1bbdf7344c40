// Checks of arguments that the host entry points share (vdc_ssm_api.cpp,
// vdc_layer_api.cpp).
#pragma once

#include "vdc.h"

#include <initializer_list>
#include <stddef.h>
#include <stdint.h>

#include "vdc_internal.h"

namespace vdc {

constexpr int64_t kMaxC = int64_t(1) << 20;
constexpr int64_t kMaxS = (int64_t(1) << 31) - 1;
// Threads of a launch, all dimensions together.
constexpr int64_t kMaxThreads = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 31;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline bool valid_dtype(int d) { return d == VDC_F32 || d == VDC_BF16; }
inline size_t dtype_bytes(int d) { return d == VDC_BF16 ? 2 : 4; }

// A buffer of a call: where it is and how many bytes it spans (0: absent).
struct Span {
  const void* p;
  size_t n;
};

inline bool overlaps(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.n && pb < pa + a.n;
}

// Bytes from the first to the last element of `rows` BF16 rows.
inline size_t rows_bytes(int64_t rows, int64_t width, int64_t stride) {
  return rows > 0 ? (size_t)((rows - 1) * stride + width) * 2 : 0;
}

// Whether an output shares memory with an input or another output.
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span& i : ins)
      if (overlaps(*o, i)) return true;
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlaps(*o, *q)) return true;
  }
  return false;
}

// Launches and the state a call needs, in turn: the first that the runtime
// refuses ends it.
inline int done(hipError_t e) {
  count_launch();
  return e == hipSuccess ? VDC_OK : VDC_EHIP;
}

}  // namespace vdc
