// Device helpers shared by the kernels of the state space layer (the convolution
// with carried state, the selective scan and the gated group norm) and of the
// recurrent layer (the gated recurrence, the layer norm, states put aside).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vdc.h"
#include "vdc_search.h"

namespace vdc {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// FP32 -> BF16, round to nearest even.
__device__ __forceinline__ uint32_t bf16_pack2(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
}
__device__ __forceinline__ uint16_t bf16_of(float a) { return (uint16_t)bf16_pack2(a, 0.0f); }

// Element i of a parameter vector of dtype VDC_F32 / VDC_BF16.
__device__ __forceinline__ float param_at(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void param_put(void* p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<uint16_t*>(p)[i] = bf16_of(v);
  else static_cast<float*>(p)[i] = v;
}

// 1 / (1 + exp(-z)).  Below z = -87 the exponential overflows and the result
// is 0: less than the smallest normal number off.
__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2E));
}

// d silu(z) / dz.
__device__ __forceinline__ float dsilu_f32(float z, float s) {
  return s * __builtin_fmaf(z, 1.0f - s, 1.0f);
}

// log(1 + exp(v)) with a small relative error on all of its range: the result
// is a step size, which may be many orders below 1.  With e = exp(-|v|) <= 1 and
// s = e / (2 + e) <= 1/3,
//
//   log1p(e) = 2 atanh(s) = s P(s^2),
//
// P the polynomial of degree 4 nearest to 2 atanh(s) / s in relative error
// (8e-9).  The exponent v log2(e) is rounded once, with a constant that is
// rounded too: at most 1.23 |v| 2^-24 of e.  It is taken from v, the sum of an
// input and its bias, and not from the two of them, whose own roundings do not
// get smaller where they cancel.  A step of -inf has the size 0: e is 0 then, and
// so is max(v, 0).  That maximum drops a NaN, which s brings back.
__device__ __forceinline__ float softplus_f32(float v) {
  const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(v * kLog2E));
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
  const float u = s * s;
  float r = 0.28178334f;
  r = __builtin_fmaf(r, u, 0.27960604f);
  r = __builtin_fmaf(r, u, 0.4002491f);
  r = __builtin_fmaf(r, u, 0.66666317f);
  r = __builtin_fmaf(r, u, 2.0f);
  return __builtin_fmaf(s, r, __builtin_fmaxf(v, 0.0f));
}

// The value of the lane that the DPP control kCtrl names.
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kRor4 = 0x124, kRor8 = 0x128,  // quad_perm, row_ror
              kMirror = 0x140, kHalfMirror = 0x141;

// Sum over the aligned group of L lanes that a lane is in, left in all of
// them, in one fixed order.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (L >= 2) v += dpp<kXor1>(v);
  if constexpr (L >= 4) v += dpp<kXor2>(v);
  if constexpr (L >= 8) v += dpp<kHalfMirror>(v);
  if constexpr (L >= 16) v += dpp<kMirror>(v);
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// Their largest value, in the same way; NaN are left out.
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (L >= 2) v = __builtin_fmaxf(v, dpp<kXor1>(v));
  if constexpr (L >= 4) v = __builtin_fmaxf(v, dpp<kXor2>(v));
  if constexpr (L >= 8) v = __builtin_fmaxf(v, dpp<kHalfMirror>(v));
  if constexpr (L >= 16) v = __builtin_fmaxf(v, dpp<kMirror>(v));
  if constexpr (L >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  if constexpr (L >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  return v;
}

// Eight channels of a row.
struct Vec8 {
  float v[8];
};
__device__ __forceinline__ Vec8 unpack8(u32x4_t r) {
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.v[2 * i] = bf16_lo(r[i]), o.v[2 * i + 1] = bf16_hi(r[i]);
  return o;
}
__device__ __forceinline__ u32x4_t pack8(const Vec8& a) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = bf16_pack2(a.v[2 * i], a.v[2 * i + 1]);
  return r;
}
// At any address that holds BF16 values.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight values, of which there are `count`; the others are zeros.
template <bool kWhole>
__device__ __forceinline__ u32x4_t load8(const uint16_t* p, int32_t count) {
  if (kWhole || count >= 8) {
    if (kWhole) return *reinterpret_cast<const u32x4_t*>(p);
    const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p);
    return (u32x4_t){v[0], v[1], v[2], v[3]};
  }
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = 2 * i < count ? p[2 * i] : 0u, hi = 2 * i + 1 < count ? p[2 * i + 1] : 0u;
    r[i] = lo | hi << 16;
  }
  return r;
}
template <bool kWhole>
__device__ __forceinline__ void store8(uint16_t* p, u32x4_t v, int32_t count) {
  // Every output byte is written once and not read here.
  if (kWhole) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
  else if (count >= 8) *reinterpret_cast<u32x4_any*>(p) = (u32x4_any){v[0], v[1], v[2], v[3]};
  else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
  }
}

typedef const __attribute__((address_space(4))) uint32_t* scalar_ptr;

// Entry i of an int32 array the whole wave asks for, in a scalar register.
__device__ __forceinline__ int32_t uniform_at(const int32_t* p, int64_t i) {
  return (int32_t)((scalar_ptr)(uintptr_t)p)[i];
}

// The slot of sequence `i`, the same for a whole wave, in a cache of `slots`
// sequences, or -1 where it has none (an index outside the cache marks a row
// of padding).
__device__ __forceinline__ int64_t slot_of(const int32_t* index, int64_t i, int64_t slots) {
  const int64_t s = index ? (int64_t)uniform_at(index, i) : i;
  return s >= 0 && s < slots ? s : -1;
}

// First index i in [0, n) with cu[i] >= v (n if none), by a whole wave.
__device__ __forceinline__ int32_t first_at_least(const int32_t* cu, int32_t n, int32_t v) {
  const int lane = (int)(threadIdx.x & 63);
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t step = search_step(lo, hi);
    const int64_t idx = search_probe(lo, hi, step, lane);
    const uint64_t ball = __ballot(idx >= 0 && cu[idx] < v);
    search_narrow(lo, hi, step, ~ball == 0 ? 64 : (int)__builtin_ctzll(~ball));
  }
  return __builtin_amdgcn_readfirstlane((int32_t)lo);
}

}  // namespace vdc
