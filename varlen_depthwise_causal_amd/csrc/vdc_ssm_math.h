// Device helpers shared by the state space layer's kernels (the convolution
// with carried state, the selective scan and the gated group norm).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vdc.h"

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

}  // namespace vdc
