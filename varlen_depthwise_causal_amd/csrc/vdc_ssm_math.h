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

constexpr float kLog2E = 1.4426950408889634f;       // log2(e) to binary32 ...
constexpr float kLog2ELow = 1.925963033500e-8f;     // ... and what that leaves
constexpr float kLn2 = 0.6931471805599453f;

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

// log(1 + exp(v)) with a small relative error on all of its range: the
// result is a step size, which may be many orders below 1.  With
// e = exp(-|v|) <= 1 and s = e / (2 + e) <= 1/3, log1p(e) = 2 atanh(s), by
// its series up to s^15 (what is left is below 2e-9 of it).  Above 20 the
// result is v, half a unit in binary32's last place off at most.
__device__ __forceinline__ float softplus_f32(float v) {
  const float m = -__builtin_fabsf(v);
  const float hi = m * kLog2E;
  const float lo = __builtin_fmaf(m, kLog2ELow, __builtin_fmaf(m, kLog2E, -hi));
  float e = __builtin_amdgcn_exp2f(hi);
  e = __builtin_fmaf(e, lo * kLn2, e);
  const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
  const float q = s * s;
  float r = 1.0f / 15.0f;
  r = __builtin_fmaf(r, q, 1.0f / 13.0f);
  r = __builtin_fmaf(r, q, 1.0f / 11.0f);
  r = __builtin_fmaf(r, q, 1.0f / 9.0f);
  r = __builtin_fmaf(r, q, 1.0f / 7.0f);
  r = __builtin_fmaf(r, q, 1.0f / 5.0f);
  r = __builtin_fmaf(r, q, 1.0f / 3.0f);
  r = __builtin_fmaf(r, q, 1.0f);
  const float l = 2.0f * s * r + __builtin_fmaxf(v, 0.0f);
  return v > 20.0f ? v : l;
}

// The slot of sequence `i` in a cache of `slots` sequences, or -1 where it
// has none (an index outside the cache marks a row of padding).
__device__ __forceinline__ int64_t slot_of(const int32_t* index, int64_t i, int64_t slots) {
  const int64_t s = index ? (int64_t)index[i] : i;
  return s >= 0 && s < slots ? s : -1;
}

}  // namespace vdc
