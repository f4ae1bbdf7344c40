// Carried states put aside in 8 bits and taken back.  For a block of 64 values v
// of a state, with L = 127 (int8) or 448 (e4m3):
//
//   scale = max |v| / L,   code = nearest(v / scale),   v' = code scale
//
// Bound by HBM: a value is 4 (FP32) or 2 (BF16) bytes of state and 17/16 of code
// and scale.

#include "vdc_layer.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

constexpr int kPoolValues = 4096;  // values of a state a workgroup has

// The state's slot and the pool's place of row `row`; false: the row is left out.
__device__ __forceinline__ bool pool_row(const PoolArgs& a, int64_t row, int64_t* slot, int64_t* place) {
  *slot = slot_of(a.state_index, row, a.slots);
  *place = slot_of(a.pool_index, row, a.pool);
  return *slot >= 0 && *place >= 0;
}

// v / s rounded to odd: the quotient's 24 bits with the last one set where it is
// not exact, so that rounding it once more to a code gives the code nearest to the
// quotient itself.  Below 2^-20 every code is 0.  s is at least 2^-72, so that the
// remainder has all its bits.
__device__ __forceinline__ float odd_quotient(float v, float s) {
  const float t = v / s;
  const float rest = __builtin_fmaf(-t, s, v);
  uint32_t b = __float_as_uint(t);
  if (__builtin_fabsf(t) >= 0x1p-20f && rest != 0.0f && (b & 1u) == 0u)
    b += (rest > 0.0f) == (t > 0.0f) ? 1u : 0xffffffffu;
  return __uint_as_float(b);
}

__device__ __forceinline__ float max64(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

template <bool kBf16, bool kE4m3>
__global__ __launch_bounds__(256) void pool_quantize_kernel(PoolArgs a, int32_t parts) {
  const int64_t row = blockIdx.x / parts;
  const int64_t part = blockIdx.x - row * parts;
  int64_t slot, place;
  if (!pool_row(a, row, &slot, &place)) return;
  const int64_t blocks = (a.E + kPoolBlock - 1) / kPoolBlock;
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int k = threadIdx.x / 64; k < kPoolValues / kPoolBlock; k += 4) {
    const int64_t block = part * (kPoolValues / kPoolBlock) + k, at = block * kPoolBlock + lane;
    if (block >= blocks) return;
    float v = 0.0f;
    if (at < a.E)
      v = kBf16 ? bf16_f32(static_cast<const uint16_t*>(a.state)[slot * a.E + at])
                : static_cast<const float*>(a.state)[slot * a.E + at];
    const float most = max64(__builtin_fabsf(v));
    // a maximum drops a NaN
    const bool bad = __ballot(!(__builtin_fabsf(v) < __builtin_inff())) != 0;
    const bool none = bad || most < 0x1p-64f;
    const float scale = bad ? __builtin_nanf("") : none ? 0.0f : most / (kE4m3 ? 448.0f : 127.0f);
    const float t = none ? 0.0f : odd_quotient(v, scale);
    uint32_t code;
    if (kE4m3) code = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, t, 0, false) & 0xffu;
    else code = (uint32_t)(int32_t)__builtin_rintf(t) & 0xffu;
    if (at < a.E) a.codes[place * a.E + at] = (uint8_t)code;
    if (lane == 0) a.scales[place * blocks + block] = scale;
  }
}

template <bool kBf16, bool kE4m3>
__global__ __launch_bounds__(256) void pool_dequantize_kernel(PoolArgs a, int32_t parts) {
  const int64_t row = blockIdx.x / parts;
  const int64_t part = blockIdx.x - row * parts;
  int64_t slot, place;
  if (!pool_row(a, row, &slot, &place)) return;
  const int64_t blocks = (a.E + kPoolBlock - 1) / kPoolBlock;
#pragma unroll 1
  for (int k = threadIdx.x; k < kPoolValues; k += 256) {
    const int64_t at = part * kPoolValues + k;
    if (at >= a.E) return;
    const uint32_t code = a.codes[place * a.E + at];
    const float scale = a.scales[place * blocks + at / kPoolBlock];
    const float q = kE4m3 ? __builtin_amdgcn_cvt_f32_fp8((int)code, 0) : (float)(int8_t)code;
    const float v = q * scale;
    if (kBf16) static_cast<uint16_t*>(a.state)[slot * a.E + at] = bf16_of(v);
    else static_cast<float*>(a.state)[slot * a.E + at] = v;
  }
}

}  // namespace

hipError_t launch_pool_quantize(const PoolArgs& a, hipStream_t s) {
  const int32_t parts = (int32_t)((a.E + kPoolValues - 1) / kPoolValues);
  const dim3 grid((uint32_t)(a.rows * parts)), block(256);
  if (a.bf16 && a.e4m3) hipLaunchKernelGGL((pool_quantize_kernel<true, true>), grid, block, 0, s, a, parts);
  else if (a.bf16) hipLaunchKernelGGL((pool_quantize_kernel<true, false>), grid, block, 0, s, a, parts);
  else if (a.e4m3) hipLaunchKernelGGL((pool_quantize_kernel<false, true>), grid, block, 0, s, a, parts);
  else hipLaunchKernelGGL((pool_quantize_kernel<false, false>), grid, block, 0, s, a, parts);
  return hipGetLastError();
}

hipError_t launch_pool_dequantize(const PoolArgs& a, hipStream_t s) {
  const int32_t parts = (int32_t)((a.E + kPoolValues - 1) / kPoolValues);
  const dim3 grid((uint32_t)(a.rows * parts)), block(256);
  if (a.bf16 && a.e4m3) hipLaunchKernelGGL((pool_dequantize_kernel<true, true>), grid, block, 0, s, a, parts);
  else if (a.bf16) hipLaunchKernelGGL((pool_dequantize_kernel<true, false>), grid, block, 0, s, a, parts);
  else if (a.e4m3) hipLaunchKernelGGL((pool_dequantize_kernel<false, true>), grid, block, 0, s, a, parts);
  else hipLaunchKernelGGL((pool_dequantize_kernel<false, false>), grid, block, 0, s, a, parts);
  return hipGetLastError();
}

}  // namespace vdc
