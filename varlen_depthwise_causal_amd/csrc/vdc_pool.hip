// Carried states put aside in 8 bits and taken back.  For a block of 64 values v
// of a state, with L = 127 (int8) or 448 (e4m3):
//
//   scale = max |v| / L,   code = nearest(v / scale),   v' = code scale
//
// Bound by HBM: a value is 4 (FP32) or 2 (BF16) bytes of state and 17/16 of code
// and scale.  512 states of 65536 FP32 values in e4m3: put aside in 36.5 us, 4.7 TB/s,
// with VALU issue 77% busy, taken back in 33.6, 5.1 TB/s (a copy: 5.1).  One state of
// 32768: 4.2 and 3.0 us, a launch and one turn of loads.

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
// quotient itself.  Below 2^-20 every code is 0.  s is at least 2^-64 / 448, above 2^-73: the
// remainder of a quotient from 2^-20 on is a multiple of 2^-139 (the last bits of t and s
// are 2^-43 and 2^-96), which FP32 holds.
__device__ __forceinline__ float odd_quotient(float v, float s) {
  const float t = v / s;
  const float rest = __builtin_fmaf(-t, s, v);
  uint32_t b = __float_as_uint(t);
  if (__builtin_fabsf(t) >= 0x1p-20f && rest != 0.0f && (b & 1u) == 0u)
    b += (rest > 0.0f) == (t > 0.0f) ? 1u : 0xffffffffu;
  return __uint_as_float(b);
}

// V values a lane, 64 / V lanes a block: 16 bytes of a state (V = 4 or 8) where states
// have a multiple of 64 values and vectors of them and of their codes are aligned,
// else one value (the 512 states: 75 us put aside, 29 taken back).
template <int V, bool kBf16>
__device__ __forceinline__ void state_load(const PoolArgs& a, int64_t at, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = kBf16 ? bf16_f32(static_cast<const uint16_t*>(a.state)[at]) : static_cast<const float*>(a.state)[at];
  } else if constexpr (kBf16) {
    const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.state) + at));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(w[k]), v[2 * k + 1] = bf16_hi(w[k]);
  } else {
    const f32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.state) + at));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = w[k];
  }
}
template <int V, bool kBf16>
__device__ __forceinline__ void state_store(const PoolArgs& a, int64_t at, const float (&v)[V]) {
  if constexpr (V == 1) {
    if (kBf16) static_cast<uint16_t*>(a.state)[at] = bf16_of(v[0]);
    else static_cast<float*>(a.state)[at] = v[0];
  } else if constexpr (kBf16) {
    u32x4_t w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = bf16_pack2(v[2 * k], v[2 * k + 1]);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.state) + at));
  } else {
    __builtin_nontemporal_store((f32x4_t){v[0], v[1], v[2], v[3]},
                                reinterpret_cast<f32x4_t*>(static_cast<float*>(a.state) + at));
  }
}

// V codes, four to a word.
template <int V>
struct Codes {
  static constexpr int kWords = (V + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (V == 1) w[0] = *p;
    else if constexpr (V == 4) w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
    else {
      const u32x2_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
      w[0] = v[0], w[1] = v[1];
    }
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (V == 1) *p = (uint8_t)w[0];
    else if constexpr (V == 4) __builtin_nontemporal_store(w[0], reinterpret_cast<uint32_t*>(p));
    else __builtin_nontemporal_store((u32x2_t){w[0], w[1]}, reinterpret_cast<u32x2_t*>(p));
  }
};

template <bool kE4m3>
__device__ __forceinline__ uint32_t code_of(float t) {
  if (kE4m3) return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, t, 0, false) & 0xffu;
  return (uint32_t)(int32_t)__builtin_rintf(t) & 0xffu;
}

// A workgroup has a part of 4096 values of one state: all its loads at once, sixteen values
// a lane.
template <int V, bool kBf16, bool kE4m3>
__global__ __launch_bounds__(256) void pool_quantize_kernel(PoolArgs a, int32_t parts) {
  const int64_t row = blockIdx.x / parts, part = blockIdx.x - row * parts;
  int64_t slot, place;
  if (!pool_row(a, row, &slot, &place)) return;
  const int64_t blocks = (a.E + kPoolBlock - 1) / kPoolBlock;
  constexpr int kTurns = kPoolValues / (256 * V), kLanes = kPoolBlock / V;
  const int64_t at0 = part * kPoolValues + (int64_t)threadIdx.x * V;
  float v[kTurns][V];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int64_t at = at0 + k * 256 * V;
#pragma unroll
    for (int q = 0; q < V; ++q) v[k][q] = 0.0f;
    if (at < a.E) state_load<V, kBf16>(a, slot * a.E + at, v[k]);
  }
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int64_t at = at0 + k * 256 * V;
    // a maximum drops a NaN, a sum of products with 0 keeps that of an infinity too
    float most = 0.0f, bad = 0.0f;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      most = __builtin_fmaxf(most, __builtin_fabsf(v[k][q]));
      bad = __builtin_fmaf(v[k][q], 0.0f, bad);
    }
    most = lanes_max<kLanes>(most);
    bad = lanes_sum<kLanes>(bad);
    const bool none = !(most >= 0x1p-64f) || bad != bad;
    const float scale = bad != bad ? __builtin_nanf("") : none ? 0.0f : most / (kE4m3 ? 448.0f : 127.0f);
    Codes<V> codes = {};
#pragma unroll
    for (int q = 0; q < V; ++q)
      codes.w[q / 4] |= code_of<kE4m3>(none ? 0.0f : odd_quotient(v[k][q], scale)) << (q % 4 * 8);
    if (at >= a.E) continue;
    codes.store(a.codes + place * a.E + at);
    if (threadIdx.x % kLanes == 0) a.scales[place * blocks + at / kPoolBlock] = scale;
  }
}

template <int V, bool kBf16, bool kE4m3>
__global__ __launch_bounds__(256) void pool_dequantize_kernel(PoolArgs a, int32_t parts) {
  const int64_t row = blockIdx.x / parts, part = blockIdx.x - row * parts;
  int64_t slot, place;
  if (!pool_row(a, row, &slot, &place)) return;
  const int64_t blocks = (a.E + kPoolBlock - 1) / kPoolBlock;
  constexpr int kTurns = kPoolValues / (256 * V);
  const int64_t at0 = part * kPoolValues + (int64_t)threadIdx.x * V;
  Codes<V> codes[kTurns];
  float scale[kTurns];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int64_t at = at0 + k * 256 * V;
    if (at >= a.E) continue;
    codes[k].load(a.codes + place * a.E + at);
    scale[k] = a.scales[place * blocks + at / kPoolBlock];
  }
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int64_t at = at0 + k * 256 * V;
    if (at >= a.E) continue;
    float v[V];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const uint32_t b = codes[k].w[q / 4] >> (q % 4 * 8) & 0xffu;
      v[q] = (kE4m3 ? __builtin_amdgcn_cvt_f32_fp8((int)b, 0) : (float)(int8_t)b) * scale[k];
    }
    state_store<V, kBf16>(a, slot * a.E + at, v);
  }
}

template <int V, bool kBf16, bool kE4m3>
void launch_as(const PoolArgs& a, bool back, hipStream_t s) {
  const int32_t parts = (int32_t)((a.E + kPoolValues - 1) / kPoolValues);
  const dim3 grid((uint32_t)(a.rows * parts)), block(256);
  if (back) hipLaunchKernelGGL((pool_dequantize_kernel<V, kBf16, kE4m3>), grid, block, 0, s, a, parts);
  else hipLaunchKernelGGL((pool_quantize_kernel<V, kBf16, kE4m3>), grid, block, 0, s, a, parts);
}

template <bool kE4m3>
hipError_t launch(const PoolArgs& a, bool back, hipStream_t s) {
  const bool vectors = a.E % kPoolBlock == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(a.codes) % 8 == 0;
  if (vectors && a.bf16) launch_as<8, true, kE4m3>(a, back, s);
  else if (vectors) launch_as<4, false, kE4m3>(a, back, s);
  else if (a.bf16) launch_as<1, true, kE4m3>(a, back, s);
  else launch_as<1, false, kE4m3>(a, back, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pool_quantize(const PoolArgs& a, hipStream_t s) {
  return a.e4m3 ? launch<true>(a, false, s) : launch<false>(a, false, s);
}
hipError_t launch_pool_dequantize(const PoolArgs& a, hipStream_t s) {
  return a.e4m3 ? launch<true>(a, true, s) : launch<false>(a, true, s);
}

}  // namespace vdc
