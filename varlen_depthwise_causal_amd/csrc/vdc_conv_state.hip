// The width-4 depthwise causal convolution + SiLU with a carried state: the
// last three inputs of each sequence, kept between calls in a cache
// [slots][3][C] (row 0 the oldest), so that prompts may continue and single
// tokens may follow.  The arithmetic is the packed forward's: FP32, taps
// oldest first with FMAs, then the bias.

#include "vdc_ssm.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

constexpr float kDeepZ = -80.0f;

// Eight channels of a lane.
struct Row8 {
  float v[8];
};

__device__ __forceinline__ Row8 unpack8(u32x4_t r) {
  Row8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.v[2 * i] = bf16_lo(r[i]);
    o.v[2 * i + 1] = bf16_hi(r[i]);
  }
  return o;
}

__device__ __forceinline__ u32x4_t load8(const uint16_t* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}
__device__ __forceinline__ void store8(uint16_t* p, u32x4_t v) {
  *reinterpret_cast<u32x4_t*>(p) = v;
}

struct Taps8 {
  float w[8][4];
  float b[8];
};

// Weight and bias of eight channels: 16-byte loads for either dtype.
__device__ __forceinline__ Taps8 load_taps(const ConvStateArgs& a, int64_t c) {
  Taps8 t;
  if (a.w_bf16) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.w) + c * 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const Row8 r = unpack8(p[q]);
#pragma unroll
      for (int k = 0; k < 8; ++k) t.w[2 * q + k / 4][k % 4] = r.v[k];
    }
  } else {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.w) + c * 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4_t v = p[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) t.w[i][k] = v[k];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) t.b[i] = 0.0f;
  if (a.b && a.b_bf16) {
    const Row8 r = unpack8(load8(static_cast<const uint16_t*>(a.b) + c));
#pragma unroll
    for (int i = 0; i < 8; ++i) t.b[i] = r.v[i];
  } else if (a.b) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.b) + c);
    const f32x4_t lo = p[0], hi = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) t.b[i] = lo[i], t.b[4 + i] = hi[i];
  }
  return t;
}

// bf16(silu(p)) of one token; far below zero, where sigmoid leaves the normal
// range, it is evaluated scaled by 2^64 and rounded by integer arithmetic,
// which is exact for subnormal results too (as in the packed forward).
__device__ __forceinline__ u32x4_t conv_row(const Taps8& t, bool bias, const Row8& h3,
                                            const Row8& h2, const Row8& h1, const Row8& x) {
  float y[8];
  float p[8], pmin = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = t.w[i][0] * h3.v[i];
    v = __builtin_fmaf(t.w[i][1], h2.v[i], v);
    v = __builtin_fmaf(t.w[i][2], h1.v[i], v);
    v = __builtin_fmaf(t.w[i][3], x.v[i], v);
    if (bias) v = v + t.b[i];
    p[i] = v;
    pmin = __builtin_fminf(pmin, v);
    y[i] = v * sigmoid_f32(v);
  }
  u32x4_t out;
#pragma unroll
  for (int d = 0; d < 4; ++d) out[d] = bf16_pack2(y[2 * d], y[2 * d + 1]);
  if (pmin < kDeepZ) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t h[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float z = p[2 * d + q];
        float f = y[2 * d + q];
        if (z < kDeepZ) {
          const float s = __builtin_amdgcn_rcpf(
              0x1p-64f + __builtin_amdgcn_exp2f(__builtin_fmaf(z, -kLog2E, -64.0f)));
          f = (z * s) * 0x1p-64f;
        }
        const uint32_t u = __float_as_uint(f);
        h[q] = ((u + 0x7fffu + ((u >> 16) & 1u)) >> 16) & 0xffffu;
        if (f != f) h[q] = 0x7fc0u;
      }
      out[d] = h[0] | (h[1] << 16);
    }
  }
  return out;
}

// One token of each row: reads the row's three last inputs, writes the
// output and the inputs moved up by one.  A wave has 64 vectors of eight
// channels, keeps their weights and takes `rows` rows one after another, the
// next row's loads requested before the current is computed.
//
// Bound by HBM and the last cache, 16 bytes a channel, and below some hundred
// rows by the launch: 1000 rows of 8192 channels 21.6 us (6.1 TB/s), one row of
// 2048 channels 3.2.  Loads and stores past the caches take 25 us there; where
// 20 such layers take turns, 29 us against 31.
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStateArgs a, int32_t rows) {
  const int64_t nvec = a.C / 8, vblocks = (nvec + 63) / 64;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
  const int64_t rb = wave / vblocks;
  const int64_t v = (wave - rb * vblocks) * 64 + (threadIdx.x & 63);
  if (v >= nvec) return;
  const uint32_t c = (uint32_t)v * 8;
  const int64_t row1 = min((rb + 1) * rows, a.rows);
  struct Row {
    int64_t slot;
    u32x4_t h3, h2, h1, x;
  };
  auto load = [&](int64_t row) {
    Row r;
    r.slot = slot_of(a.index, row, a.slots);
    r.x = load8(a.x + row * a.x_stride + c);
    if (r.slot >= 0) {
      const uint16_t* st = a.state + r.slot * 3 * a.C + c;
      r.h3 = load8(st);
      r.h2 = load8(st + a.C);
      r.h1 = load8(st + 2 * a.C);
    }
    return r;
  };
  int64_t row = rb * rows;
  if (row >= row1) return;
  Row next = load(row);
  const Taps8 t = load_taps(a, c);
#pragma unroll 1
  for (; row < row1; ++row) {
    const Row r = next;
    if (row + 1 < row1) next = load(row + 1);
    uint16_t* y = a.y + row * a.C + c;
    if (r.slot < 0) {
      store8(y, (u32x4_t){0u, 0u, 0u, 0u});
      continue;
    }
    uint16_t* st = a.state + r.slot * 3 * a.C + c;
    store8(y, conv_row(t, a.b != nullptr, unpack8(r.h3), unpack8(r.h2), unpack8(r.h1), unpack8(r.x)));
    store8(st, r.h2);
    store8(st + a.C, r.h1);
    store8(st + 2 * a.C, r.x);
  }
}

// What a prompt's carried state changes after the packed forward has run
// with zero history: the first three outputs of a resumed document, and the
// document's last three inputs, which go to its slot.  A lane reads the slot
// before it writes it, so the cache is updated in place.  A launch of its own
// leaves the packed forward as it is, for 2.3 us at 37 documents of 520 channels
// and 4.5 at 22 of 4096 (behind a forward of 175 us).
__global__ __launch_bounds__(64) void conv_edges_kernel(ConvStateArgs a) {
  const int64_t nvec = a.C / 8, per = (nvec + 63) / 64;
  const int64_t doc = blockIdx.x / per;
  const int64_t v = (int64_t)(blockIdx.x - doc * per) * 64 + threadIdx.x;
  const int64_t slot = slot_of(a.index, doc, a.slots);
  if (slot < 0 || v >= nvec) return;
  const int64_t lo = a.cu[doc], hi = a.cu[doc + 1], len = hi - lo;
  if (lo < 0 || hi > a.rows || len < 0) return;  // malformed prefix sums
  const int64_t c = v * 8;
  uint16_t* st = a.state + slot * 3 * a.C + c;
  const uint16_t* x = a.x + lo * a.C + c;
  const bool resume = a.resume && a.resume[doc];
  u32x4_t seq[6];  // three rows of history, then up to three tokens
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    seq[k] = resume ? load8(st + k * a.C) : (u32x4_t){0u, 0u, 0u, 0u};
    seq[3 + k] = k < len ? load8(x + k * a.C) : (u32x4_t){0u, 0u, 0u, 0u};
  }
  if (resume && len > 0) {
    const Taps8 t = load_taps(a, c);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < len)
        store8(a.y + (lo + k) * a.C + c,
               conv_row(t, a.b != nullptr, unpack8(seq[k]), unpack8(seq[k + 1]),
                        unpack8(seq[k + 2]), unpack8(seq[k + 3])));
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    // Row len - 3 + k of the document, or of its history.
    u32x4_t r;
    if (len >= 3) r = load8(x + (len - 3 + k) * a.C);
    else r = len == 2 ? seq[2 + k] : len == 1 ? seq[1 + k] : seq[k];
    store8(st + k * a.C, r);
  }
}

}  // namespace

hipError_t launch_conv_step(const ConvStateArgs& a, hipStream_t s) {
  const int64_t vblocks = (a.C / 8 + 63) / 64;
  // Rows a wave takes: as many as leave four waves a SIMD, at most 8.
  int64_t rows = vblocks * a.rows / 4096;
  rows = rows < 1 ? 1 : rows > 8 ? 8 : rows;
  const int64_t waves = vblocks * ((a.rows + rows - 1) / rows);
  hipLaunchKernelGGL(conv_step_kernel, dim3((uint32_t)((waves + 3) / 4)), dim3(256), 0, s, a, (int32_t)rows);
  return hipGetLastError();
}

hipError_t launch_conv_edges(const ConvStateArgs& a, int64_t docs, hipStream_t s) {
  const int64_t per = (a.C / 8 + 63) / 64;
  hipLaunchKernelGGL(conv_edges_kernel, dim3((uint32_t)(docs * per)), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
