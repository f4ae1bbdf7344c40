// Group norm with a SiLU, channels last: each token's channels are normalised
// in groups, the output norm of a linear-attention or state space layer.
// For one token and group, with P = C / G channels:
//
//   xhat = (x - mean) rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   v = w xhat + b,   y = silu(v),  or v silu(z) where a gate z is given
//
//   dv = dy silu'(v)  or  dy silu(z),   dz = dy v silu'(z)
//   q = w dv,   dx = rstd (q - mean(q) - xhat mean(q xhat))
//   dw = sum_t dv xhat,   db = sum_t dv

#include "vdc_ssm.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
  return v;
}

struct Stats {
  float mean, rstd;
};

// The mean first, then the squares of the differences from it.
__device__ __forceinline__ Stats stats_of(const NormArgs& a, const uint16_t* x) {
  const int lane = threadIdx.x & 63;
  float s = 0.0f;
  for (int i = lane; i < a.per; i += 64) s += bf16_f32(x[i]);
  const float mean = wave_sum(s) / (float)a.per;
  float q = 0.0f;
  for (int i = lane; i < a.per; i += 64) {
    const float d = bf16_f32(x[i]) - mean;
    q = __builtin_fmaf(d, d, q);
  }
  return Stats{mean, 1.0f / __builtin_sqrtf(wave_sum(q) / (float)a.per + a.eps)};
}

__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const int lane = threadIdx.x & 63;
  if (e >= a.S * a.G) return;
  const int64_t t = e / a.G, c0 = (e - t * a.G) * a.per;
  const uint16_t* x = a.x + t * a.xs + c0;
  const Stats st = stats_of(a, x);
  for (int i = lane; i < a.per; i += 64) {
    const float xh = (bf16_f32(x[i]) - st.mean) * st.rstd;
    const float v = __builtin_fmaf(xh, param_at(a.w, a.w_bf16, c0 + i),
                                   a.b ? param_at(a.b, a.b_bf16, c0 + i) : 0.0f);
    const float u = a.z ? bf16_f32(a.z[t * a.zs + c0 + i]) : v;
    a.y[t * a.C + c0 + i] = bf16_of(v * (a.z ? u * sigmoid_f32(u) : sigmoid_f32(v)));
  }
}

// A wave takes one group of every prows-th token and keeps its sums for dw
// and db in its own partial row.
__global__ __launch_bounds__(64) void norm_bwd_kernel(NormArgs a) {
  const int64_t row = blockIdx.x / a.G, c0 = (blockIdx.x - row * a.G) * (int64_t)a.per;
  const int lane = threadIdx.x;
  float* pw = a.part + row * 2 * a.C + c0;
  float* pb = pw + a.C;
  for (int i = lane; i < a.per; i += 64) pw[i] = pb[i] = 0.0f;
  const float inv = 1.0f / (float)a.per;
  for (int64_t t = row; t < a.S; t += a.prows) {
    const uint16_t* x = a.x + t * a.xs + c0;
    const Stats st = stats_of(a, x);
    float s1 = 0.0f, s2 = 0.0f;
    for (int i = lane; i < a.per; i += 64) {
      const float w = param_at(a.w, a.w_bf16, c0 + i), b = a.b ? param_at(a.b, a.b_bf16, c0 + i) : 0.0f;
      const float xh = (bf16_f32(x[i]) - st.mean) * st.rstd, v = __builtin_fmaf(xh, w, b);
      const float dy = bf16_f32(a.dy[t * a.dys + c0 + i]);
      const float u = a.z ? bf16_f32(a.z[t * a.zs + c0 + i]) : v, s = sigmoid_f32(u);
      const float dv = dy * (a.z ? u * s : dsilu_f32(u, s));
      if (a.z) a.dz[t * a.C + c0 + i] = bf16_of(dy * v * dsilu_f32(u, s));
      pw[i] = __builtin_fmaf(dv, xh, pw[i]);
      pb[i] += dv;
      s1 = __builtin_fmaf(dv, w, s1);
      s2 = __builtin_fmaf(dv * w, xh, s2);
    }
    s1 = wave_sum(s1) * inv;
    s2 = wave_sum(s2) * inv;
    for (int i = lane; i < a.per; i += 64) {
      const float w = param_at(a.w, a.w_bf16, c0 + i), b = a.b ? param_at(a.b, a.b_bf16, c0 + i) : 0.0f;
      const float xh = (bf16_f32(x[i]) - st.mean) * st.rstd, v = __builtin_fmaf(xh, w, b);
      const float dy = bf16_f32(a.dy[t * a.dys + c0 + i]);
      const float u = a.z ? bf16_f32(a.z[t * a.zs + c0 + i]) : v, s = sigmoid_f32(u);
      const float dv = dy * (a.z ? u * s : dsilu_f32(u, s));
      a.dx[t * a.C + c0 + i] = bf16_of(st.rstd * (dv * w - s1 - xh * s2));
    }
  }
}

// The partial rows of dw and db in order, summed in FP64.
__global__ __launch_bounds__(256) void norm_bwd_sum_kernel(NormArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= 2 * a.C) return;
  double s = 0.0;
  for (int32_t r = 0; r < a.prows; ++r) s += a.part[(int64_t)r * 2 * a.C + i];
  if (i < a.C) param_put(a.dw, a.w_bf16, i, (float)s);
  else if (a.db) param_put(a.db, a.b_bf16, i - a.C, (float)s);
}

}  // namespace

int norm_bwd_rows(int64_t S, int64_t C, int64_t G) {
  (void)C;
  const int64_t want = 8192 / G + 1;
  return (int)(S < want ? S : want);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_fwd_kernel, dim3((uint32_t)((a.S * a.G + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_bwd_kernel, dim3((uint32_t)((int64_t)a.prows * a.G)), dim3(64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd_sum(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((uint32_t)((2 * a.C + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
