// The gated linear recurrence over packed documents: forward for prompts and
// training, backward, and the form for single tokens.  For token t, channel c,
// with u = 2 scale softplus(decay) sigmoid(r):
//
//   a = exp(-u / 2),  m = sqrt(1 - exp(-u)),  h[t] = a h[t-1] + m sigmoid(i) x
//   y = h silu(z),  or h
//
// Backward, with g = dy silu(z) and l the gradient at h:
//
//   l[t] = g[t] + a[t+1] l[t+1],   E = l (sigmoid(i) x a^2 u / (2 m) - u/2 a h[t-1])
//   dx = l m sigmoid(i),  di = l m x sigmoid'(i),  dr = E (1 - sigmoid(r))
//   ddecay = sigmoid(decay) / softplus(decay) sum_t E,  dz = dy h silu'(z)
//
// Everything between documents is assigned, never multiplied by zero, so that
// an infinity or a NaN stays in its document.

#include <cfloat>

#include "vdc_layer.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

// u / sigmoid(r) of a channel.
__device__ __forceinline__ float decay_rate(const RecurArgs& a, int64_t c) {
  return 2.0f * a.scale * softplus_f32(param_at(a.decay, a.decay_bf16, c));
}

// What one token does to the state of a channel.
struct Gates {
  float si, sr;  // sigmoids of the two gates
  float u, a;    // the decay exp(-u / 2)
  float v;       // 1 - exp(-u)
  bool none;     // the token leaves the state as it is
  float rm, m;   // 1 / sqrt(v) and sqrt(v); both 0 without a step
  float gx;      // sigmoid(i) x
  float b;       // what the token adds to the state
};

// 1 - a^2 cancels where a is near 1: below u = 1/4 it is the series of 1 - exp(-u),
// whose first term left out is less than u^6 / 5040 of it, 2^-24.  A token whose u
// is below the normal numbers has no step.
__device__ __forceinline__ Gates gates(float rate, float x, float r, float i) {
  Gates g;
  g.sr = sigmoid_f32(r);
  g.si = sigmoid_f32(i);
  const float u = rate * g.sr;
  g.u = u > 256.0f ? 256.0f : u;  // no infinity times zero; a NaN stays
  g.a = __builtin_amdgcn_exp2f(g.u * (-0.5f * kLog2E));
  float s = __builtin_fmaf(g.u, -1.0f / 720.0f, 1.0f / 120.0f);
  s = __builtin_fmaf(g.u, -s, 1.0f / 24.0f);
  s = __builtin_fmaf(g.u, -s, 1.0f / 6.0f);
  s = __builtin_fmaf(g.u, -s, 0.5f);
  s = __builtin_fmaf(g.u, -s, 1.0f);
  g.v = g.u < 0.25f ? g.u * s : __builtin_fmaf(-g.a, g.a, 1.0f);
  g.none = g.v < FLT_MIN;
  g.rm = g.none ? 0.0f : __builtin_amdgcn_rsqf(g.v);
  g.m = g.v * g.rm;
  g.gx = g.si * x;
  // A token without a step adds nothing, whatever x holds.
  g.b = g.none ? 0.0f : g.m * g.gx;
  return g;
}

// One lane a channel, one token after another.
__global__ __launch_bounds__(64) void recur_fwd_kernel(RecurArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (c >= a.C) return;
  const float rate = decay_rate(a, c);
  float h = 0.0f;
  int32_t t = 0;
  for (int32_t d = 0; d < a.num_docs; ++d) {
    const int32_t end = min(a.cu[d + 1], a.S);
    const int64_t slot = a.state ? slot_of(a.index, d, a.slots) : -1;
    const bool go_on = slot >= 0 && a.resume && a.resume[d];
    h = go_on ? a.state[slot * a.C + c] : 0.0f;
    for (; t < end; ++t) {
      const Gates g = gates(rate, bf16_f32(a.x[t * a.xs + c]), bf16_f32(a.r[t * a.rs + c]),
                            bf16_f32(a.i[t * a.is + c]));
      if (a.keep && t % kRecurKeep == 0) a.keep[(int64_t)(t / kRecurKeep) * a.C + c] = h;
      h = __builtin_fmaf(g.a, h, g.b);
      float y = h;
      if (a.z) {
        const float z = bf16_f32(a.z[t * a.zs + c]);
        y = h * (z * sigmoid_f32(z));
      }
      a.y[(int64_t)t * a.C + c] = bf16_of(y);
    }
    if (slot >= 0) a.state[slot * a.C + c] = h;
  }
}

__global__ __launch_bounds__(64) void recur_bwd_kernel(RecurArgs a) {
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (c >= a.C) return;
  const float decay = param_at(a.decay, a.decay_bf16, c), rate = decay_rate(a, c);
  float l = 0.0f;  // what the tokens behind send to this one
  double sum = 0.0;
  int32_t d = a.num_docs;  // the document of the token at hand begins at cu[d] or before
  for (int32_t k = (a.S + kRecurKeep - 1) / kRecurKeep - 1; k >= 0; --k) {
    const int32_t t0 = k * kRecurKeep, t1 = min(a.S, t0 + kRecurKeep);
    float h = a.keep[(int64_t)k * a.C + c];
    int32_t e = d;
    while (e > 0 && a.cu[e] > t0) --e;  // the last that begins at t0 or before
    for (int32_t t = t0; t < t1; ++t) {
      bool first = a.cu[e] == t;
      while (e < a.num_docs && a.cu[e + 1] <= t) ++e, first = true;
      if (first) h = 0.0f;
      a.h[(int64_t)(t - t0) * a.C + c] = h;
      const Gates g = gates(rate, bf16_f32(a.x[t * a.xs + c]), bf16_f32(a.r[t * a.rs + c]),
                            bf16_f32(a.i[t * a.is + c]));
      h = __builtin_fmaf(g.a, h, g.b);
    }
    for (int32_t t = t1 - 1; t >= t0; --t) {
      const float x = bf16_f32(a.x[t * a.xs + c]);
      const Gates g = gates(rate, x, bf16_f32(a.r[t * a.rs + c]), bf16_f32(a.i[t * a.is + c]));
      const float before = a.h[(int64_t)(t - t0) * a.C + c], dy = bf16_f32(a.dy[t * a.dys + c]);
      float own = dy;
      const int64_t at = (int64_t)t * a.C + c;
      if (a.z) {
        const float z = bf16_f32(a.z[t * a.zs + c]), s = sigmoid_f32(z);
        own = dy * (z * s);
        a.dz[at] = bf16_of(dy * __builtin_fmaf(g.a, before, g.b) * dsilu_f32(z, s));
      }
      while (d > 0 && a.cu[d] > t + 1) --d;
      l = a.cu[d] == t + 1 ? own : l + own;
      const float lm = l * g.m, half = 0.5f * g.u;
      a.dx[at] = bf16_of(lm * g.si);
      a.di[at] = bf16_of(g.none ? 0.0f : lm * g.gx * (1.0f - g.si));
      const float own_part = g.none ? 0.0f : g.gx * (g.a * g.a) * (half * g.rm);
      const float E = l * __builtin_fmaf(-half * g.a, before, own_part);
      a.dr[at] = bf16_of(E * (1.0f - g.sr));
      sum += E;
      l *= g.a;
    }
  }
  const float soft = softplus_f32(decay);
  const float ratio = soft > 0.0f ? sigmoid_f32(decay) / soft : 1.0f;
  param_put(a.ddecay, a.decay_bf16, c, ratio * (float)sum);
}

__global__ __launch_bounds__(64) void recur_step_kernel(RecurArgs a) {
  const int64_t blocks = (a.C + 63) / 64, row = blockIdx.x / blocks;
  const int64_t c = (blockIdx.x - row * blocks) * 64 + threadIdx.x;
  const int64_t slot = slot_of(a.index, row, a.slots);
  if (c >= a.C) return;
  float y = 0.0f;
  if (slot >= 0) {
    const Gates g = gates(decay_rate(a, c), bf16_f32(a.x[row * a.xs + c]), bf16_f32(a.r[row * a.rs + c]),
                          bf16_f32(a.i[row * a.is + c]));
    float* p = a.state + slot * a.C + c;
    y = __builtin_fmaf(g.a, *p, g.b);
    *p = y;
    if (a.z) {
      const float z = bf16_f32(a.z[row * a.zs + c]);
      y *= z * sigmoid_f32(z);
    }
  }
  a.y[row * a.C + c] = bf16_of(y);
}

}  // namespace

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_fwd_kernel, dim3((uint32_t)((a.C + 63) / 64)), dim3(64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_bwd_kernel, dim3((uint32_t)((a.C + 63) / 64)), dim3(64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_recur_step(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_step_kernel, dim3((uint32_t)((int64_t)a.S * ((a.C + 63) / 64))), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
