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
//
// All of it is bound by HBM: a token's group is read once and stays in
// registers over its sums.  A team of lanes has a group; the mean is taken
// first and the squares of the differences from it after, both in FP32.
// 16384 tokens, C = 4096 in 32 groups, with a gate: forward 73 us (5.5 TB/s),
// backward 120 (5.6 TB/s) and 5 for the sums over its partial rows.

#include "vdc_ssm.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

// ------------------------------------------------------ groups in registers --
//
// Groups of a multiple of 8 channels on rows aligned to 16 bytes: L lanes a
// group (within a wave, or 256: a whole workgroup), K vectors of 8 channels a
// lane.  A workgroup keeps its channels and takes tokens one after another,
// the next one's vectors requested before the current is computed; within a
// wave, the four waves of a workgroup have the same channels and different
// tokens.

constexpr int kThreads = 256;

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
__device__ __forceinline__ u32x4_t load8(const uint16_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }
__device__ __forceinline__ void store8(uint16_t* p, u32x4_t v) {
  // Every output byte is written once and not read here.
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
}

template <int L, int K>
struct Place {
  static constexpr bool kWide = L > 64;            // a workgroup has one group
  static constexpr int kTokens = kWide ? 1 : 4;    // tokens a workgroup has at a time
  static constexpr int kGroups = kWide ? 1 : 64 / L;
  int64_t token, step, c0;  // first token, tokens between two of its turns, first channel
  int32_t li;               // lane of the team
  bool active;
  __device__ __forceinline__ Place(const NormArgs& a, int32_t rows) {
    const int32_t sets = (a.G + kGroups - 1) / kGroups;
    const int32_t rb = blockIdx.x / sets, set = blockIdx.x - rb * sets;
    const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
    const int32_t g = kWide ? set : set * kGroups + lane / L;
    li = kWide ? (int32_t)threadIdx.x : lane % L;
    active = g < a.G;
    c0 = (int64_t)(active ? g : 0) * a.per;
    token = (int64_t)rb * kTokens + (kWide ? 0 : wave);
    step = (int64_t)rows * kTokens;
  }
  // Channel of vector k within the group, and whether it is one.
  __device__ __forceinline__ int32_t at(int k) const { return (k * L + li) * 8; }
  __device__ __forceinline__ bool has(const NormArgs& a, int k) const { return active && at(k) < a.per; }
};

// Sum over a team; `lds` has four floats for each call between barriers.
template <int L>
__device__ __forceinline__ float team_sum(float v, float* lds) {
  if constexpr (L <= 64) {
    return lanes_sum<L>(v);
  } else {
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
}

template <int K>
struct Affine {
  Vec8 w[K], b[K];
  template <int L>
  __device__ __forceinline__ void load(const NormArgs& a, const Place<L, K>& p) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = p.c0 + p.at(k) + i;
        w[k].v[i] = p.has(a, k) ? param_at(a.w, a.w_bf16, c) : 0.0f;
        b[k].v[i] = p.has(a, k) && a.b ? param_at(a.b, a.b_bf16, c) : 0.0f;
      }
  }
};

template <int L, int K>
__device__ __forceinline__ void request(const NormArgs& a, const Place<L, K>& p, const uint16_t* t,
                                        int64_t stride, int64_t token, u32x4_t (&r)[K]) {
  const int64_t row = token < a.S ? token : a.S - 1;
#pragma unroll
  for (int k = 0; k < K; ++k)
    r[k] = p.has(a, k) ? load8(t + row * stride + p.c0 + p.at(k)) : (u32x4_t){0u, 0u, 0u, 0u};
}

// Differences from the mean, and 1 / sqrt(var + eps).
template <int L, int K>
__device__ __forceinline__ float centre(const NormArgs& a, const Place<L, K>& p, const u32x4_t (&r)[K],
                                        Vec8 (&d)[K], float* lds) {
  const float inv = 1.0f / (float)a.per;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    d[k] = unpack8(r[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) s += d[k].v[i];
  }
  const float mean = team_sum<L>(s, lds) * inv;
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[k].v[i] = p.has(a, k) ? d[k].v[i] - mean : 0.0f;
      q = __builtin_fmaf(d[k].v[i], d[k].v[i], q);
    }
  return 1.0f / __builtin_sqrtf(team_sum<L>(q, lds + 4) * inv + a.eps);
}

template <int L, int K, bool kGate>
__global__ __launch_bounds__(kThreads) void norm_fwd_kernel(NormArgs a, int32_t rows) {
  __shared__ float lds[2][8];
  const Place<L, K> p(a, rows);
  Affine<K> f;
  f.load(a, p);
  u32x4_t x[K], z[K];
  request(a, p, a.x, a.xs, p.token, x);
  if (kGate) request(a, p, a.z, a.zs, p.token, z);
  int turn = 0;
#pragma unroll 1
  for (int64_t t = p.token; t < a.S; t += p.step, turn ^= 1) {
    u32x4_t xc[K], zc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) xc[k] = x[k], zc[k] = kGate ? z[k] : x[k];
    request(a, p, a.x, a.xs, t + p.step, x);
    if (kGate) request(a, p, a.z, a.zs, t + p.step, z);
    Vec8 d[K];
    const float rstd = centre(a, p, xc, d, lds[turn]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Vec8 zk = unpack8(zc[k]);
      Vec8 y;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = __builtin_fmaf(d[k].v[i] * rstd, f.w[k].v[i], f.b[k].v[i]);
        y.v[i] = kGate ? v * (zk.v[i] * sigmoid_f32(zk.v[i])) : v * sigmoid_f32(v);
      }
      if (p.has(a, k)) store8(a.y + t * a.C + p.c0 + p.at(k), pack8(y));
    }
  }
}

template <int L, int K, bool kGate>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs a, int32_t rows) {
  typedef Place<L, K> P;
  __shared__ float lds[2][16];
  __shared__ float sums[P::kWide ? 1 : 3][P::kWide ? 1 : 2 * K * 8][64];
  const P p(a, rows);
  const float inv = 1.0f / (float)a.per;
  Affine<K> f;
  f.load(a, p);
  Vec8 dw[K], db[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k].v[i] = db[k].v[i] = 0.0f;
  u32x4_t x[K], z[K], dy[K];
  request(a, p, a.x, a.xs, p.token, x);
  request(a, p, a.dy, a.dys, p.token, dy);
  if (kGate) request(a, p, a.z, a.zs, p.token, z);
  int turn = 0;
#pragma unroll 1
  for (int64_t t = p.token; t < a.S; t += p.step, turn ^= 1) {
    u32x4_t xc[K], zc[K], dc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) xc[k] = x[k], dc[k] = dy[k], zc[k] = kGate ? z[k] : x[k];
    request(a, p, a.x, a.xs, t + p.step, x);
    request(a, p, a.dy, a.dys, t + p.step, dy);
    if (kGate) request(a, p, a.z, a.zs, t + p.step, z);
    Vec8 d[K], q[K];
    const float rstd = centre(a, p, xc, d, lds[turn]);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Vec8 zk = unpack8(zc[k]), dyk = unpack8(dc[k]);
      Vec8 dz;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = d[k].v[i] * rstd;
        const float v = __builtin_fmaf(xh, f.w[k].v[i], f.b[k].v[i]);
        const float u = kGate ? zk.v[i] : v, s = sigmoid_f32(u);
        const float dv = dyk.v[i] * (kGate ? u * s : dsilu_f32(u, s));
        if (kGate) dz.v[i] = dyk.v[i] * v * dsilu_f32(u, s);
        dw[k].v[i] = __builtin_fmaf(dv, xh, dw[k].v[i]);
        db[k].v[i] += dv;
        d[k].v[i] = xh;
        q[k].v[i] = dv * f.w[k].v[i];
        s1 += q[k].v[i];
        s2 = __builtin_fmaf(q[k].v[i], xh, s2);
      }
      if (kGate && p.has(a, k)) store8(a.dz + t * a.C + p.c0 + p.at(k), pack8(dz));
    }
    s1 = team_sum<L>(s1, lds[turn] + 8) * inv;
    s2 = team_sum<L>(s2, lds[turn] + 12) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = rstd * __builtin_fmaf(-d[k].v[i], s2, q[k].v[i] - s1);
      if (p.has(a, k)) store8(a.dx + t * a.C + p.c0 + p.at(k), pack8(o));
    }
  }
  // The workgroup's partial row: its waves' sums in order.
  if (!P::kWide) {
    const int32_t wave = threadIdx.x / 64, lane = threadIdx.x & 63;
    if (wave > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[wave - 1][k * 8 + i][lane] = dw[k].v[i];
          sums[wave - 1][(K + k) * 8 + i][lane] = db[k].v[i];
        }
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[k].v[i] += sums[o][k * 8 + i][lane];
          db[k].v[i] += sums[o][(K + k) * 8 + i][lane];
        }
  }
  const int32_t sets = (a.G + P::kGroups - 1) / P::kGroups;
  float* part = a.part + (int64_t)(blockIdx.x / sets) * 2 * a.C + p.c0;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p.has(a, k)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        part[p.at(k) + i] = dw[k].v[i];
        part[a.C + p.at(k) + i] = db[k].v[i];
      }
    }
}

// ------------------------------------------------- any group, any alignment --
//
// A wave has one group of a token and goes over it three times, from L2 after
// the first.

struct Stats {
  float mean, rstd;
};

__device__ __forceinline__ Stats stats_of(const NormArgs& a, const uint16_t* x) {
  const int lane = threadIdx.x & 63;
  float s = 0.0f;
  for (int i = lane; i < a.per; i += 64) s += bf16_f32(x[i]);
  const float mean = lanes_sum<64>(s) / (float)a.per;
  float q = 0.0f;
  for (int i = lane; i < a.per; i += 64) {
    const float d = bf16_f32(x[i]) - mean;
    q = __builtin_fmaf(d, d, q);
  }
  return Stats{mean, 1.0f / __builtin_sqrtf(lanes_sum<64>(q) / (float)a.per + a.eps)};
}

__global__ __launch_bounds__(256) void norm_fwd_any_kernel(NormArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t e = (int64_t)blockIdx.x * 4 + threadIdx.x / 64; e < a.S * a.G; e += step) {
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
}

// A wave takes one group of every prows-th token and keeps its sums for dw
// and db in its own partial row.
__global__ __launch_bounds__(64) void norm_bwd_any_kernel(NormArgs a) {
  const int64_t row = blockIdx.x / a.G, c0 = (blockIdx.x - row * a.G) * (int64_t)a.per;
  const int lane = threadIdx.x;
  float* pw = a.part + row * 2 * a.C + c0;
  float* pb = pw + a.C;
  for (int i = lane; i < a.per; i += 64) pw[i] = pb[i] = 0.0f;
  const float inv = 1.0f / (float)a.per;
  for (int64_t t = row; t < a.S; t += a.prows) {
    const uint16_t* x = a.x + t * a.xs + c0;
    const Stats st = stats_of(a, x);
    // Channel i's xhat, and w times its dv.
    auto terms = [&](int i, float& xh, float& v, float& u, float& s, float& dy, float& dv) {
      xh = (bf16_f32(x[i]) - st.mean) * st.rstd;
      v = __builtin_fmaf(xh, param_at(a.w, a.w_bf16, c0 + i), a.b ? param_at(a.b, a.b_bf16, c0 + i) : 0.0f);
      dy = bf16_f32(a.dy[t * a.dys + c0 + i]);
      u = a.z ? bf16_f32(a.z[t * a.zs + c0 + i]) : v;
      s = sigmoid_f32(u);
      dv = dy * (a.z ? u * s : dsilu_f32(u, s));
      return dv * param_at(a.w, a.w_bf16, c0 + i);
    };
    float xh, v, u, s, dy, dv, s1 = 0.0f, s2 = 0.0f;
    for (int i = lane; i < a.per; i += 64) {
      const float q = terms(i, xh, v, u, s, dy, dv);
      if (a.z) a.dz[t * a.C + c0 + i] = bf16_of(dy * v * dsilu_f32(u, s));
      pw[i] = __builtin_fmaf(dv, xh, pw[i]);
      pb[i] += dv;
      s1 += q;
      s2 = __builtin_fmaf(q, xh, s2);
    }
    s1 = lanes_sum<64>(s1) * inv;
    s2 = lanes_sum<64>(s2) * inv;
    for (int i = lane; i < a.per; i += 64) {
      const float q = terms(i, xh, v, u, s, dy, dv);
      a.dx[t * a.C + c0 + i] = bf16_of(st.rstd * __builtin_fmaf(-xh, s2, q - s1));
    }
  }
}

// The partial rows of dw and db in order, summed in FP64, 16 loads at once.
__global__ __launch_bounds__(64) void norm_bwd_sum_kernel(NormArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (i >= 2 * a.C) return;
  double s = 0.0;
  int32_t r = 0;
  for (; r + 16 <= a.prows; r += 16) {
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = a.part[(int64_t)(r + j) * 2 * a.C + i];
#pragma unroll
    for (int j = 0; j < 16; ++j) s += v[j];
  }
  for (; r < a.prows; ++r) s += a.part[(int64_t)r * 2 * a.C + i];
  if (i < a.C) param_put(a.dw, a.w_bf16, i, (float)s);
  else if (a.db) param_put(a.db, a.b_bf16, i - a.C, (float)s);
}

// ------------------------------------------------------------------ launch --

bool vectors(const uint16_t* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

// Whether the groups go to registers: whole vectors on aligned rows, at most
// 4 a lane of a workgroup (8 would spill the backward's sums).
bool in_registers(const NormArgs& a) {
  return a.per % 8 == 0 && a.per <= kThreads * 8 * 4 && a.C % 8 == 0 && vectors(a.x, a.xs) &&
         (!a.z || vectors(a.z, a.zs)) && (!a.dy || vectors(a.dy, a.dys)) &&
         vectors(a.y, 8) && vectors(a.dx, 8) && vectors(a.dz, 8);
}

// Lanes of a team and vectors of a lane for groups of `per` channels; one
// vector a lane as long as that leaves a wave or less, then two, then a
// workgroup.
struct Shape {
  int lanes, vecs;
};
Shape shape_of(int64_t per) {
  const int64_t n = (per + 7) / 8;
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  return {256, n <= 512 ? 2 : 4};
}

template <int L, int K>
void launch_vec(const NormArgs& a, bool back, hipStream_t s) {
  const int64_t sets = (a.G + Place<L, K>::kGroups - 1) / Place<L, K>::kGroups;
  const int64_t turns = (a.S + Place<L, K>::kTokens - 1) / Place<L, K>::kTokens;
  int64_t rows = back ? a.prows : turns;
  if (!back) rows = rows * sets > 4096 ? (4096 + sets - 1) / sets : rows;
  const dim3 grid((uint32_t)(rows * sets)), block(kThreads);
  if (back) {
    if (a.z) hipLaunchKernelGGL((norm_bwd_kernel<L, K, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((norm_bwd_kernel<L, K, false>), grid, block, 0, s, a, (int32_t)rows);
  } else {
    if (a.z) hipLaunchKernelGGL((norm_fwd_kernel<L, K, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((norm_fwd_kernel<L, K, false>), grid, block, 0, s, a, (int32_t)rows);
  }
}

void launch_shape(const NormArgs& a, bool back, hipStream_t s) {
  const Shape h = shape_of(a.per);
  if (h.lanes == 8) launch_vec<8, 1>(a, back, s);
  else if (h.lanes == 16) launch_vec<16, 1>(a, back, s);
  else if (h.lanes == 32) launch_vec<32, 1>(a, back, s);
  else if (h.lanes == 64 && h.vecs == 1) launch_vec<64, 1>(a, back, s);
  else if (h.lanes == 64) launch_vec<64, 2>(a, back, s);
  else if (h.vecs == 2) launch_vec<256, 2>(a, back, s);
  else launch_vec<256, 4>(a, back, s);
}

}  // namespace

// Partial rows of the backward: about 1024 workgroups, four on each CU, by
// the shape that aligned rows take.
int norm_bwd_rows(int64_t S, int64_t C, int64_t G) {
  const Shape h = shape_of(C / G);
  const int64_t groups = h.lanes > 64 ? 1 : 64 / h.lanes, tokens = h.lanes > 64 ? 1 : 4;
  const int64_t sets = (G + groups - 1) / groups, turns = (S + tokens - 1) / tokens;
  const int64_t want = (1024 + sets - 1) / sets;
  return (int)(turns < want ? turns : want);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) {
  if (in_registers(a)) launch_shape(a, false, s);
  else {
    const int64_t blocks = (a.S * a.G + 3) / 4;
    hipLaunchKernelGGL(norm_fwd_any_kernel, dim3((uint32_t)(blocks < 65536 ? blocks : 65536)), dim3(256), 0,
                       s, a);
  }
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  if (in_registers(a)) launch_shape(a, true, s);
  else hipLaunchKernelGGL(norm_bwd_any_kernel, dim3((uint32_t)((int64_t)a.prows * a.G)), dim3(64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd_sum(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((uint32_t)((2 * a.C + 63) / 64)), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
