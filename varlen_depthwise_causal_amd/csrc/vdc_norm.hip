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

// L lanes have a group (within a wave, or a whole workgroup of 256 or 512), K
// vectors of 8 channels a lane.  A workgroup keeps its channels and takes tokens
// one after another, the next one's vectors requested before the current is
// computed; within a wave, the four waves of a workgroup have the same channels
// and different tokens.  kWhole: groups of a multiple of 8 channels on rows
// aligned to 16 bytes; others end in a part of a vector and are read at any
// address.  16384 tokens, C = 520 in 8 groups, with a gate: forward 27 us,
// backward 49; three times over a row with a channel a lane takes 54 and 190.

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

template <int L, int K, bool kWhole>
struct Place {
  static constexpr int kThreads = L > 64 ? L : 256;
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
  __device__ __forceinline__ int32_t count(const NormArgs& a, int k) const { return a.per - at(k); }
  __device__ __forceinline__ bool has(const NormArgs& a, int k, int i) const {
    return active && at(k) + (kWhole ? 0 : i) < a.per;
  }
};

// Sum over a team; `lds` has a float a wave for each call between barriers.
template <int L>
__device__ __forceinline__ float team_sum(float v, float* lds) {
  if constexpr (L <= 64) {
    return lanes_sum<L>(v);
  } else {
    v = lanes_sum<64>(v);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x / 64] = v;
    __syncthreads();
    const float four = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    return L == 256 ? four : four + ((lds[4] + lds[5]) + (lds[6] + lds[7]));
  }
}

template <int K>
struct Affine {
  Vec8 w[K], b[K];
  template <class P>
  __device__ __forceinline__ void load(const NormArgs& a, const P& p) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t c = p.c0 + p.at(k) + i;
        w[k].v[i] = p.has(a, k, i) ? param_at(a.w, a.w_bf16, c) : 0.0f;
        b[k].v[i] = p.has(a, k, i) && a.b ? param_at(a.b, a.b_bf16, c) : 0.0f;
      }
  }
};

template <int L, int K, bool kWhole>
__device__ __forceinline__ void request(const NormArgs& a, const Place<L, K, kWhole>& p, const uint16_t* t,
                                        int64_t stride, int64_t token, u32x4_t (&r)[K]) {
  const int64_t row = token < a.S ? token : a.S - 1;
#pragma unroll
  for (int k = 0; k < K; ++k)
    r[k] = p.has(a, k) ? load8<kWhole>(t + row * stride + p.c0 + p.at(k), p.count(a, k)) : (u32x4_t){0u, 0u, 0u, 0u};
}

// Differences from the mean, and 1 / sqrt(var + eps).
template <int L, int K, bool kWhole>
__device__ __forceinline__ float centre(const NormArgs& a, const Place<L, K, kWhole>& p, const u32x4_t (&r)[K],
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
      d[k].v[i] = p.has(a, k, i) ? d[k].v[i] - mean : 0.0f;
      q = __builtin_fmaf(d[k].v[i], d[k].v[i], q);
    }
  return 1.0f / __builtin_sqrtf(team_sum<L>(q, lds + 8) * inv + a.eps);
}

template <int L, int K, bool kWhole, bool kGate>
__global__ __launch_bounds__(L > 64 ? L : 256) void norm_fwd_kernel(NormArgs a, int32_t rows) {
  __shared__ float lds[2][16];
  const Place<L, K, kWhole> p(a, rows);
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
      if (p.has(a, k)) store8<kWhole>(a.y + t * a.C + p.c0 + p.at(k), pack8(y), p.count(a, k));
    }
  }
}

template <int L, int K, bool kWhole, bool kGate>
__global__ __launch_bounds__(L > 64 ? L : 256) void norm_bwd_kernel(NormArgs a, int32_t rows) {
  typedef Place<L, K, kWhole> P;
  __shared__ float lds[2][32];
  __shared__ float sums[P::kWide ? 1 : 3][P::kWide ? 1 : 2 * K * 8][64];
  const P p(a, rows);
  const float inv = 1.0f / (float)a.per;
  // Eight waves a workgroup, two a SIMD, have no registers for the next token.
  // Even so some go to scratch memory: 32 with a gate on aligned rows, on others
  // 79 with one and 31 without.  4096 tokens of one group of 16384 channels with
  // a gate, aligned: 400 us, against 3360 by going over each row three times.
  constexpr bool kAhead = L <= 256;
  Affine<K> f;
  f.load(a, p);
  Vec8 dw[K], db[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k].v[i] = db[k].v[i] = 0.0f;
  u32x4_t x[K], z[K], dy[K];
  auto fetch = [&](int64_t t) {
    request(a, p, a.x, a.xs, t, x);
    request(a, p, a.dy, a.dys, t, dy);
    if (kGate) request(a, p, a.z, a.zs, t, z);
  };
  if (kAhead) fetch(p.token);
  int turn = 0;
#pragma unroll 1
  for (int64_t t = p.token; t < a.S; t += p.step, turn ^= 1) {
    if (!kAhead) fetch(t);
    u32x4_t xc[K], zc[K], dc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) xc[k] = x[k], dc[k] = dy[k], zc[k] = kGate ? z[k] : x[k];
    if (kAhead) fetch(t + p.step);
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
      if (kGate && p.has(a, k)) store8<kWhole>(a.dz + t * a.C + p.c0 + p.at(k), pack8(dz), p.count(a, k));
    }
    s1 = team_sum<L>(s1, lds[turn] + 16) * inv;
    s2 = team_sum<L>(s2, lds[turn] + 24) * inv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = rstd * __builtin_fmaf(-d[k].v[i], s2, q[k].v[i] - s1);
      if (p.has(a, k)) store8<kWhole>(a.dx + t * a.C + p.c0 + p.at(k), pack8(o), p.count(a, k));
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
      for (int i = 0; i < 8; ++i)
        if (p.has(a, k, i)) {
          part[p.at(k) + i] = dw[k].v[i];
          part[a.C + p.at(k) + i] = db[k].v[i];
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

// Whether all vectors are whole and aligned (kWhole above).
bool whole(const NormArgs& a) {
  return a.per % 8 == 0 && a.C % 8 == 0 && vectors(a.x, a.xs) && (!a.z || vectors(a.z, a.zs)) &&
         (!a.dy || vectors(a.dy, a.dys)) && vectors(a.y, 8) && vectors(a.dx, 8) && vectors(a.dz, 8);
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
  if (n <= 1024) return {256, n <= 512 ? 2 : 4};
  return {512, 4};  // eight vectors a lane of 256 would spill the backward's sums
}

template <int L, int K, bool kWhole>
void launch_vec(const NormArgs& a, bool back, hipStream_t s) {
  typedef Place<L, K, kWhole> P;
  const int64_t sets = (a.G + P::kGroups - 1) / P::kGroups;
  const int64_t turns = (a.S + P::kTokens - 1) / P::kTokens;
  int64_t rows = back ? a.prows : turns;
  // A workgroup reads its weights once: the larger they are, the more tokens it
  // takes.  Forward, one group of 16384 channels, 4096 tokens: 512 workgroups 97
  // us, 4096 282; of 4096 channels, 8192 tokens: 1024 41 us, 4096 69.
  const int64_t most = L <= 64 ? 4096 : K == 2 ? 1024 : 512;
  if (!back) rows = rows * sets > most ? (most + sets - 1) / sets : rows;
  const dim3 grid((uint32_t)(rows * sets)), block(P::kThreads);
  if (back) {
    if (a.z) hipLaunchKernelGGL((norm_bwd_kernel<L, K, kWhole, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((norm_bwd_kernel<L, K, kWhole, false>), grid, block, 0, s, a, (int32_t)rows);
  } else {
    if (a.z) hipLaunchKernelGGL((norm_fwd_kernel<L, K, kWhole, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((norm_fwd_kernel<L, K, kWhole, false>), grid, block, 0, s, a, (int32_t)rows);
  }
}

template <bool kWhole>
void launch_shape(const NormArgs& a, bool back, hipStream_t s) {
  const Shape h = shape_of(a.per);
  if (h.lanes == 8) launch_vec<8, 1, kWhole>(a, back, s);
  else if (h.lanes == 16) launch_vec<16, 1, kWhole>(a, back, s);
  else if (h.lanes == 32) launch_vec<32, 1, kWhole>(a, back, s);
  else if (h.lanes == 64 && h.vecs == 1) launch_vec<64, 1, kWhole>(a, back, s);
  else if (h.lanes == 64) launch_vec<64, 2, kWhole>(a, back, s);
  else if (h.lanes == 256 && h.vecs == 2) launch_vec<256, 2, kWhole>(a, back, s);
  else if (h.lanes == 256) launch_vec<256, 4, kWhole>(a, back, s);
  else launch_vec<512, 4, kWhole>(a, back, s);
}

hipError_t launch(const NormArgs& a, bool back, hipStream_t s) {
  if (whole(a)) launch_shape<true>(a, back, s);
  else launch_shape<false>(a, back, s);
  return hipGetLastError();
}

}  // namespace

int norm_bwd_rows(int64_t S, int64_t C, int64_t G) {
  const Shape h = shape_of(C / G);
  const int64_t groups = h.lanes > 64 ? 1 : 64 / h.lanes, tokens = h.lanes > 64 ? 1 : 4;
  const int64_t sets = (G + groups - 1) / groups, turns = (S + tokens - 1) / tokens;
  const int64_t want = (1024 + sets - 1) / sets;
  return (int)(turns < want ? turns : want);
}

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s) { return launch(a, false, s); }
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) { return launch(a, true, s); }

hipError_t launch_norm_bwd_sum(const NormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_bwd_sum_kernel, dim3((uint32_t)((2 * a.C + 63) / 64)), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
