// Layer norm of each token's channels on a residual stream, forward and
// backward.  For one token of C channels:
//
//   s = bf16(x + residual),  or x
//   xhat = (s - mean) rstd,  rstd = 1 / sqrt(mean((s - mean)^2) + eps)
//   y = w xhat + b
//
//   q = w dy,   dx = rstd (q - mean(q) - xhat mean(q xhat)) + dstream
//   dw = sum_t dy xhat,   db = sum_t dy
//
// All of it is bound by HBM: a token is read once and stays in registers over
// its sums.  A team of lanes has a token: part of a wave, a wave, or a workgroup,
// whose waves take their own means first and exchange their sums once: with m_w
// the mean of wave w's n_w channels,
//
//   sum (s - mean)^2     = sum_w [ sum (s - m_w)^2 + n_w (m_w - mean)^2 ]
//   sum q (s - mean)     = sum_w [ sum q (s - m_w) + (m_w - mean) sum q ]
//
// which cancels no more than the sums about the mean themselves.
//
// Measured, with a residual: 16384 tokens, C = 4096 forward 92 us, 5.8 TB/s, backward 105,
// 5.1 TB/s (a copy: 5.1), and the sum of its partial rows 5.8; 8192 tokens, C = 8192
// forward 79 us, 6.8 TB/s, the last cache's part in it.  Few tokens are latency: 33 tokens,
// C = 520 3.6 us; 1543 tokens of 1001 channels 5.0 forward, 8.6 and 4.6 backward.

#include <algorithm>

#include "vdc_layer.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

// L lanes have a token (L > 64: a workgroup of L), K vectors of 8 channels a lane.
// kWhole: rows of a multiple of 8 channels, aligned to 16 bytes; others end in a
// part of a vector and are read at any address.
template <int L, int K, bool kWhole>
struct Team {
  static constexpr bool kWide = L > 64;
  static constexpr int kThreads = kWide ? L : 256;
  static constexpr int kTokens = kWide ? 1 : 256 / L;  // tokens a workgroup has at a time
  static constexpr int kWaves = kWide ? L / 64 : 1;    // waves of a team
  static constexpr int kUnroll = kWaves > 8 ? 2 : kWaves;  // of loops over them: registers
  int32_t li, wave;  // lane and wave of the team
  int64_t token, step;
  float inv_own;  // 1 / channels of the wave
  float own;      // channels of the wave
  __device__ __forceinline__ Team(const LayerNormArgs& a, int32_t rows) {
    li = kWide ? (int32_t)threadIdx.x : (int32_t)threadIdx.x % L;
    wave = kWide ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64u) : 0;
    token = (int64_t)blockIdx.x * kTokens + (kWide ? 0 : threadIdx.x / L);
    step = (int64_t)rows * kTokens;
    own = (float)channels(a, wave);
    inv_own = own > 0.0f ? 1.0f / own : 0.0f;
  }
  // Channels of wave w.
  static __device__ __forceinline__ int32_t channels(const LayerNormArgs& a, int32_t w) {
    int32_t n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) n += min(max(a.C - (k * L + w * 64) * 8, 0), (kWide ? 64 : L) * 8);
    return n;
  }
  __device__ __forceinline__ int32_t at(int k) const { return (k * L + li) * 8; }
  __device__ __forceinline__ bool has(const LayerNormArgs& a, int k) const { return at(k) < a.C; }
  __device__ __forceinline__ int32_t count(const LayerNormArgs& a, int k) const { return a.C - at(k); }
  __device__ __forceinline__ bool has(const LayerNormArgs& a, int k, int i) const {
    return at(k) + (kWhole ? 0 : i) < a.C;
  }
};

template <int L, int K, bool kWhole>
__device__ __forceinline__ void request(const LayerNormArgs& a, const Team<L, K, kWhole>& p, const uint16_t* t,
                                        int64_t stride, int64_t token, u32x4_t (&r)[K]) {
  const int64_t row = token < a.S ? token : a.S - 1;
#pragma unroll
  for (int k = 0; k < K; ++k)
    r[k] = p.has(a, k) ? load8<kWhole>(t + row * stride + p.at(k), p.count(a, k)) : (u32x4_t){0u, 0u, 0u, 0u};
}

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

// A lane's channels of a parameter, by vectors but for a part of one; zeros without
// the parameter and past the last channel.
template <int K, class P>
__device__ __forceinline__ void params(const LayerNormArgs& a, const P& p, const void* t, int bf16, Vec8 (&o)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[k].v[i] = 0.0f;
    if (!t || !p.has(a, k)) continue;
    if (bf16) {
      o[k] = unpack8(load8<false>(static_cast<const uint16_t*>(t) + p.at(k), p.count(a, k)));
    } else if (p.count(a, k) >= 8) {
      const f32x4_any* q = reinterpret_cast<const f32x4_any*>(static_cast<const float*>(t) + p.at(k));
      const f32x4_any lo = q[0], hi = q[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[k].v[i] = lo[i], o[k].v[4 + i] = hi[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (p.at(k) + i < a.C) o[k].v[i] = static_cast<const float*>(t)[p.at(k) + i];
    }
  }
}

// d = s - m_w, the differences from the wave's own mean m_w; returns m_w and the
// sum of d^2.
template <int L, int K, bool kWhole>
__device__ __forceinline__ void centre(const LayerNormArgs& a, const Team<L, K, kWhole>& p, Vec8 (&d)[K], float* mean,
                                       float* square) {
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += d[k].v[i];
  *mean = lanes_sum<L < 64 ? L : 64>(s) * p.inv_own;
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[k].v[i] = p.has(a, k, i) ? d[k].v[i] - *mean : 0.0f;
      q = __builtin_fmaf(d[k].v[i], d[k].v[i], q);
    }
  *square = lanes_sum<L < 64 ? L : 64>(q);
}

// The row's mean and 1 / sqrt(var + eps) from the waves' means and squares in lds.
template <class P>
__device__ __forceinline__ void join(const LayerNormArgs& a, const float (*lds)[4], float* mean, float* rstd) {
  const float inv = 1.0f / (float)a.C;
  float s = 0.0f, q = 0.0f;
#pragma unroll P::kUnroll
  for (int w = 0; w < P::kWaves; ++w) s = __builtin_fmaf((float)P::channels(a, w), lds[w][0], s);
  *mean = s * inv;
#pragma unroll P::kUnroll
  for (int w = 0; w < P::kWaves; ++w) {
    const float off = lds[w][0] - *mean;
    q += __builtin_fmaf((float)P::channels(a, w) * off, off, lds[w][1]);
  }
  *rstd = 1.0f / __builtin_sqrtf(q * inv + a.eps);
}

template <int L, int K, bool kWhole, bool kRes>
__global__ __launch_bounds__(L > 64 ? L : 256) void layer_norm_fwd_kernel(LayerNormArgs a, int32_t rows) {
  typedef Team<L, K, kWhole> P;
  __shared__ float lds[2][P::kWaves][4];
  const P p(a, rows);
  Vec8 w[K], b[K];
  params<K>(a, p, a.w, a.w_bf16, w);
  params<K>(a, p, a.b, a.b_bf16, b);
  u32x4_t x[K], res[K];
  request(a, p, a.x, a.xs, p.token, x);
  if (kRes) request(a, p, a.res, a.ress, p.token, res);
  int turn = 0;
#pragma unroll 1
  for (int64_t t = p.token; t < a.S; t += p.step, turn ^= 1) {
    Vec8 d[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      u32x4_t s = x[k];
      d[k] = unpack8(s);
      if (kRes) {
        const Vec8 rk = unpack8(res[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[k].v[i] += rk.v[i];
        s = pack8(d[k]);
        d[k] = unpack8(s);
        if (p.has(a, k)) store8<kWhole>(a.stream + t * a.C + p.at(k), s, p.count(a, k));
      }
    }
    request(a, p, a.x, a.xs, t + p.step, x);
    if (kRes) request(a, p, a.res, a.ress, t + p.step, res);
    float mean, square, rstd, off = 0.0f;
    centre(a, p, d, &mean, &square);
    if (P::kWide) {
      if ((threadIdx.x & 63) == 0) lds[turn][p.wave][0] = mean, lds[turn][p.wave][1] = square;
      __syncthreads();
      float all;
      join<P>(a, lds[turn], &all, &rstd);
      off = mean - all;
    } else {
      rstd = 1.0f / __builtin_sqrtf(square * p.inv_own + a.eps);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Vec8 y;
#pragma unroll
      for (int i = 0; i < 8; ++i) y.v[i] = __builtin_fmaf((d[k].v[i] + off) * rstd, w[k].v[i], b[k].v[i]);
      if (p.has(a, k)) store8<kWhole>(a.y + t * a.C + p.at(k), pack8(y), p.count(a, k));
    }
  }
}

// A lane's part of a partial row, `count` values of 8 or more: by words its lanes' would
// be 32 bytes apart.
__device__ __forceinline__ void part_put(float* p, const Vec8& v, int32_t count) {
  if (count >= 8) {
#pragma unroll
    for (int h = 0; h < 8; h += 4)
      *reinterpret_cast<f32x4_any*>(p + h) = (f32x4_any){v.v[h], v.v[h + 1], v.v[h + 2], v.v[h + 3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = v.v[i];
  }
}

template <int L, int K, bool kWhole, bool kRes>
__global__ __launch_bounds__(L > 64 ? L : 256) void layer_norm_bwd_kernel(LayerNormArgs a, int32_t rows,
                                                                          int32_t turns, int32_t parts) {
  typedef Team<L, K, kWhole> P;
  __shared__ float lds[2][P::kWaves][4];
  __shared__ float sums[P::kWide ? 1 : P::kTokens][P::kWide ? 1 : 2 * K * 8][P::kWide ? 1 : L + 1];
  const P p(a, rows);
  const float inv = 1.0f / (float)a.C;
  Vec8 w[K], dw[K], db[K];
  params<K>(a, p, a.w, a.w_bf16, w);
  u32x4_t x[K], dy[K], ds[K];
  auto fetch = [&](int64_t t) {
    request(a, p, a.x, a.xs, t, x);
    request(a, p, a.dy, a.dys, t, dy);
    if (kRes) request(a, p, a.dstream, a.dss, t, ds);
  };
  // Sixteen waves a workgroup, four a SIMD, have no registers for the next token.
  constexpr bool kAhead = L < 1024;
  if (kAhead) fetch(p.token);
  int turn = 0;
  int64_t t = p.token, end = 0;
#pragma unroll 1
  for (int64_t part = 0; part < parts; ++part) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) dw[k].v[i] = db[k].v[i] = 0.0f;
    end = min(a.S, end + turns * p.step);
#pragma unroll 1
    for (; t < end; t += p.step, turn ^= 1) {
      if (!kAhead) fetch(t);
      Vec8 d[K], g[K];
      u32x4_t dc[K];
#pragma unroll
      for (int k = 0; k < K; ++k) d[k] = unpack8(x[k]), g[k] = unpack8(dy[k]), dc[k] = kRes ? ds[k] : x[k];
      if (kAhead) fetch(t + p.step);
      float mean, square, rstd, off = 0.0f;
      centre(a, p, d, &mean, &square);
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = g[k].v[i] * w[k].v[i];
          s1 += q;
          s2 = __builtin_fmaf(q, d[k].v[i], s2);
        }
      s1 = lanes_sum<L < 64 ? L : 64>(s1);
      s2 = lanes_sum<L < 64 ? L : 64>(s2);
      if (P::kWide) {
        if ((threadIdx.x & 63) == 0) {
          lds[turn][p.wave][0] = mean;
          lds[turn][p.wave][1] = square;
          lds[turn][p.wave][2] = s1;
          lds[turn][p.wave][3] = s2;
        }
        __syncthreads();
        float all;
        join<P>(a, lds[turn], &all, &rstd);
        off = mean - all;
        s1 = s2 = 0.0f;
#pragma unroll P::kUnroll
        for (int v = 0; v < P::kWaves; ++v) {
          const float o = lds[turn][v][0] - all;
          s1 += lds[turn][v][2];
          s2 += __builtin_fmaf(o, lds[turn][v][2], lds[turn][v][3]);
        }
      } else {
        rstd = 1.0f / __builtin_sqrtf(square * p.inv_own + a.eps);
      }
      s1 *= inv;
      s2 *= inv * rstd;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Vec8 o;
        const Vec8 e = unpack8(dc[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = (d[k].v[i] + off) * rstd, q = g[k].v[i] * w[k].v[i];
          dw[k].v[i] = __builtin_fmaf(g[k].v[i], xh, dw[k].v[i]);
          db[k].v[i] += g[k].v[i];
          o.v[i] = rstd * __builtin_fmaf(-xh, s2, q - s1);
          if (kRes) o.v[i] += e.v[i];
        }
        if (p.has(a, k)) store8<kWhole>(a.dx + t * a.C + p.at(k), pack8(o), p.count(a, k));
      }
    }
    // The workgroup's partial row: its teams' sums in order.
    float* row = a.part + (part * rows + blockIdx.x) * 2 * a.C;
    if (P::kWide) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!p.has(a, k)) continue;
        part_put(row + p.at(k), dw[k], p.count(a, k));
        part_put(row + a.C + p.at(k), db[k], p.count(a, k));
      }
      continue;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[threadIdx.x / L][k * 8 + i][p.li] = dw[k].v[i];
        sums[threadIdx.x / L][(K + k) * 8 + i][p.li] = db[k].v[i];
      }
    __syncthreads();
    for (int32_t o = threadIdx.x; o < 2 * a.C; o += 256) {
      const int32_t c = o < a.C ? o : o - a.C, q = c / (8 * L) * 8 + c % 8 + (o < a.C ? 0 : K * 8), l = c / 8 % L;
      float s = 0.0f;
#pragma unroll
      for (int g = 0; g < P::kTokens; ++g) s += sums[g][q][l];
      row[o] = s;
    }
    if (part + 1 < parts) __syncthreads();  // the sums have been read
  }
}

// The partial rows of dw and db, summed in FP64: sixteen waves take their part of
// the rows each, and the first adds their sums in order.
__global__ __launch_bounds__(1024) void layer_norm_bwd_sum_kernel(LayerNormArgs a) {
  __shared__ double lds[16][64];
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int64_t i = (int64_t)blockIdx.x * 64 + lane, width = 2 * (int64_t)a.C;
  const int32_t per = (a.prows + 15) / 16, r0 = wave * per, r1 = min(r0 + per, a.prows);
  double s = 0.0;
  if (i < width) {
    int32_t r = r0;
    for (; r + 8 <= r1; r += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = a.part[(r + j) * width + i];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; r < r1; ++r) s += a.part[r * width + i];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave > 0 || i >= width) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) s += lds[w][lane];
  if (i < a.C) param_put(a.dw, a.w_bf16, i, (float)s);
  else if (a.db) param_put(a.db, a.b_bf16, i - a.C, (float)s);
}

// ------------------------------------------------------------------ launch --

bool vectors(const uint16_t* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

// Whether all vectors are whole and aligned (kWhole above).
bool whole(const LayerNormArgs& a) {
  return a.C % 8 == 0 && vectors(a.x, a.xs) && (!a.res || vectors(a.res, a.ress)) &&
         (!a.dy || vectors(a.dy, a.dys)) && (!a.dstream || vectors(a.dstream, a.dss)) && vectors(a.y, 8) &&
         vectors(a.stream, 8) && vectors(a.dx, 8);
}

struct Shape {
  int lanes, vecs;
};
// The fewest lanes that hold a row in one or two vectors each, whole waves alone past 64:
// exchanges between waves cost more than idle lanes.  16384 tokens, C = 1000, forward and
// backward 21.4 and 24.1 us by a wave, 23.5 and 53.4 by four; C = 4096 101 and 114 by four
// waves, 94 and 169 by eight; 8192 tokens, C = 8192 96 and 129 by eight, 130 and 177 by
// sixteen.
Shape shape_of(int64_t C) {
  const int64_t n = (C + 7) / 8;
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  if (n <= 512) return {256, n <= 256 ? 1 : 2};
  return {n <= 1024 ? 512 : 1024, 2};
}

// The forward's workgroups: sixteen waves a SIMD of single waves' tokens, and of wider
// ones as many as are at work at once, but half of those where they have four tokens or
// more each, whose requests are under way before they are needed: 16384 tokens, C = 4096
// and a residual 92 against 101 us, 8192 tokens, C = 8192 92 against 96; 700 tokens, C =
// 4096 6.6 against 5.4.
template <int L>
int64_t forward_rows(int64_t turns) {
  constexpr int64_t full = L <= 64 ? 4096 : L == 256 ? 1024 : L == 512 ? 512 : 256;
  if (L > 64 && L < 1024 && turns >= 4 * full) return full / 2;
  return turns < full ? turns : full;
}

// The backward's workgroups and their partial rows.  A row costs its writing and reading,
// too few leave the machine idle.  Forward and backward of 16384 tokens, C = 520 and a
// residual: 39 us with 512 rows, 47 with 256, 43 with 1024; backward, C = 2048: 32768
// tokens 105 with 1024 and 129 with 512, 1500 tokens 11.4 and 9.9; C = 4096, 16384
// tokens: 107 with 512, 120 with 1024, 142 with 256; C = 8192, 8192 tokens: 113 with 256,
// 128 with 512.  No more of them than take the same number of turns.
//
// A team adds its turns up in FP32, and the rows are added in FP64: what FP32 loses grows
// with the turns where terms are alike, so a row has 256 at most, and a workgroup of a long
// input several rows, one part of the tokens after the other.  1048577 tokens of the same
// values, C = 4096: dw off by 1.4e-5 in rows of 2048 turns, by 1.9e-6 so.
struct Rows {
  int64_t groups, turns, parts;
};
Rows backward_rows(int64_t S, int64_t C) {
  const Shape h = shape_of(C);
  const int64_t tokens = h.lanes > 64 ? 1 : 256 / h.lanes, turns = (S + tokens - 1) / tokens;
  const int64_t most = h.lanes >= 512 ? 256 : h.lanes == 256 && h.vecs == 1 && turns >= 4096 ? 1024 : 512;
  const int64_t each = (turns + most - 1) / most;
  if (each == 0) return {0, 0, 0};
  const int64_t parts = (each + 255) / 256;
  return {(turns + each - 1) / each, (each + parts - 1) / parts, parts};
}

template <int L, int K, bool kWhole>
void launch_vec(const LayerNormArgs& a, bool back, hipStream_t s) {
  typedef Team<L, K, kWhole> P;
  if (back) {
    const Rows r = backward_rows(a.S, a.C);
    const dim3 grid((uint32_t)r.groups), block(P::kThreads);
    const int32_t rows = (int32_t)r.groups, turns = (int32_t)r.turns, parts = (int32_t)r.parts;
    if (a.dstream) hipLaunchKernelGGL((layer_norm_bwd_kernel<L, K, kWhole, true>), grid, block, 0, s, a, rows, turns, parts);
    else hipLaunchKernelGGL((layer_norm_bwd_kernel<L, K, kWhole, false>), grid, block, 0, s, a, rows, turns, parts);
  } else {
    const int64_t rows = forward_rows<L>((a.S + P::kTokens - 1) / P::kTokens);
    const dim3 grid((uint32_t)rows), block(P::kThreads);
    if (a.res) hipLaunchKernelGGL((layer_norm_fwd_kernel<L, K, kWhole, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((layer_norm_fwd_kernel<L, K, kWhole, false>), grid, block, 0, s, a, (int32_t)rows);
  }
}

template <bool kWhole>
void launch_shape(const LayerNormArgs& a, bool back, hipStream_t s) {
  const Shape h = shape_of(a.C);
  if (h.lanes == 8) launch_vec<8, 1, kWhole>(a, back, s);
  else if (h.lanes == 16) launch_vec<16, 1, kWhole>(a, back, s);
  else if (h.lanes == 32) launch_vec<32, 1, kWhole>(a, back, s);
  else if (h.lanes == 64 && h.vecs == 1) launch_vec<64, 1, kWhole>(a, back, s);
  else if (h.lanes == 64) launch_vec<64, 2, kWhole>(a, back, s);
  else if (h.lanes == 256 && h.vecs == 1) launch_vec<256, 1, kWhole>(a, back, s);
  else if (h.lanes == 256) launch_vec<256, 2, kWhole>(a, back, s);
  else if (h.lanes == 512) launch_vec<512, 2, kWhole>(a, back, s);
  else launch_vec<1024, 2, kWhole>(a, back, s);
}

hipError_t launch(const LayerNormArgs& a, bool back, hipStream_t s) {
  if (whole(a)) launch_shape<true>(a, back, s);
  else launch_shape<false>(a, back, s);
  return hipGetLastError();
}

}  // namespace

int layer_norm_bwd_rows(int64_t S, int64_t C) {
  const Rows r = backward_rows(S, C);
  return (int)(r.groups * r.parts);
}

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, hipStream_t s) { return launch(a, false, s); }
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s) { return launch(a, true, s); }

hipError_t launch_layer_norm_bwd_sum(const LayerNormArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(layer_norm_bwd_sum_kernel, dim3((uint32_t)((2 * (int64_t)a.C + 63) / 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
