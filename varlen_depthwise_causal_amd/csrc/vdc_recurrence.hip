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
// Bound by HBM, where a token's inputs are read once: 8 bytes a token and channel
// forward (10 with a gate), 14 (18) backward.  So both directions are one pass: a
// workgroup has a tile of 64 channels by 128 (backward 64) tokens in registers,
// finds what the tile makes of any state, h -> P h + H, hands that on, takes the
// state that the tiles before it leave (backward: the gradient that the tiles
// behind it send), and finishes.  Two passes over a long row would read 14 bytes
// instead of 8.
//
// What a tile hands on is one 64-bit word a channel: P and H, or, once the state
// after the tile is known, that state and a mark in place of P.  A tile reads the
// words of the eight before it and folds them in order from the nearest marked one.
// A marked word is by its definition the fold of the word before it with its own P
// and H, so where a fold begins makes no difference to its bits.
//
// No wait is for ever: tiles are numbered by a ticket as their workgroups begin,
// each waits for lower numbers alone, and those have begun.  A word is written and
// read whole and holds all that its reader needs, so no fence is needed either.
//
// Everything between documents is assigned, never multiplied by zero, so that
// an infinity or a NaN stays in its document.

#include <cfloat>
#include <climits>

#include "vdc_layer.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

constexpr int kW = kRecurWaves;

// u / sigmoid(r) of a channel.
__device__ __forceinline__ float decay_rate(const RecurArgs& a, int64_t c) {
  return 2.0f * a.scale * softplus_f32(param_at(a.decay, a.decay_bf16, c));
}

// What the decay's gate makes of a token.
struct Decay {
  float u, a;   // the decay exp(-u / 2)
  float rm, m;  // 1 / sqrt(1 - exp(-u)) and its inverse; both 0 without a step
};

// 1 - a^2 cancels where a is near 1: below u = 1/4 it is the series of 1 - exp(-u),
// whose first term left out is less than u^6 / 5040 of it, 2^-24.  A token whose u
// is below the normal numbers has no step.
__device__ __forceinline__ float decay_step(float rate, float sr) {
  const float u = rate * sr;
  return u > 256.0f ? 256.0f : u;  // no infinity times zero; a NaN stays
}
__device__ __forceinline__ float decay_of(float u) { return __builtin_amdgcn_exp2f(u * (-0.5f * kLog2E)); }
__device__ __forceinline__ Decay decay_from(float u, float a) {
  Decay g;
  g.u = u;
  g.a = a;
  float s = __builtin_fmaf(u, -1.0f / 720.0f, 1.0f / 120.0f);
  s = __builtin_fmaf(u, -s, 1.0f / 24.0f);
  s = __builtin_fmaf(u, -s, 1.0f / 6.0f);
  s = __builtin_fmaf(u, -s, 0.5f);
  s = __builtin_fmaf(u, -s, 1.0f);
  const float v = u < 0.25f ? u * s : __builtin_fmaf(-a, a, 1.0f);
  g.rm = v < FLT_MIN ? 0.0f : __builtin_amdgcn_rsqf(v);
  g.m = v * g.rm;
  return g;
}
// What a token adds to the state: nothing without a step, whatever x holds.
__device__ __forceinline__ float input_of(const Decay& g, float si, float x) {
  return g.rm == 0.0f ? 0.0f : g.m * (si * x);
}

// ------------------------------------------------------------------- tiles --

// A lane's channel; lanes past the last one go by the first one's addresses and
// store nothing.
struct Col {
  uint32_t c;
  bool has;
};
__device__ __forceinline__ Col col_of(const RecurArgs& a, int32_t block) {
  const uint32_t c = (uint32_t)block * kRecurCols + (threadIdx.x & 63u);
  const bool has = c < (uint32_t)a.C;
  return {has ? c : 0u, has};
}

// Rows t0 .. t0 + N - 1; past the last token the last one again.
template <int N>
__device__ __forceinline__ void rows(Col c, const uint16_t* t, int64_t stride, int32_t t0, int32_t S,
                                     uint16_t (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = (t + (int64_t)min(t0 + j, S - 1) * stride)[c.c];
}

// The documents that start or end among a tile's tokens.
template <int T, bool kState>
struct Starts {
  uint32_t mask[T / 32 + 1];       // bit j: a document starts at token j of the tile
  int32_t first[kState ? T + 1 : 1];  // the last entry of cu_seqlens that is token j: the document that starts there
  int32_t last[kState ? T + 1 : 1];   // the first one; the document before it ends there
};

template <int T, bool kState>
__device__ __forceinline__ void clear_starts(Starts<T, kState>& s) {
  for (int i = threadIdx.x; i <= T; i += 64 * kW) {
    if (i <= T / 32) s.mask[i] = 0;
    if (kState) s.first[i] = -1, s.last[i] = INT_MAX;
  }
}

// All threads of the workgroup; the masks are complete after the next barrier.
template <int T, bool kState>
__device__ __forceinline__ void find_starts(const RecurArgs& a, int32_t t0, Starts<T, kState>& s) {
  const int32_t entries = a.num_docs + 1;
  int32_t e = entries > 64 * kW ? first_at_least(a.cu, entries, t0) : 0;
  e += threadIdx.x;
  while (true) {
    int32_t v = INT_MAX;
    if (e < entries) v = a.cu[e];
    const int64_t j = (int64_t)v - t0;
    if (v <= a.S && j >= 0 && j <= T) {
      atomicOr(&s.mask[j / 32], 1u << (j % 32));
      if (kState) {
        atomicMax(&s.first[j], e);
        atomicMin(&s.last[j], e);
      }
    }
    if (__ballot(e < entries && j <= T) == 0) return;
    e += 64 * kW;
  }
}

// Bits [at, at + N] of the mask, at a multiple of N.
template <int N>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* mask, int at) {
  const uint32_t lo = mask[at / 32] >> (at % 32) & ((1u << N) - 1u), hi = mask[(at + N) / 32] >> ((at + N) % 32) & 1u;
  return __builtin_amdgcn_readfirstlane(lo | hi << N);
}

// Words.  The upper half is P, or one of two marks, which no P is: a product of
// decays is at least 0, and a NaN is written as the usual one.
constexpr uint32_t kEmpty = 0xffffffffu, kKnown = 0xfffffffeu;
// Reads of a word before its reader gives up: about a second.  Only two calls that
// share a workspace come here.
constexpr int kPolls = 1 << 18;

__device__ __forceinline__ uint64_t word_of(float P, float H) {
  const uint32_t p = P != P ? 0x7fc00000u : __float_as_uint(P);
  return (uint64_t)p << 32 | __float_as_uint(H);
}
__device__ __forceinline__ uint64_t known(float H) { return (uint64_t)kKnown << 32 | __float_as_uint(H); }
__device__ __forceinline__ uint32_t mark(uint64_t w) { return (uint32_t)(w >> 32); }

__device__ __forceinline__ void hand_on(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A wave's words once all of them are there, or once all are known.
template <bool kAll>
__device__ __forceinline__ uint64_t take(uint64_t* p) {
  uint64_t v = 0;
  for (int n = 0; n < kPolls; ++n) {
    v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__ballot(kAll ? mark(v) != kKnown : mark(v) == kEmpty) == 0) break;
    __builtin_amdgcn_s_sleep(1);
  }
  return v;
}

// What reaches this tile from those of lower numbers, `far` tiles of which there
// are; `step` leads from a tile's words to those of the next lower number.  All
// waves call it and have the result.
__device__ __forceinline__ float look_back(uint64_t* words, int64_t step, int32_t far, uint64_t (&seen)[kW][64]) {
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  seen[wave][lane] = wave < far ? take<false>(words + (wave + 1) * step) : known(0.0f);
  __syncthreads();
  bool found = false;
#pragma unroll
  for (int w = 0; w < kW; ++w) found |= mark(seen[w][lane]) == kKnown;
  if (__ballot(!found) != 0) {  // the same in all waves; there are more than eight tiles
    __syncthreads();
    if (wave == kW - 1) seen[wave][lane] = take<true>(words + kW * step);
    __syncthreads();
  }
  float carry = 0.0f;
#pragma unroll
  for (int w = kW - 1; w >= 0; --w) {
    const uint64_t v = seen[w][lane];
    const float H = __uint_as_float((uint32_t)v), P = __uint_as_float(mark(v));
    carry = mark(v) == kKnown ? H : __builtin_fmaf(P, carry, H);
  }
  return carry;
}

// The tile of this workgroup: its number and channel block.
struct Place {
  int32_t n, block;
};
__device__ __forceinline__ Place place_of(const RecurArgs& a, uint32_t* lds) {
  if (a.tiles > 1 && threadIdx.x == 0) *lds = atomicAdd(a.ticket, 1u);
  __syncthreads();
  const uint32_t t = a.tiles > 1 ? __builtin_amdgcn_readfirstlane(*lds) : blockIdx.x;
  // Two calls that share a workspace run past the last.
  const uint32_t n = min(t / (uint32_t)a.blocks, (uint32_t)a.tiles - 1u);
  return {(int32_t)n, (int32_t)(t % (uint32_t)a.blocks)};
}

// Documents without tokens leave zeros, or their slot as it is where they resume;
// part `k` of `parts`.
__device__ __forceinline__ void empty_documents(const RecurArgs& a, int32_t k, int32_t parts, Col c) {
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int64_t per = ((int64_t)a.num_docs + parts - 1) / parts, end = min((k + 1) * per, (int64_t)a.num_docs);
  for (int64_t d0 = k * per + wave * 64; d0 < end; d0 += 64 * kW) {
    const int64_t d = d0 + lane;
    bool empty = false;
    if (d < end) empty = a.cu[d] == a.cu[d + 1] && !(a.resume && a.resume[d]);
    for (uint64_t m = __ballot(empty); m; m &= m - 1) {
      const int64_t slot = slot_of(a.index, d0 + __builtin_ctzll(m), a.slots);
      if (slot >= 0 && c.has) a.state[slot * a.C + c.c] = 0.0f;
    }
  }
}

__global__ __launch_bounds__(256) void recur_clear_kernel(RecurArgs a, int64_t words) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
  if (i == 0) *a.ticket = 0;
  if (i < words) *reinterpret_cast<u32x4_t*>(a.words + i) = (u32x4_t){kEmpty, kEmpty, kEmpty, kEmpty};
}

// No tokens, but documents that leave their states.
__global__ __launch_bounds__(64 * kW) void recur_empty_kernel(RecurArgs a) {
  empty_documents(a, 0, 1, col_of(a, blockIdx.x));
}

// Runs of a tile for which `bit` says so, as a mask.
template <int N, class F>
__device__ __forceinline__ uint32_t runs(const uint32_t* mask, F bit) {
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) m |= bit(bits_at<N>(mask, w * N)) ? 1u << w : 0u;
  return m;
}

template <bool kGate, bool kState>
__global__ __launch_bounds__(64 * kW) __attribute__((amdgpu_waves_per_eu(4)))
void recur_fwd_kernel(RecurArgs a) {
  constexpr int N = kRecurFwdRun, T = kRecurFwdTile;
  __shared__ Starts<T, kState> docs;
  __shared__ float2 sums[kW][64];  // P and H of the waves' runs
  __shared__ uint64_t seen[kW][64];
  __shared__ uint32_t ticket;
  clear_starts(docs);
  const Place p = place_of(a, &ticket);
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int32_t tile0 = p.n * T, t0 = tile0 + wave * N;
  const Col c = col_of(a, p.block);
  uint16_t x[N], r[N], i[N], z[N];
  rows(c, a.r, a.rs, t0, a.S, r);
  rows(c, a.i, a.is, t0, a.S, i);
  rows(c, a.x, a.xs, t0, a.S, x);
  if (kGate) rows(c, a.z, a.zs, t0, a.S, z);
  const float rate = decay_rate(a, c.c);
  find_starts(a, tile0, docs);
  if (kState) empty_documents(a, p.n, a.tiles, c);
  __syncthreads();
  const uint32_t bits = bits_at<N>(docs.mask, wave * N), own = bits & ((1u << N) - 1u);

  float A[N], B[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float u = decay_step(rate, sigmoid_f32(bf16_f32(r[j])));
    const Decay g = decay_from(u, decay_of(u));
    A[j] = g.a;
    B[j] = input_of(g, sigmoid_f32(bf16_f32(i[j])), bf16_f32(x[j]));
  }
  // A resumed document goes on from its slot's state.
  if (kState && a.resume && own) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (own >> j & 1u) {
        const int32_t d = __builtin_amdgcn_readfirstlane(docs.first[wave * N + j]);
        const bool go_on = d >= 0 && d < a.num_docs && __builtin_amdgcn_readfirstlane((int32_t)a.resume[d]) != 0;
        const int64_t slot = go_on ? slot_of(a.index, d, a.slots) : -1;
        if (slot >= 0) B[j] = __builtin_fmaf(A[j], a.state[slot * a.C + c.c], B[j]);
      }
  }
  float P = 1.0f, H = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    P *= A[j];
    H = own >> j & 1u ? B[j] : __builtin_fmaf(A[j], H, B[j]);
  }
  sums[wave][lane] = {P, H};
  __syncthreads();

  const uint32_t starts = runs<N>(docs.mask, [](uint32_t b) { return (b & ((1u << N) - 1u)) != 0; });
  uint64_t* const mine = a.words + ((int64_t)p.n * a.blocks + p.block) * kRecurCols + lane;
  const bool waits = p.n > 0 && (docs.mask[0] & 1u) == 0;  // on what comes from the left
  const bool cut = !waits || starts != 0;                  // the tile's last state does not go by it
  const bool hands = wave == 0 && p.n + 1 < a.tiles;
  float tp = 1.0f, th = 0.0f;
  if (hands) {
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      const float2 s = sums[w][lane];
      th = starts >> w & 1u ? s.y : __builtin_fmaf(s.x, th, s.y);
      tp *= s.x;
    }
    hand_on(mine, cut ? known(th) : word_of(tp, th));
  }
  float h = 0.0f;
  if (waits) {
    h = look_back(mine, -(int64_t)a.blocks * kRecurCols, p.n, seen);
    if (hands && !cut) hand_on(mine, known(__builtin_fmaf(tp, h, th)));
  }
  for (int w = 0; w < wave; ++w) {
    const float2 s = sums[w][lane];
    h = starts >> w & 1u ? s.y : __builtin_fmaf(s.x, h, s.y);
  }
  if (a.keep && t0 % kRecurKeep == 0 && t0 < a.S && c.has) a.keep[(int64_t)(t0 / kRecurKeep) * a.C + c.c] = h;

#pragma unroll
  for (int j = 0; j < N; ++j) {
    h = own >> j & 1u ? B[j] : __builtin_fmaf(A[j], h, B[j]);
    float y = h;
    if (kGate) {
      const float zj = bf16_f32(z[j]);
      y *= zj * sigmoid_f32(zj);
    }
    if (t0 + j < a.S && c.has) (a.y + (int64_t)(t0 + j) * a.C)[c.c] = bf16_of(y);
    if (kState && bits >> (j + 1) & 1u) {
      const int32_t d = __builtin_amdgcn_readfirstlane(docs.last[wave * N + j + 1]) - 1;
      const int64_t slot = d >= 0 && d < a.num_docs ? slot_of(a.index, d, a.slots) : -1;
      if (slot >= 0 && c.has) a.state[slot * a.C + c.c] = h;
    }
  }
}

template <bool kGate>
__global__ __launch_bounds__(64 * kW) __attribute__((amdgpu_waves_per_eu(4)))
void recur_bwd_kernel(RecurArgs a) {
  constexpr int N = kRecurBwdRun, T = kRecurBwdTile;
  __shared__ Starts<T, false> docs;
  __shared__ float2 sums[kW][64];  // P and H of the waves' runs
  __shared__ float sent[kW][64];   // what a run sends to its left without any from its right
  __shared__ uint64_t seen[kW][64];
  __shared__ uint32_t ticket;
  clear_starts(docs);
  const Place p = place_of(a, &ticket);
  const int32_t k = a.tiles - 1 - p.n;  // the last tile first
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int32_t tile0 = k * T, t0 = tile0 + wave * N;
  const Col c = col_of(a, p.block);
  uint16_t x[N], r[N], i[N], z[N], dy[N];
  rows(c, a.r, a.rs, t0, a.S, r);
  rows(c, a.i, a.is, t0, a.S, i);
  rows(c, a.x, a.xs, t0, a.S, x);
  if (kGate) rows(c, a.z, a.zs, t0, a.S, z);
  rows(c, a.dy, a.dys, t0, a.S, dy);
  float h = a.keep[(int64_t)k * a.C + c.c];
  const float rate = decay_rate(a, c.c);
  find_starts(a, tile0, docs);
  __syncthreads();
  const uint32_t bits = bits_at<N>(docs.mask, wave * N);

  float A[N], B[N], si[N], sr[N], g[N];
  float P = 1.0f, H = 0.0f, M = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    sr[j] = sigmoid_f32(bf16_f32(r[j]));
    si[j] = sigmoid_f32(bf16_f32(i[j]));
    const float u = decay_step(rate, sr[j]);
    const Decay d = decay_from(u, decay_of(u));
    A[j] = d.a;
    B[j] = input_of(d, si[j], bf16_f32(x[j]));
    g[j] = bf16_f32(dy[j]);
    if (kGate) {
      const float zj = bf16_f32(z[j]);
      g[j] *= zj * sigmoid_f32(zj);
    }
    if (t0 + j >= a.S) g[j] = 0.0f;  // rows past the last token send nothing
    P *= A[j];
    H = bits >> j & 1u ? B[j] : __builtin_fmaf(A[j], H, B[j]);
  }
#pragma unroll
  for (int j = N - 1; j >= 0; --j) M = A[j] * (bits >> (j + 1) & 1u ? g[j] : g[j] + M);
  sums[wave][lane] = {P, H};
  sent[wave][lane] = M;
  __syncthreads();

  const uint32_t starts = runs<N>(docs.mask, [](uint32_t b) { return (b & ((1u << N) - 1u)) != 0; });
  // Runs with a start behind their first token, up to the token after them: nothing
  // from the right gets through.
  const uint32_t shut = runs<N>(docs.mask, [](uint32_t b) { return b >> 1 != 0; });
  uint64_t* const mine = a.words + ((int64_t)k * a.blocks + p.block) * kRecurCols + lane;
  const bool waits = p.n > 0 && (docs.mask[T / 32] & 1u) == 0;
  const bool cut = !waits || shut != 0;
  const bool hands = wave == 0 && p.n + 1 < a.tiles;
  float tp = 1.0f, tm = 0.0f;
  if (hands) {
#pragma unroll
    for (int w = kW - 1; w >= 0; --w) {
      const float s = sums[w][lane].x, m = sent[w][lane];
      tm = shut >> w & 1u ? m : __builtin_fmaf(s, tm, m);
      tp *= s;
    }
    hand_on(mine, cut ? known(tm) : word_of(tp, tm));
  }
  // The states before this run, from the one that the forward kept.
  for (int w = 0; w < wave; ++w) {
    const float2 s = sums[w][lane];
    h = starts >> w & 1u ? s.y : __builtin_fmaf(s.x, h, s.y);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float before = bits >> j & 1u ? 0.0f : h;
    h = bits >> j & 1u ? B[j] : __builtin_fmaf(A[j], h, B[j]);
    B[j] = before;  // from here on the state before the token
    if (kGate) {
      const float zj = bf16_f32(z[j]), dz = bf16_f32(dy[j]) * h * dsilu_f32(zj, sigmoid_f32(zj));
      if (t0 + j < a.S && c.has) (a.dz + (int64_t)(t0 + j) * a.C)[c.c] = bf16_of(dz);
    }
  }

  float m = 0.0f;
  if (waits) {
    m = look_back(mine, (int64_t)a.blocks * kRecurCols, p.n, seen);
    if (hands && !cut) hand_on(mine, known(__builtin_fmaf(tp, m, tm)));
  }
  for (int w = kW - 1; w > wave; --w) {
    const float o = sent[w][lane];
    m = shut >> w & 1u ? o : __builtin_fmaf(sums[w][lane].x, m, o);
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = N - 1; j >= 0; --j) {
    const float l = bits >> (j + 1) & 1u ? g[j] : g[j] + m;
    const Decay d = decay_from(decay_step(rate, sr[j]), A[j]);
    const float xj = bf16_f32(x[j]), half = 0.5f * d.u;
    m = d.a * l;
    const float dx = l * d.m * si[j];
    const float di = d.rm == 0.0f ? 0.0f : dx * xj * (1.0f - si[j]);
    const float in = d.rm == 0.0f ? 0.0f : si[j] * xj * (d.a * d.a) * (half * d.rm);
    const float E = l * __builtin_fmaf(-half * d.a, B[j], in);
    if (t0 + j < a.S) {
      sum += E;
      if (c.has) {
        const int64_t at = (int64_t)(t0 + j) * a.C;
        (a.dx + at)[c.c] = bf16_of(dx);
        (a.di + at)[c.c] = bf16_of(di);
        (a.dr + at)[c.c] = bf16_of(E * (1.0f - sr[j]));
      }
    }
  }
  // The tile's partial sum: its waves' in order.
  __syncthreads();
  sent[wave][lane] = sum;
  __syncthreads();
  if (wave > 0 || !c.has) return;
#pragma unroll
  for (int w = 1; w < kW; ++w) sum += sent[w][lane];
  a.part[(int64_t)k * a.C + c.c] = sum;
}

// The tiles' sums of E in FP64, sixteen waves a part of the tiles each.
__global__ __launch_bounds__(1024) void recur_bwd_sum_kernel(RecurArgs a) {
  __shared__ double lds[16][64];
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int32_t per = (a.tiles + 15) / 16, r0 = wave * per, r1 = min(r0 + per, a.tiles);
  double s = 0.0;
  if (c < a.C) {
    int32_t r = r0;
    for (; r + 8 <= r1; r += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = a.part[(int64_t)(r + j) * a.C + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; r < r1; ++r) s += a.part[(int64_t)r * a.C + c];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave > 0 || c >= a.C) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) s += lds[w][lane];
  const float decay = param_at(a.decay, a.decay_bf16, c), soft = softplus_f32(decay);
  // sigmoid / softplus, which tends to 1 where both are too small to be told from 0
  const float ratio = soft > FLT_MIN ? sigmoid_f32(decay) / soft : 1.0f;
  param_put(a.ddecay, a.decay_bf16, c, ratio * (float)s);
}

// ----------------------------------------------------------- single tokens --

__global__ __launch_bounds__(64) void recur_step_kernel(RecurArgs a) {
  const int64_t blocks = (a.C + 63) / 64, row = blockIdx.x / blocks;
  const int64_t c = (blockIdx.x - row * blocks) * 64 + threadIdx.x;
  const int64_t slot = slot_of(a.index, row, a.slots);
  if (c >= a.C) return;
  float y = 0.0f;
  if (slot >= 0) {
    const float u = decay_step(decay_rate(a, c), sigmoid_f32(bf16_f32(a.r[row * a.rs + c])));
    const Decay g = decay_from(u, decay_of(u));
    const float b = input_of(g, sigmoid_f32(bf16_f32(a.i[row * a.is + c])), bf16_f32(a.x[row * a.xs + c]));
    float* p = a.state + slot * a.C + c;
    y = __builtin_fmaf(g.a, *p, b);
    *p = y;
    if (a.z) {
      const float z = bf16_f32(a.z[row * a.zs + c]);
      y *= z * sigmoid_f32(z);
    }
  }
  a.y[row * a.C + c] = bf16_of(y);
}

// ------------------------------------------------------------------ launch --

dim3 tile_grid(const RecurArgs& a) { return dim3((uint32_t)((int64_t)a.tiles * a.blocks)); }

template <bool kGate>
void launch_fwd_gate(const RecurArgs& a, hipStream_t s) {
  if (a.state) hipLaunchKernelGGL((recur_fwd_kernel<kGate, true>), tile_grid(a), dim3(64 * kW), 0, s, a);
  else hipLaunchKernelGGL((recur_fwd_kernel<kGate, false>), tile_grid(a), dim3(64 * kW), 0, s, a);
}

}  // namespace

hipError_t launch_recur_clear(const RecurArgs& a, hipStream_t s) {
  const int64_t words = (int64_t)a.tiles * a.blocks * kRecurCols;
  hipLaunchKernelGGL(recur_clear_kernel, dim3((uint32_t)((words + 511) / 512)), dim3(256), 0, s, a, words);
  return hipGetLastError();
}

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  if (a.S == 0) hipLaunchKernelGGL(recur_empty_kernel, dim3((uint32_t)a.blocks), dim3(64 * kW), 0, s, a);
  else if (a.z) launch_fwd_gate<true>(a, s);
  else launch_fwd_gate<false>(a, s);
  return hipGetLastError();
}

hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  if (a.z) hipLaunchKernelGGL((recur_bwd_kernel<true>), tile_grid(a), dim3(64 * kW), 0, s, a);
  else hipLaunchKernelGGL((recur_bwd_kernel<false>), tile_grid(a), dim3(64 * kW), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_recur_bwd_sum(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_bwd_sum_kernel, dim3((uint32_t)((a.C + 63) / 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_recur_step(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_step_kernel, dim3((uint32_t)((int64_t)a.S * ((a.C + 63) / 64))), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
