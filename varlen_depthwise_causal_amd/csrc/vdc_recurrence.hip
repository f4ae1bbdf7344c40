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
// workgroup has a tile of 64 or 128 channels by 128 (backward 64) tokens in
// registers, finds what the tile makes of any state, h -> P h + H, hands that on,
// takes the state that the tiles before it leave (backward: the gradient that the
// tiles behind it send), and finishes.  Two passes over a long row would read 14
// bytes instead of 8.
//
// Measured: 65536 tokens, C = 4096 with a gate, forward 543 us, 4.9 TB/s (a copy: 5.1);
// 16384 tokens 144 us, 4.7 TB/s, and backward 257, 4.7 TB/s, with VALU issue 67% and 64%
// busy at 48 and 82 instructions a token and 64 channels.  A few tiles are latency: 1543
// tokens, C = 520, 25 tiles in a row, 7.9 us forward and 11.7 backward.
//
// What a tile hands on is one 64-bit word a channel: P and H, or, once the state
// after the tile is known, that state and a mark in place of P.  A tile reads the
// words of those before it, one a wave, and folds them in order from the nearest
// marked one.  A marked word is by its definition the fold of the word before it with
// its own P and H, so where a fold begins makes no difference to its bits.
//
// No wait is for ever: a block of channels' tiles are numbered as their workgroups
// begin, each waits for lower numbers alone, and those have begun.  A word is written and
// read whole and holds all that its reader needs, so no fence is needed either.  The words
// and their folds are vdc_words.h's.
//
// Everything between documents is assigned, never multiplied by zero, so that
// an infinity or a NaN stays in its document.
//
// The decay's gradient is a sum in FP32 over a tile's 64 tokens, whose terms are rounded
// to FP32 already, and in FP64 over the tiles.

#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "vdc_layer.h"
#include "vdc_ssm_math.h"
#include "vdc_words.h"

namespace vdc {
namespace {

// u / sigmoid(r) of a channel, at most 2^126: no product of it is an infinity, which
// a decay of 0 would make a NaN.  The scale is not doubled first: where that is an
// infinity, a softplus of 0 would make a NaN too.
__device__ __forceinline__ float decay_rate(const RecurArgs& a, int64_t c) {
  const float rate = 2.0f * (a.scale * softplus_f32(param_at(a.decay, a.decay_bf16, c)));
  return rate > 0x1p126f ? 0x1p126f : rate;  // a NaN stays
}

// The decay exp(-u / 2).
__device__ __forceinline__ float decay_of(float u) { return __builtin_amdgcn_exp2f(u * (-0.5f * kLog2E)); }

// m = sqrt(1 - exp(-u)), with a = exp(-u / 2).  1 - a^2 cancels where a is near 1:
// below u = 1/4 it is u (1 - u q(u)), q the polynomial of degree 3 that makes that
// nearest in relative error (6e-9).
__device__ __forceinline__ float input_scale(float u, float a) {
  float q = -0.007534402422606945f;
  q = __builtin_fmaf(q, u, 0.04150218889117241f);
  q = __builtin_fmaf(q, u, -0.16665320098400116f);
  q = __builtin_fmaf(q, u, 0.49999964237213135f);
  const float small = u * __builtin_fmaf(-q, u, 1.0f);
  return __builtin_amdgcn_sqrtf(u < 0.25f ? small : __builtin_fmaf(-a, a, 1.0f));
}

// a b, and 0 where either is 0: a token without a step adds nothing, whatever its
// input holds.
extern "C" __device__ float vdc_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float gated(float a, float b) { return vdc_fmul_legacy(a, b); }

// ------------------------------------------------------------------- tiles --

// A lane's channel.  Lanes past the last one read the first one's values and store
// nothing.
struct Col {
  uint32_t c;
  bool has;
  __device__ __forceinline__ Col(const RecurArgs& a, int32_t block) {
    c = (uint32_t)block * 64u + (threadIdx.x & 63u);
    has = c < (uint32_t)a.C;
    if (!has) c = 0;
  }
};

// A run's rows of BF16, addressed by a buffer resource at the first of them: the
// lane's byte and a scalar offset per row, no address arithmetic in the lanes.  Rows
// past the last token are out of the resource's range, as are lanes past the last
// channel when they store: they read as zeros, and a store there is dropped.  The
// host keeps offsets below 2^31.
struct Run {
  __amdgpu_buffer_rsrc_t r;
  uint32_t stride;  // bytes
  int32_t left;     // rows from the first to the last token
  __device__ __forceinline__ Run(const uint16_t* base, int64_t stride_, int32_t t0, int32_t S)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + (int64_t)t0 * stride_), (short)0, 0x7fffffff,
                                            0x00020000)),
        stride((uint32_t)stride_ * 2u), left(S - t0) {
    // Known to this run alone: which rows are there would otherwise be kept in scalar
    // registers for all of a tile's tensors, and these run out.
    asm volatile("" : "+s"(left));
  }
  __device__ __forceinline__ int row(int j) const { return (int)(j < left ? (uint32_t)j * stride : 0x7fffffffu); }
  __device__ __forceinline__ uint32_t get(const Col& c, int j) const {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)(c.c * 2u), row(j), kOnce);
  }
  __device__ __forceinline__ void put(const Col& c, int j, float v) const {
    __builtin_amdgcn_raw_buffer_store_b16(bf16_of(v), r, (int)(c.has ? c.c * 2u : 0x80000000u), row(j), kOnce);
  }
  // Nothing is read or written twice: loads and stores do not stay in the caches.
  static constexpr int kOnce = 2;
};

template <int N>
__device__ __forceinline__ void rows(const Col& c, const uint16_t* t, int64_t stride, int32_t t0, int32_t S,
                                     uint32_t (&v)[N]) {
  const Run b(t, stride, t0, S);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = b.get(c, j);
}

// The documents that start or end among a tile's tokens.
template <int T, bool kState>
struct Starts {
  uint32_t mask[T / 32 + 1];          // bit j: a document starts at token j of the tile, or the last one ends before it
  int32_t from[kState ? T + 1 : 1];   // the slot whose state the document that starts there goes on from, or -1
  int32_t to[kState ? T + 1 : 1];     // the slot of the document that ends before it, or -1
};

template <int W, int T, bool kState>
__device__ __forceinline__ void clear_starts(Starts<T, kState>& s) {
  for (int i = threadIdx.x; i <= T; i += 64 * W) {
    if (i <= T / 32) s.mask[i] = 0;
    if (kState) s.from[i] = s.to[i] = -1;
  }
}

// All threads of the workgroup, an entry of cu_seqlens each and all its loads at
// once; the result is complete after the next barrier.  Where a wave has not come past
// the tile's tokens after sixteen entries a thread, nearly all of these are empty
// documents'; a search for each token, 62 loads one after another, passes the others, so
// that a tile has its word soon, while others wait for it.
template <int W, int T, bool kState>
__device__ __forceinline__ void find_starts(const RecurArgs& a, int32_t t0, Starts<T, kState>& s) {
  const int32_t entries = a.num_docs + 1;
  int32_t e = entries > 64 * W ? first_at_least(a.cu, entries, t0) : 0;
  e += threadIdx.x;
#pragma unroll 1
  for (int n = 0; n < 16; ++n, e += 64 * W) {
    int32_t v = INT_MAX, next = INT_MAX, past = INT_MAX, from = -1, to = -1;
    if (e < entries) v = a.cu[e];
    if (kState && e < a.num_docs) {
      next = a.cu[e + 1];
      if (a.resume && a.resume[e]) from = a.index ? a.index[e] : e;
    }
    if (kState && e > 0 && e < entries) {
      past = a.cu[e - 1];
      to = a.index ? a.index[e - 1] : e - 1;
    }
    const int64_t j = (int64_t)v - t0;
    if (v <= a.S && j >= 0 && j <= T) {
      atomicOr(&s.mask[j / 32], 1u << (j % 32));
      // Of the entries at one token the last is that of the document which starts
      // there, and the first follows the one that ends; others are empty ones'.
      if (kState && e < a.num_docs && next > v && from >= 0 && from < a.slots) s.from[j] = from;
      if (kState && past < v && to >= 0 && to < a.slots) s.to[j] = to;
    }
    if (__ballot(e < entries && j <= T) == 0) return;
  }
  const int32_t* const cu = a.cu;
#pragma unroll 1
  for (int j = threadIdx.x & 63; j <= T && t0 + j <= a.S; j += 64) {
    const TokenDocs d = token_docs([cu](int64_t i) { return cu[i]; }, entries, t0 + j);
    if (!d.any) continue;
    atomicOr(&s.mask[j / 32], 1u << (j % 32));
    if (!kState) continue;
    const int64_t from = d.starts >= 0 && a.resume && a.resume[d.starts] ? slot_of(a.index, d.starts, a.slots) : -1;
    const int64_t to = d.ends >= 0 ? slot_of(a.index, d.ends, a.slots) : -1;
    // other waves may write the same, and none another slot
    if (from >= 0) s.from[j] = (int32_t)from;
    if (to >= 0) s.to[j] = (int32_t)to;
  }
}

// Bits [at, at + N] of the mask, at a multiple of N.
template <int N>
__device__ __forceinline__ uint32_t bits_at(const uint32_t* mask, int at) {
  const uint32_t lo = mask[at / 32] >> (at % 32) & ((1u << N) - 1u), hi = mask[(at + N) / 32] >> ((at + N) % 32) & 1u;
  return __builtin_amdgcn_readfirstlane(lo | hi << N);
}

// Reads of a word before its reader gives up and has a NaN in its place: 0.6 s, at 0.14
// us each, while a tile's word is there within a fraction of a millisecond of the tile's
// beginning and those of all tiles before it.  Only calls that share a workspace come here.
constexpr int kPolls = 1 << 22;
// How often a tile looks at the next W words for a known one, before it waits for
// one.
constexpr int kLooks = 2;

__device__ __forceinline__ void hand_on(uint64_t* p, uint64_t w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A wave's words once all of them are there, or once all are known (kAll).
template <bool kAll>
__device__ __forceinline__ uint64_t take(uint64_t* p) {
  uint64_t w = 0;
  for (int n = 0; n < kPolls; ++n) {
    w = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__ballot(!there<kAll>(w)) == 0) break;
    __builtin_amdgcn_s_sleep(1);
  }
  return taken<kAll>(w);
}

// The words of the tiles before this one, W at a time, and which lanes have found a
// known one among those of each time.
template <int W>
struct Seen {
  uint64_t w[kLooks * W][64];
  uint64_t known[kLooks][W];
};

// What reaches this tile from those of lower numbers, `far` tiles of which there
// are; `step` leads from a tile's words to those of the next lower number.  All
// waves call it and have the result.
template <int W>
__device__ __forceinline__ float look_back(uint64_t* words, int64_t step, int32_t far, Seen<W>& seen) {
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  uint64_t missing = ~(uint64_t)0;
  int32_t looks = 0;
  bool all = false;  // the same in all waves
#pragma unroll 1
  while (looks < kLooks && !all) {
    const int32_t d = looks * W + wave;
    const uint64_t w = d < far ? take<false>(words + (int64_t)(d + 1) * step) : known(0.0f);
    seen.w[d][lane] = w;
    seen.known[looks][wave] = __ballot(mark(w) == kKnown);
    __syncthreads();
    uint64_t k = seen.known[looks][lane % W];
#pragma unroll
    for (int i = 1; i < W; i <<= 1) k |= __shfl_xor(k, i, 64);
    missing &= ~k;
    all = __builtin_amdgcn_readfirstlane((uint32_t)missing | (uint32_t)(missing >> 32)) == 0;
    ++looks;
  }
  if (!all) {  // so there are more than kLooks * W of them
    __syncthreads();
    if (wave == W - 1) seen.w[kLooks * W - 1][lane] = take<true>(words + (int64_t)(kLooks * W) * step);
    __syncthreads();
  }
  float carry = 0.0f;
#pragma unroll 4
  for (int d = looks * W - 1; d >= 0; --d) carry = folded(seen.w[d][lane], carry);
  return carry;
}

// The tile of this workgroup: its number, of its channel block, and that block.  Each
// block of channels has a counter of its own, 512 bytes apart: one for all of them hands
// its numbers out one after the other (1543 tokens, C = 520, 225 tiles, forward and
// backward: 26.2 against 22.5 us; 8192 tokens, C = 2048, forward: 48.4 against 43.4).
struct Place {
  int32_t n, block;
};
__device__ __forceinline__ Place place_of(const RecurArgs& a, uint32_t* lds) {
  const uint32_t blocks = (uint32_t)a.blocks;
  // Of `blocks` workgroups each has another block, and a block's are on all XCDs in turn
  // (on one XCD each: 16384 tokens, C = 4096, forward and backward 446 against 416 us).
  const uint32_t block = (blockIdx.x + blockIdx.x / blocks) % blocks;
  if (a.tiles > 1 && threadIdx.x == 0) *lds = atomicAdd(reinterpret_cast<uint32_t*>(a.tickets + block * 64), 1u) + 1u;
  __syncthreads();
  // Two calls that share a workspace run past the last.
  const uint32_t n = a.tiles > 1 ? min(__builtin_amdgcn_readfirstlane(*lds), (uint32_t)a.tiles - 1u) : 0;
  return {(int32_t)n, (int32_t)block};
}

// Documents without tokens leave zeros, or their slot as it is where they resume: those of
// [first, end).
template <int W>
__device__ __forceinline__ void empty_documents(const RecurArgs& a, int32_t first, int32_t end, const Col& c) {
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  for (int32_t d0 = first + wave * 64; d0 < end; d0 += 64 * W) {
    const int32_t d = d0 + lane;
    int32_t slot = -1;
    if (d < end && a.cu[d] == a.cu[d + 1] && !(a.resume && a.resume[d])) slot = (int32_t)slot_of(a.index, d, a.slots);
    for (uint64_t m = __ballot(slot >= 0); m; m &= m - 1) {
      const int64_t s = __builtin_amdgcn_readlane(slot, __builtin_ctzll(m));
      if (c.has) a.state[s * a.C + c.c] = 0.0f;
    }
  }
}

// A tile's part of the documents that it looks through for empty ones: the first of them,
// a thread's each, beside its loads, the others at its end.  Many of them take longer than
// the tiles behind this one wait for its word.
template <int W>
struct Part {
  int32_t first, then, end;
  __device__ __forceinline__ Part(const RecurArgs& a, int32_t k) {
    first = (int32_t)min((int64_t)k * a.docs_each, (int64_t)a.num_docs);
    end = first + min(a.docs_each, a.num_docs - first);
    then = first + min(64 * W, end - first);
  }
};

// 16 bytes a lane: 2 us for few words, 8.2 for 65536 tokens, C = 4096 (17 MB).
__global__ __launch_bounds__(256) void recur_clear_kernel(uint64_t* words, int64_t n) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
  if (i < n) *reinterpret_cast<u32x4_t*>(words + i) = (u32x4_t){kEmpty, kEmpty, kEmpty, kEmpty};
}

// No tokens, but documents that leave their states.
__global__ __launch_bounds__(512) void recur_empty_kernel(RecurArgs a) {
  empty_documents<8>(a, 0, a.num_docs, Col(a, blockIdx.x));
}

// The runs of a tile that have any of the bits kFrom .. kTo of theirs set, as a mask.
template <int N, int W, int kFrom, int kTo>
__device__ __forceinline__ uint32_t runs_with(const uint32_t* mask) {
  uint32_t w[W * N / 32 + 1], m = 0;
#pragma unroll
  for (int k = 0; k <= W * N / 32; ++k) w[k] = __builtin_amdgcn_readfirstlane(mask[k]);
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const int at = k * N;
    constexpr uint32_t low = ((kTo < N ? 2u << kTo : 1u << N) - 1u) & ~((1u << kFrom) - 1u);
    bool any = (w[at / 32] >> (at % 32) & low) != 0;
    if (kTo == N) any |= (w[(at + N) / 32] >> ((at + N) % 32) & 1u) != 0;
    m |= any ? 1u << k : 0u;
  }
  return m;
}

// W waves with a run of N tokens each.  Everything between the loads and the stores is
// in registers: 80 of them leave room for three workgroups of runs of 16 on a CU.
template <int N, int W, bool kGate, bool kState>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(6)))
void recur_fwd_kernel(RecurArgs a) {
  constexpr int T = N * W;
  static_assert(T <= kRecurFwdTile && kRecurKeep % N == 0, "");
  __shared__ Starts<T, kState> docs;
  __shared__ float2 sums[W][64];  // P and H of the waves' runs
  __shared__ Seen<W> seen;
  __shared__ uint32_t ticket;
  clear_starts<W>(docs);
  const Place p = place_of(a, &ticket);
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int32_t tile0 = p.n * T, t0 = tile0 + wave * N;
  const Col c(a, p.block);
  if (a.tiles == 1 && t0 >= a.S) {  // no tokens, but a part in finding documents
    find_starts<W>(a, tile0, docs);
    if (kState) empty_documents<W>(a, 0, a.num_docs, c);
    __syncthreads();
    __syncthreads();
    return;
  }
  uint32_t x[N], r[N], i[N], z[N];
  rows(c, a.r, a.rs, t0, a.S, r);
  rows(c, a.i, a.is, t0, a.S, i);
  rows(c, a.x, a.xs, t0, a.S, x);
  const float rate = decay_rate(a, c.c);
  find_starts<W>(a, tile0, docs);
  const Part<W> part(a, kState ? p.n : 0);
  if (kState) empty_documents<W>(a, part.first, part.then, c);
  if (kGate) rows(c, a.z, a.zs, t0, a.S, z);  // needed last; before the documents it takes 88 registers
  __syncthreads();
  const uint32_t bits = bits_at<N>(docs.mask, wave * N), own = bits & ((1u << N) - 1u);

  float A[N], B[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float u = rate * sigmoid_f32(bf16_lo(r[j]));
    A[j] = decay_of(u);
    B[j] = gated(input_scale(u, A[j]), sigmoid_f32(bf16_lo(i[j])) * bf16_lo(x[j]));
    if (j % 2) __builtin_amdgcn_sched_barrier(0);  // no more tokens side by side than registers hold
  }
  // A resumed document goes on from its slot's state.
  if (kState && a.resume && own) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (own >> j & 1u) {
        const int64_t slot = __builtin_amdgcn_readfirstlane(docs.from[wave * N + j]);
        if (slot >= 0) B[j] = __builtin_fmaf(A[j], a.state[slot * a.C + c.c], B[j]);
      }
  }
  float P = 1.0f, H = 0.0f;
  if (own == 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) P *= A[j], H = __builtin_fmaf(A[j], H, B[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) H = own >> j & 1u ? B[j] : __builtin_fmaf(A[j], H, B[j]);
  }
  sums[wave][lane] = {P, H};
  __syncthreads();

  const uint32_t starts = runs_with<N, W, 0, N - 1>(docs.mask);
  uint64_t* const mine = a.words + (int64_t)p.n * a.cols + p.block * 64 + lane;
  const bool waits = p.n > 0 && (__builtin_amdgcn_readfirstlane(docs.mask[0]) & 1u) == 0;  // on what comes from the left
  const bool cut = !waits || starts != 0;  // the tile's last state does not go by it
  const bool hands = wave == 0 && p.n + 1 < a.tiles;
  float tp = 1.0f, th = 0.0f;
  if (hands) {
#pragma unroll 2
    for (int k = 0; k < W; ++k) {
      const float2 s = sums[k][lane];
      th = starts >> k & 1u ? s.y : __builtin_fmaf(s.x, th, s.y);
      tp *= s.x;
    }
    hand_on(mine, cut ? known(th) : word_of(tp, th));
  }
  float h = 0.0f;
  if (waits) {
    h = look_back(mine, -(int64_t)a.cols, p.n, seen);
    if (hands && !cut) hand_on(mine, known(__builtin_fmaf(tp, h, th)));
  }
#pragma unroll 2
  for (int k = 0; k < wave; ++k) {
    const float2 s = sums[k][lane];
    h = starts >> k & 1u ? s.y : __builtin_fmaf(s.x, h, s.y);
  }
  if (a.keep && t0 % kRecurKeep == 0 && t0 < a.S && c.has) a.keep[(int64_t)(t0 / kRecurKeep) * a.C + c.c] = h;

  if (own == 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) h = B[j] = __builtin_fmaf(A[j], h, B[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) h = B[j] = own >> j & 1u ? B[j] : __builtin_fmaf(A[j], h, B[j]);
  }
  const Run y(a.y, a.C, t0, a.S);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float zj = kGate ? bf16_lo(z[j]) : 0.0f;
    y.put(c, j, kGate ? B[j] * (zj * sigmoid_f32(zj)) : B[j]);
  }
  // Documents that end leave their states.
  if (kState && bits >> 1) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (bits >> (j + 1) & 1u) {
        const int64_t slot = __builtin_amdgcn_readfirstlane(docs.to[wave * N + j + 1]);
        if (slot >= 0 && c.has) a.state[slot * a.C + c.c] = B[j];
      }
  }
  if (kState) empty_documents<W>(a, part.then, part.end, c);
}

// The decay's gradient from the sum of E.  sigmoid / softplus tends to 1 where both
// are too small to be told from 0.
__device__ __forceinline__ void put_ddecay(const RecurArgs& a, int64_t c, double s) {
  const float decay = param_at(a.decay, a.decay_bf16, c), soft = softplus_f32(decay);
  const float ratio = soft > FLT_MIN ? sigmoid_f32(decay) / soft : 1.0f;
  param_put(a.ddecay, a.decay_bf16, c, ratio * (float)s);
}

// N tokens a run, W runs a tile.  dy silu'(z) waits for the states in LDS: with it in
// registers two workgroups fit on a CU instead of three.
template <int N, int W, bool kGate>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(3)))
void recur_bwd_kernel(RecurArgs a) {
  constexpr int T = N * W;
  static_assert(T <= kRecurBwdTile, "");
  __shared__ Starts<T, false> docs;
  __shared__ float2 sums[W][64];  // P and H of the waves' runs
  __shared__ float sent[W][64];   // what a run sends to its left without any from its right
  __shared__ Seen<W> seen;
  __shared__ float gate[kGate ? W : 1][N][64];
  __shared__ double total[W][64];
  __shared__ uint32_t ticket;
  clear_starts<W>(docs);
  const Place p = place_of(a, &ticket);
  const int32_t k = a.tiles - 1 - p.n;  // the last tile first
  const int32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u), lane = threadIdx.x & 63;
  const int32_t tile0 = k * T, t0 = tile0 + wave * N;
  const Col c(a, p.block);
  if (a.tiles == 1 && t0 >= a.S) {  // no tokens
    find_starts<W>(a, tile0, docs);
    sums[wave][lane] = {1.0f, 0.0f};
    sent[wave][lane] = 0.0f;  // nothing to the left, and nothing to the sum
    __syncthreads();
    __syncthreads();
    __syncthreads();
    __syncthreads();
    if (a.sums) {
      total[wave][lane] = 0.0;
      __syncthreads();
    }
    return;
  }
  uint32_t x[N], r[N], i[N], z[N], dy[N];
  rows(c, a.r, a.rs, t0, a.S, r);
  rows(c, a.i, a.is, t0, a.S, i);
  rows(c, a.x, a.xs, t0, a.S, x);
  if (kGate) rows(c, a.z, a.zs, t0, a.S, z);
  rows(c, a.dy, a.dys, t0, a.S, dy);
  float h = a.keep[(int64_t)k * a.C + c.c];
  const float rate = decay_rate(a, c.c);
  find_starts<W>(a, tile0, docs);
  __syncthreads();
  const uint32_t bits = bits_at<N>(docs.mask, wave * N);

  float A[N], B[N], m[N], sr[N], si[N], g[N];
  float P = 1.0f, H = 0.0f, M = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    sr[j] = sigmoid_f32(bf16_lo(r[j]));
    si[j] = sigmoid_f32(bf16_lo(i[j]));
    const float u = rate * sr[j];
    A[j] = decay_of(u);
    m[j] = input_scale(u, A[j]);
    B[j] = gated(m[j], si[j] * bf16_lo(x[j]));
    g[j] = bf16_lo(dy[j]);
    if (kGate) {
      // dy silu(z), the gradient at the state, and dy silu'(z), dz but for the state
      const float zj = bf16_lo(z[j]), s = sigmoid_f32(zj);
      gate[wave][j][lane] = g[j] * dsilu_f32(zj, s);
      g[j] *= zj * s;
    }
    if (j % 2) __builtin_amdgcn_sched_barrier(0);  // no more tokens side by side than registers hold
  }
  if (bits == 0) {
#pragma unroll
    for (int j = 0; j < N; ++j) P *= A[j], H = __builtin_fmaf(A[j], H, B[j]);
#pragma unroll
    for (int j = N - 1; j >= 0; --j) M = A[j] * (g[j] + M);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      P *= A[j];
      H = bits >> j & 1u ? B[j] : __builtin_fmaf(A[j], H, B[j]);
    }
#pragma unroll
    for (int j = N - 1; j >= 0; --j) M = A[j] * (bits >> (j + 1) & 1u ? g[j] : g[j] + M);
  }
  sums[wave][lane] = {P, H};
  sent[wave][lane] = M;
  __syncthreads();

  const uint32_t starts = runs_with<N, W, 0, N - 1>(docs.mask);
  // Runs with a start behind their first token, up to the token after them: nothing
  // from the right gets through.
  const uint32_t shut = runs_with<N, W, 1, N>(docs.mask);
  uint64_t* const mine = a.words + (int64_t)k * a.cols + p.block * 64 + lane;
  const bool waits = p.n > 0 && (__builtin_amdgcn_readfirstlane(docs.mask[T / 32]) & 1u) == 0;
  const bool cut = !waits || shut != 0;
  const bool hands = wave == 0 && p.n + 1 < a.tiles;
  float tp = 1.0f, tm = 0.0f;
  if (hands) {
#pragma unroll 2
    for (int q = W - 1; q >= 0; --q) {
      const float s = sums[q][lane].x, o = sent[q][lane];
      tm = shut >> q & 1u ? o : __builtin_fmaf(s, tm, o);
      tp *= s;
    }
    hand_on(mine, cut ? known(tm) : word_of(tp, tm));
  }
  // The states before this run, from the one that the forward kept.
#pragma unroll 2
  for (int q = 0; q < wave; ++q) {
    const float2 s = sums[q][lane];
    h = starts >> q & 1u ? s.y : __builtin_fmaf(s.x, h, s.y);
  }
  const Run dz(a.dz, a.C, t0, a.S);
  // B becomes the state before the token.
  auto states = [&](auto plain) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool first = !decltype(plain)::value && (bits >> j & 1u);
      const float before = first ? 0.0f : h;
      h = first ? B[j] : __builtin_fmaf(A[j], h, B[j]);
      B[j] = before;
      if (kGate) dz.put(c, j, gate[wave][j][lane] * h);
      if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (bits == 0) states(std::true_type());
  else states(std::false_type());

  float left = 0.0f;  // l, and a l once a token is done
  if (waits) {
    left = look_back(mine, (int64_t)a.cols, p.n, seen);
    if (hands && !cut) hand_on(mine, known(__builtin_fmaf(tp, left, tm)));
  }
#pragma unroll 2
  for (int q = W - 1; q > wave; --q) {
    const float o = sent[q][lane];
    left = shut >> q & 1u ? o : __builtin_fmaf(sums[q][lane].x, left, o);
  }
  const Run dx(a.dx, a.C, t0, a.S), di(a.di, a.C, t0, a.S), dr(a.dr, a.C, t0, a.S);
  float sum = 0.0f;
#pragma unroll
  for (int j = N - 1; j >= 0; --j) {
    const float xj = bf16_lo(x[j]);
    left = bits >> (j + 1) & 1u ? g[j] : g[j] + left;
    const float lx = gated(m[j], left * si[j]);
    dx.put(c, j, lx);
    di.put(c, j, gated(lx, xj * (1.0f - si[j])));
    // u / 2 and u / (2 m): without a step the first is 0, or too small to matter
    const float half = 0.5f * rate * sr[j];
    const float w = half * __builtin_amdgcn_rcpf(m[j] < 0x1p-60f ? 0x1p-60f : m[j]);
    const float E = left * __builtin_fmaf(-half * A[j], B[j], gated(A[j] * A[j] * w, si[j] * xj));
    sum += E;
    dr.put(c, j, E * (1.0f - sr[j]));
    left *= A[j];
  }
  // The tile's partial sum: its waves' in order.
  __syncthreads();
  sent[wave][lane] = sum;
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int q = 1; q < W; ++q) sum += sent[q][lane];
    if (!a.sums) {
      if (c.has) a.part[(int64_t)k * a.C + c.c] = sum;
    } else if (a.tiles > 1) {
      hand_on(a.sums + (int64_t)k * a.cols + p.block * 64 + lane, known(sum));
    }
  }
  if (!a.sums || p.n + 1 < a.tiles) return;
  // Few tiles: the last one's workgroup adds them, in FP64, as their sums come.
  double s = a.tiles == 1 && wave == 0 ? sum : 0.0;
  const int32_t per = (a.tiles + W - 1) / W;
  if (a.tiles > 1)
    for (int32_t q = wave * per; q < min((wave + 1) * per, a.tiles); ++q)
      s += word_value(take<true>(a.sums + (int64_t)q * a.cols + p.block * 64 + lane));
  total[wave][lane] = s;
  __syncthreads();
  if (wave > 0 || !c.has) return;
#pragma unroll
  for (int q = 1; q < W; ++q) s += total[q][lane];
  put_ddecay(a, c.c, s);
}

// The tiles' sums of E in FP64, sixteen waves a part of the tiles each: chains of loads,
// 5.0 us for 256 tiles, C = 4096.
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
  put_ddecay(a, c, s);
}

// ----------------------------------------------------------- single tokens --

// V channels of a row a lane.  Bound by HBM for many rows, 18 bytes a row and channel with
// a gate (1000 rows, C = 4096: 15.8 us, 4.7 TB/s; 4000 rows 46.8, 6.3 TB/s, the last
// cache's part in it), by the host for few (one row: 2.8 us of 4.6).  Several rows a wave
// save no time (4000 rows 45.7), loads and stores past the caches lose some (52.8; 1000
// rows 15.4).  The rate's loads come first: behind the row's they hold it up (19.9).
template <int V>
struct StepRow {
  int64_t slot;
  uint32_t x[(V + 1) / 2], r[(V + 1) / 2], i[(V + 1) / 2], z[(V + 1) / 2];
  float h[V];
};
template <int V>
__device__ __forceinline__ void step_words(const uint16_t* p, uint32_t (&w)[(V + 1) / 2]) {
  if constexpr (V == 4) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = v[0], w[1] = v[1];
  } else {
    w[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void step_load(const RecurArgs& a, int64_t row, int64_t c, StepRow<V>* s) {
  s->slot = slot_of(a.index, row, a.slots);
  if (s->slot < 0) return;
  step_words<V>(a.x + row * a.xs + c, s->x);
  step_words<V>(a.r + row * a.rs + c, s->r);
  step_words<V>(a.i + row * a.is + c, s->i);
  if (a.z) step_words<V>(a.z + row * a.zs + c, s->z);
  const float* p = a.state + s->slot * a.C + c;
  if constexpr (V == 4) {
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int k = 0; k < V; ++k) s->h[k] = v[k];
  } else {
    s->h[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void step_row(const RecurArgs& a, int64_t row, int64_t c, const float (&rate)[V],
                                         const StepRow<V>& s) {
  float h[V], y[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    auto value = [&](const uint32_t* w) { return k % 2 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]); };
    const float u = rate[k] * sigmoid_f32(value(s.r)), decay = decay_of(u);
    h[k] = __builtin_fmaf(decay, s.h[k], gated(input_scale(u, decay), sigmoid_f32(value(s.i)) * value(s.x)));
    y[k] = h[k];
    if (a.z) {
      const float z = value(s.z);
      y[k] *= z * sigmoid_f32(z);
    }
    if (s.slot < 0) y[k] = 0.0f;
  }
  uint16_t* out = a.y + row * a.C + c;
  float* p = a.state + s.slot * a.C + c;
  if constexpr (V == 4) {
    const u32x2_t w = {bf16_pack2(y[0], y[1]), bf16_pack2(y[2], y[3])};
    *reinterpret_cast<u32x2_t*>(out) = w;
    if (s.slot >= 0) *reinterpret_cast<f32x4_t*>(p) = (f32x4_t){h[0], h[1], h[2], h[3]};
  } else {
    *out = bf16_of(y[0]);
    if (s.slot >= 0) *p = h[0];
  }
}

constexpr int64_t kStepGroups = int64_t(1) << 22;  // 2^30 threads; more rows take turns
template <int V>
__global__ __launch_bounds__(256) void recur_step_kernel(RecurArgs a) {
  const int64_t waves = (int64_t)a.blocks * a.S;
#pragma unroll 1
  for (int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64u); w < waves;
       w += (int64_t)gridDim.x * 4) {
    const int64_t row = w / a.blocks, c = ((w % a.blocks) * 64 + (threadIdx.x & 63)) * V;
    if (c >= a.C) continue;
    float rate[V];
#pragma unroll
    for (int k = 0; k < V; ++k) rate[k] = decay_rate(a, c + k);
    StepRow<V> s;
    step_load(a, row, c, &s);
    step_row(a, row, c, rate, s);
  }
}

// ------------------------------------------------------------------ launch --

template <int N, int W>
void launch_fwd(RecurArgs a, hipStream_t s) {
  a.blocks = (a.C + 63) / 64;
  const dim3 grid((uint32_t)((int64_t)a.tiles * a.blocks)), block(64 * W);
  if (a.z && a.state) hipLaunchKernelGGL((recur_fwd_kernel<N, W, true, true>), grid, block, 0, s, a);
  else if (a.z) hipLaunchKernelGGL((recur_fwd_kernel<N, W, true, false>), grid, block, 0, s, a);
  else if (a.state) hipLaunchKernelGGL((recur_fwd_kernel<N, W, false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((recur_fwd_kernel<N, W, false, false>), grid, block, 0, s, a);
}

template <int N, int W>
void launch_bwd(RecurArgs a, hipStream_t s) {
  a.blocks = (a.C + 63) / 64;
  const dim3 grid((uint32_t)((int64_t)a.tiles * a.blocks)), block(64 * W);
  if (a.z) hipLaunchKernelGGL((recur_bwd_kernel<N, W, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((recur_bwd_kernel<N, W, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_recur_clear(const RecurArgs& a, hipStream_t s) {
  const int64_t n = (1 + (int64_t)a.tiles * (a.sums ? 2 : 1)) * a.cols;
  hipLaunchKernelGGL(recur_clear_kernel, dim3((uint32_t)((n + 511) / 512)), dim3(256), 0, s, a.tickets, n);
  return hipGetLastError();
}

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  if (a.S == 0) hipLaunchKernelGGL(recur_empty_kernel, dim3((uint32_t)((a.C + 63) / 64)), dim3(512), 0, s, a);
  // A tile of one takes the longer the more tokens a wave has: 20 tokens, C = 2048 4.2
  // us in runs of 4 and 4.5 in runs of 8, 50 tokens, C = 1000 5.7 with eight waves and
  // 5.9 with sixteen.
  else if (a.S <= 32) launch_fwd<4, 8>(a, s);
  else if (a.S <= 64 || a.tile == 64) launch_fwd<8, 8>(a, s);
  else if (a.tiles == 1) launch_fwd<8, 16>(a, s);
  else launch_fwd<16, 8>(a, s);
  return hipGetLastError();
}

hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  // Runs of 16 tokens make the fewest instructions a token, shorter ones more waves:
  // 8000 tokens, C = 256, 500 tiles: 16.3 us in runs of 8 and 18.7 in runs of 16, 20
  // tokens, C = 2048: 5.9 in runs of 4 and 6.4 in runs of 8; 16384 tokens, C = 512: 49.9
  // in runs of 8 and 45.0 in runs of 16, C = 4096: 379 and 286.
  if (a.S <= 32) launch_bwd<4, 8>(a, s);
  else if (recur_tiles_of_64(a.S, a.C) <= 512) launch_bwd<8, 8>(a, s);
  else launch_bwd<16, 4>(a, s);
  return hipGetLastError();
}

hipError_t launch_recur_bwd_sum(const RecurArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(recur_bwd_sum_kernel, dim3((uint32_t)((a.C + 63) / 64)), dim3(1024), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_recur_step(const RecurArgs& args, hipStream_t s) {
  RecurArgs a = args;
  // Four channels a lane where they are one aligned vector in every row.
  auto fours = [](const void* p, int64_t stride) { return reinterpret_cast<uintptr_t>(p) % 8 == 0 && stride % 4 == 0; };
  const bool vec = a.C % 4 == 0 && fours(a.x, a.xs) && fours(a.r, a.rs) && fours(a.i, a.is) && fours(a.z, a.z ? a.zs : 0) &&
                   fours(a.y, 0) && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
  const int64_t cols = vec ? 256 : 64;
  a.blocks = (int32_t)((a.C + cols - 1) / cols);
  const dim3 grid((uint32_t)std::min((a.blocks * (int64_t)a.S + 3) / 4, kStepGroups)), block(256);
  if (vec) hipLaunchKernelGGL(recur_step_kernel<4>, grid, block, 0, s, a);
  else hipLaunchKernelGGL(recur_step_kernel<1>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace vdc
