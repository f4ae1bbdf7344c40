// The selective state space scan over packed documents: forward for prompts
// and training, backward, and the form for single tokens.
//
// For token t, channel c, state n, with d = softplus(dt + bias):
//
//   h[t,c,n] = exp(d[t,c] A[c,n]) h[t-1,c,n] + d[t,c] x[t,c] B[t,n]
//   y[t,c]   = (sum_n C[t,n] h[t,c,n] + D[c] x[t,c]) silu(z[t,c])
//
// The decay differs for every (token, channel, state), so the sum over time
// is no matrix product: an element costs one exponential and four FP32
// instructions, and the kernels are bound by VALU issue, not by HBM: 24 cycles
// a wave for 64 elements where an FP32 instruction takes 4 and an exponential 8,
// that is 164 us for one pass over 16384 tokens of 4096 channels with 16 states
// on 1024 SIMDs at 2.4 GHz; a step size, a gate and the conversions of a token
// and channel cost as much as 6 states more.
//
// Time is cut into chunks that run in parallel.  The states after each chunk
// are found first with zero history (scan_local), joined in order
// (scan_join; the decay over a whole chunk is exp(A sum d), one exponential),
// and the outputs follow with the right state at each chunk's start.
// Everything between documents is assigned, never multiplied by zero, so
// that an infinity or a NaN stays in its document.

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "vdc_ssm.h"
#include "vdc_ssm_math.h"

namespace vdc {
namespace {

// A value that is the same in all lanes, back in scalar registers: where
// control flow joins the compiler may have moved it to vector registers.
__device__ __forceinline__ const uint16_t* uniform(const uint16_t* p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (const uint16_t*)(uintptr_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// Whether document d resumes, and its slot.
__device__ __forceinline__ bool resumes(const ScanArgs& a, int32_t d) {
  return a.resume && __builtin_amdgcn_readfirstlane((int32_t)a.resume[d]) != 0;
}
__device__ __forceinline__ int64_t doc_slot(const ScanArgs& a, int32_t d) {
  return slot_of(a.index, d, a.slots);
}

// The bias of a channel's step size.
__device__ __forceinline__ float step_bias(const ScanArgs& a, int64_t c) {
  return a.bias ? param_at(a.bias, a.bias_bf16, c) : 0.0f;
}
__device__ __forceinline__ float step_size(const ScanArgs& a, float dt, float bias) {
  const float v = dt + bias, s = softplus_f32(v);
  return a.softplus ? s : v;
}

// One BF16 row of activations after another, addressed by a buffer resource
// at the first of them: the lane's byte and a scalar offset per row, no
// address arithmetic in the lanes.  The host keeps every offset below 2^31.
struct RowBuffer {
  __amdgpu_buffer_rsrc_t r;
  uint32_t row, stride;  // byte offset of the current row, bytes between rows
  __device__ __forceinline__ void open(const uint16_t* base, int64_t first, int64_t stride_) {
    const uint16_t* p = base + first * stride_;
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), (short)0, 0x7fffffff, 0x00020000);
    row = 0;
    stride = (uint32_t)stride_ * 2u;
  }
  __device__ __forceinline__ uint32_t get(uint32_t lane2) const {
    return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)lane2, (int)row, 0);
  }
  __device__ __forceinline__ void put(uint32_t lane2, uint16_t v) const {
    __builtin_amdgcn_raw_buffer_store_b16(v, r, (int)lane2, (int)row, 0);
  }
};

// The piece of work of a wave, -1: none.  Neighbouring workgroups go to
// different XCDs; this hands each XCD a contiguous range of the work instead,
// so that the cache lines two waves share at their channels' border, and the
// rows of B and C that all waves of a chunk read, meet in one L2.  The waves
// are independent of each other, but come kWaves to a workgroup: those of one
// workgroup go to the four SIMDs of a CU in turn, where single waves crowd
// some SIMDs, which then finish last.  The grid is a multiple of kXcds.
constexpr uint32_t kXcds = 8, kWaves = 4;
__device__ __forceinline__ int32_t place_of(int32_t work) {
  const uint32_t p = ((blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds) * kWaves +
                     __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
  return p < (uint32_t)work ? (int32_t)p : -1;
}
inline uint32_t place_grid(int64_t work) {
  const int64_t blocks = (work + kWaves - 1) / kWaves;
  return (uint32_t)((blocks + kXcds - 1) / kXcds * kXcds);
}

// ------------------------------------------- B and C of one token, uniform --
//
// Every lane of a wave needs the same N values of B and of C, so they live in
// scalar registers: scalar loads of whole dwords, split into FP32 by the scalar
// unit.  That takes rows of NT states at multiples of 4 bytes; others are copied
// to the workspace first, padded with zeros (scan_pad_kernel).  Loads by lanes and
// reads out of them instead cost two VALU instructions a state and token: 359 us
// against 229 with the copy for 8192 tokens, C = 4096, 13 states, forward.

template <int NT>
struct Uniform {
  uint32_t v[NT / 2];
  __device__ __forceinline__ void load(const uint16_t* row) {
    scalar_ptr p = (scalar_ptr)(uintptr_t)row;
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) v[i] = p[i];
  }
  // Keeps the values in scalar registers where control flow joins.
  __device__ __forceinline__ void pin() {
#pragma unroll
    for (int i = 0; i < NT / 2; ++i) v[i] = __builtin_amdgcn_readfirstlane(v[i]);
  }
  __device__ __forceinline__ float get(int n) const {
    return n % 2 ? bf16_hi(v[n / 2]) : bf16_lo(v[n / 2]);
  }
};

// B's and C's rows, one after another, with NT states a group: a lane has two,
// and of very long rows more in turn (a launch has less than 2^32 lanes).
constexpr int64_t kPadBlocks = int64_t(1) << 22;
__global__ __launch_bounds__(256) void scan_pad_kernel(ScanArgs a, int32_t NT) {
  const int64_t each = (int64_t)a.S * a.G * (NT / 2);
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < 2 * each; e += kPadBlocks * 256) {
    const bool is_c = e >= each;
    const int64_t q = is_c ? e - each : e, row = q / (NT / 2), t = row / a.G;
    const int32_t n = (int32_t)(q - row * (NT / 2)) * 2;
    const uint16_t* p = (is_c ? a.Cm + t * a.Cs : a.B + t * a.Bs) + (row - t * a.G) * a.N;
    const uint32_t lo = n < a.N ? p[n] : 0u, hi = n + 1 < a.N ? p[n + 1] : 0u;
    a.pad[e] = lo | hi << 16;
  }
}

// ---------------------------------------------- forward, lane = channel --

// A lane's channel: column of the workspace rows, channel, and whether the
// channel exists (a group's last wave may have lanes past it; they run on
// its first channel's addresses and store nothing).
struct Column {
  int32_t group;
  uint32_t col, c;  // unsigned: 32-bit offsets from uniform addresses
  bool active;
};

__device__ __forceinline__ Column column_of(const ScanArgs& a, int32_t wave) {
  Column o;
  o.group = wave / a.wpg;
  const int32_t i = (wave - o.group * a.wpg) * 64 + (int32_t)(threadIdx.x & 63);
  o.col = (uint32_t)wave * 64u + (threadIdx.x & 63u);
  o.active = i < a.per;
  o.c = (uint32_t)(o.group * a.per + (o.active ? i : 0));
  return o;
}

// Vectors at any address that holds their elements.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// The decay of a state past the last: any finite step leaves its zero as it is,
// and so does an infinite one, for which a decay of 0 would make a NaN.
constexpr float kNoState = -FLT_MIN;

// A's row of a channel times log2(e); kNoState past the last state.  Rows of
// exactly NT states are loaded by vectors.
template <int NT>
__device__ __forceinline__ void load_decay(const ScanArgs& a, const Column& l, float (&A2)[NT]) {
  const int64_t at = (int64_t)l.c * a.N;
  const uint16_t* p2 = static_cast<const uint16_t*>(a.A) + at;
  const float* p4 = static_cast<const float*>(a.A) + at;
  if (a.N == NT && a.A_bf16) {
#pragma unroll
    for (int n = 0; n < NT; n += 8) {
      const u32x4_any v = *reinterpret_cast<const u32x4_any*>(p2 + n);
#pragma unroll
      for (int j = 0; j < 4; ++j) A2[n + 2 * j] = bf16_lo(v[j]), A2[n + 2 * j + 1] = bf16_hi(v[j]);
    }
  } else if (a.N == NT) {
#pragma unroll
    for (int n = 0; n < NT; n += 4) {
      const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p4 + n);
#pragma unroll
      for (int j = 0; j < 4; ++j) A2[n + j] = v[j];
    }
  } else if (a.A_bf16) {
#pragma unroll
    for (int n = 0; n < NT; ++n) A2[n] = bf16_f32(p2[min(n, a.N - 1)]);
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) A2[n] = p4[min(n, a.N - 1)];
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) A2[n] = n < a.N ? A2[n] * kLog2E : kNoState;
}

// A value the compiler must not compute addresses from ahead of its use: the
// rare paths' addresses would otherwise be held in registers over the loops.
__device__ __forceinline__ uint32_t here(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
// Values that are complete at this point of the program: without it the
// compiler runs the tokens of an unrolled loop side by side, which takes more
// registers than there are.
__device__ __forceinline__ void settled(float& a, float& b, float& c) {
  asm volatile("" : "+v"(a), "+v"(b), "+v"(c));
}
__device__ __forceinline__ int32_t here_uniform(int32_t v) {
  asm volatile("" : "+s"(v));
  return v;
}

// One pass over a chunk.  kOut = false: the state after the chunk from zero
// history (or a document's own start), the sum of the step sizes, and what a
// resumed document that runs past the chunk began with.  kOut = true: the
// outputs, from the joined states.  A lane has a channel with all its states, so
// that the step size, the gate and the sum over states cost no other lane
// anything, and B and C come from scalar registers, free of VALU instructions.
// 16384 tokens, C = 4096, 16 states: 187 us without the outputs and 251 with
// them, VALU busy 93 and 91% of the time; HBM moves 0.55 GB in the second.
template <int NT, bool kOut>
__global__ __launch_bounds__(64 * kWaves)
__attribute__((amdgpu_waves_per_eu(NT <= 16 ? 4 : NT == 32 ? 2 : 1)))
void scan_fwd_kernel(ScanArgs a, int32_t work) {
  constexpr int kAhead = NT <= 16 ? 8 : 4;
  const int32_t place = place_of(work);
  if (place < 0) return;
  const int32_t waves = a.G * a.wpg;
  const int32_t k = place / waves, w = place - k * waves;
  const Column l = column_of(a, w);
  const int32_t t0 = k * a.chunk;
  const int32_t t1 = (int32_t)min((int64_t)a.S, (int64_t)t0 + a.chunk);
  // Row n of a chunk's states in the workspace.
  auto row = [&](float* base, int32_t chunk, int n) {
    return base + ((int64_t)chunk * a.N + n) * a.cols;
  };
  float A2[NT], h[NT];
  load_decay<NT>(a, l, A2);
  const float Dc = a.D ? param_at(a.D, a.D_bf16, l.c) : 0.0f;
  const float bias = step_bias(a, l.c);
  const bool gated = kOut && a.z != nullptr;
  float sum = 0.0f;
  int32_t flags = 0;
#pragma unroll
  for (int n = 0; n < NT; ++n) h[n] = 0.0f;

  int32_t doc, next;  // the document of token t, and where it ends
  int32_t t = t0;
  // Document `d` is the first that may start at t: passes the empty ones
  // (whose slots hold an empty sequence's state, zero, unless they resume)
  // and begins the next.
  auto open = [&](int32_t d) {
    while (d < a.num_docs && uniform_at(a.cu, d + 1) <= t) {
      if (kOut && a.state && l.active) {
        const int64_t slot = doc_slot(a, d);
        if (slot >= 0 && !resumes(a, d))
          for (int n = 0; n < a.N; ++n) (a.state + slot * a.C * a.N)[here(l.c) * a.N + n] = 0.0f;
      }
      ++d;
    }
    doc = d;
    next = d < a.num_docs ? uniform_at(a.cu, d + 1) : INT32_MAX;
#pragma unroll
    for (int n = 0; n < NT; ++n) h[n] = 0.0f;
    flags |= t == t0 ? 1 : 2;
    if (a.state && d < a.num_docs && resumes(a, d)) {
      const int64_t slot = doc_slot(a, d);
      if (slot >= 0) {
        // The chunk that ends a document writes its slot while others may
        // still have to read it: a document that runs past its first chunk
        // has its start copied by the first pass and read from there.  The
        // first pass leaves the last chunk out: an end past the last token,
        // which only malformed prefix sums have, must not ask for a copy.
        const bool past = next > t1 && t1 < a.S;
        const uint32_t col = here(l.col);
        const int32_t kk = here_uniform(k), N = here_uniform(a.N);
        if (kOut && past) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < N) h[n] = row(a.snap, kk, n)[col];
        } else {
          const float* s = a.state + slot * a.C * a.N + here(l.c) * (uint32_t)a.N;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n < N) h[n] = s[n];
          if (past) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n < N) row(a.snap, kk, n)[col] = h[n];
          }
        }
      }
    }
  };
  auto close = [&]() {
    if (kOut && a.state && l.active) {
      const int64_t slot = doc_slot(a, doc);
      if (slot >= 0) {
        const int32_t N = here_uniform(a.N);
        float* s = a.state + slot * a.C * N + here(l.c) * (uint32_t)N;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < N) s[n] = h[n];
      }
    }
    if (t < t1 || t == a.S) open(doc + 1);
  };

  // Activations are requested kAhead tokens ahead (as many tokens as the loop
  // below is unrolled by), B and C one token ahead;
  // past the chunk the last token's are requested again.
  struct Raw {
    uint32_t x, dt, z;
  };
  RowBuffer bx, bd, bz, by;
  bx.open(a.x, t0, a.xs);
  bd.open(a.dt, t0, a.dts);
  bz.open(gated ? a.z : a.x, t0, gated ? a.zs : a.xs);  // without a gate nothing uses it
  by.open(a.y, t0, a.C);
  // Past a group's channels a lane's stores are out of the buffer's range,
  // which drops them.
  const uint32_t lane2 = l.c * 2u, put2 = l.active ? lane2 : 0x80000000u;
  const uint16_t* pB = a.B + t0 * a.Bs + l.group * a.bn;
  const uint16_t* pC = a.Cm + t0 * a.Cs + l.group * a.bn;
  int32_t left = t1 - t0;  // tokens not requested yet, and as many of B and C
  int32_t left_bc = left;
  auto request = [&]() {
    Raw r;
    r.x = bx.get(lane2);
    r.dt = bd.get(lane2);
    if (kOut) r.z = bz.get(lane2);
    --left;
    bx.row += left > 0 ? bx.stride : 0u;
    bd.row += left > 0 ? bd.stride : 0u;
    if (kOut) bz.row += left > 0 ? bz.stride : 0u;
    return r;
  };
  struct Rows {
    Uniform<NT> B, C;
  };
  auto request_bc = [&]() {
    Rows r;
    r.B.load(pB);
    if (kOut) r.C.load(pC);
    --left_bc;
    pB += left_bc > 0 ? a.Bs : 0;
    if (kOut) pC += left_bc > 0 ? a.Cs : 0;
    return r;
  };
  // One token.  `now` has its B and C, `then` receives the next token's:
  // scalar loads complete in no order, so the wait for `now` is placed before
  // `then` is requested, and nothing waits for `then` until its own token.
  auto token = [&](const Raw& r, const Rows& now, Rows& then) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    then = request_bc();
    __builtin_amdgcn_sched_barrier(0);
    const float x = bf16_lo(r.x);
    const float d = step_size(a, bf16_lo(r.dt), bias);
    const float dx = d * x;
    float y = Dc * x;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      h[n] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[n]), h[n], dx * now.B.get(n));
      if (kOut) y = __builtin_fmaf(now.C.get(n), h[n], y);
    }
    if (kOut) {
      if (gated) {
        const float z = bf16_lo(r.z);
        y *= z * sigmoid_f32(z);
      }
      by.put(put2, bf16_of(y));
      by.row += by.stride;
    } else {
      sum += d;
    }
  };

  Raw q[kAhead];
  Rows bc[2];
  if (t0 < t1) {
    bc[0] = request_bc();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) q[i] = request();
  }
  const int32_t i = first_at_least(a.cu, a.num_docs + 1, t0);
  if (i <= a.num_docs && uniform_at(a.cu, i) == t0) {
    open(i);
  } else {
    doc = i - 1;
    next = doc >= 0 && doc < a.num_docs ? uniform_at(a.cu, doc + 1) : INT32_MAX;
    if (kOut && k > 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < a.N) h[n] = row(a.hend, k - 1, n)[l.col];
    }
  }

#pragma unroll 1
  while (t < t1) {
    const int32_t end = next > t && next < t1 ? next : t1;
    static_assert(kAhead % 2 == 0, "two rows of B and C in turn");
#pragma unroll 1
    for (; t + kAhead <= end; t += kAhead) {
      pB = uniform(pB);
      pC = uniform(pC);
      bc[0].B.pin();
      if (kOut) bc[0].C.pin();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const Raw r = q[i];
        q[i] = request();
        token(r, bc[i % 2], bc[1 - i % 2]);
      }
    }
#pragma unroll 1
    for (; t < end; ++t) {
      const Raw r = q[0];
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) q[i] = q[i + 1];
      q[kAhead - 1] = request();
      token(r, bc[0], bc[1]);
      bc[0] = bc[1];
    }
    if (t == next && doc >= 0 && doc < a.num_docs) close();
  }
  if (!kOut) {
    const int32_t kk = here_uniform(k), N = here_uniform(a.N);
    const uint32_t col = here(l.col);
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n < N) row(a.hend, kk, n)[col] = h[n];
    (a.sum + (int64_t)k * a.cols)[l.col] = sum;
    if (w == 0 && (threadIdx.x & 63) == 0) a.flags[k] = flags;
  }
}

// Joins the chunks: forward in time the states after each chunk, and for the
// backward (blockIdx.z = 1) against it the gradients that leave each chunk.
// A lane has one column and state.  The chain is short, the loads are what
// takes time: the waves of a workgroup have kJoin chunks each, all requested
// at once and the next ones ahead, and tell each other through LDS what their
// chunks do to what comes in.  64 chunks, C = 4096, 16 states: 12 us in one
// direction; 65 chunks, C = 520, 8 states: 4.3 us, where one wave alone took 9.9.
constexpr int kJoin = 8, kJoinWaves = 8;

__global__ __launch_bounds__(64 * kJoinWaves) void scan_join_kernel(ScanArgs a) {
  struct Piece {
    float decay[64], own[64];
    int32_t apart;  // a document starts in it: what comes in does not pass
  };
  __shared__ Piece pieces[2][kJoinWaves];
  const int32_t lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
  const int32_t col = blockIdx.x * 64 + lane, n = blockIdx.y;
  const int32_t g = col / (a.wpg * 64), i = col - g * a.wpg * 64;
  const bool active = i < a.per;  // columns without a channel are read and not written
  const float A2 = active ? param_at(a.A, a.A_bf16, ((int64_t)g * a.per + i) * a.N + n) * kLog2E : 0.0f;
  const bool back = blockIdx.z == 1;
  float* v = (back ? a.mu : a.hend) + (int64_t)n * a.cols + col;
  const int64_t row = (int64_t)a.rows * a.cols;
  const int32_t steps = a.chunks - 1;
  struct Batch {
    float own[kJoin], sum[kJoin];
    int32_t flags[kJoin];
  };
  auto chunk_at = [&](int32_t s) { return back ? a.chunks - 1 - s : s; };
  auto load = [&](int32_t s0) {
    Batch r;
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      const int32_t k = chunk_at(min(s0 + j, steps - 1));
      r.own[j] = v[k * row];
      r.sum[j] = a.sum[(int64_t)k * a.cols + col];
      r.flags[j] = uniform_at(a.flags, k);
    }
    return r;
  };
  // What passes a chunk or several; 0 times an infinite decay is 0.
  auto pass = [](bool apart, float decay, float in, float own) {
    return !apart && in != 0.0f ? __builtin_fmaf(decay, in, own) : own;
  };
  float carry = 0.0f;
  Batch next = load(w * kJoin);
#pragma unroll 1
  for (int32_t s0 = 0, turn = 0; s0 < steps; s0 += kJoin * kJoinWaves, turn ^= 1) {
    const int32_t s = s0 + w * kJoin;
    const Batch now = next;
    if (s0 + kJoin * kJoinWaves < steps) next = load(s + kJoin * kJoinWaves);
    float decay[kJoin], sums = 0.0f, own = 0.0f;
    int32_t apart = 0;
    auto step = [&](int j, float in) {
      const int32_t f = now.flags[j];
      const float out = pass(f != 0, decay[j], in, now.own[j]);
      return back && (f & 1) ? 0.0f : out;  // nothing leaves a chunk that a document starts with
    };
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      decay[j] = __builtin_amdgcn_exp2f(A2 * now.sum[j]);
      own = step(j, own);
      sums += now.sum[j];
      apart |= now.flags[j];
    }
    Piece* const p = pieces[turn];
    // Of the sum and not a product: with steps of either sign one chunk's decay
    // may be 0 and the next one's infinite, whose product is no number.
    p[w].decay[lane] = __builtin_amdgcn_exp2f(A2 * sums);
    p[w].own[lane] = own;
    if (lane == 0) p[w].apart = apart;
    __syncthreads();
    float in = carry;
#pragma unroll
    for (int u = 0; u < kJoinWaves; ++u) {
      if (u == w) in = carry;
      carry = pass(p[u].apart != 0, p[u].decay[lane], carry, p[u].own[lane]);
    }
#pragma unroll
    for (int j = 0; j < kJoin; ++j) {
      in = step(j, in);
      if (active && s + j < steps) v[chunk_at(s + j) * row] = in;
    }
  }
}

// ------------------------------------------------------------- backward --
//
// With g = dy silu(z) and lambda[t] the gradient at h[t]:
//
//   lambda[t] = C[t] g[t] + exp(d[t+1] A) lambda[t+1]
//   v[t]      = lambda[t] exp(d[t] A) h[t-1]
//   dx = D g + d sum_n lambda B      dd  = x sum_n lambda B + sum_n v A
//   dB = sum_c lambda d x            dC  = sum_c g h
//   dA = sum_t v d                   dD  = sum_t g x
//
// A pass over the chunks first (scan_bwd_local) leaves each chunk's state from
// zero history, the gradient its own tokens send to its left, and the state
// every kScanKeep tokens; both are joined; the main pass then runs every
// chunk backwards from what its neighbours send.

// Forward over a chunk from zero history.  With p the decay since the chunk's
// start, the gradient that leaves to the left is sum_t p[t] C[t] g[t] over the
// tokens of the chunk's first document.  16384 tokens, C = 4096, 16 states: 336
// us, VALU busy 86% of the time; it writes 0.59 GB, the kept states, meanwhile.
template <int NT>
__global__ __launch_bounds__(64 * kWaves)
__attribute__((amdgpu_waves_per_eu(NT <= 16 ? 4 : NT == 32 ? 2 : 1)))
void scan_bwd_local_kernel(ScanArgs a, int32_t work) {
  constexpr int kAhead = 2;
  static_assert(kAhead % 2 == 0, "two rows of B and C in turn");
  const int32_t place = place_of(work);
  if (place < 0) return;
  const int32_t waves = a.G * a.wpg;
  const int32_t k = place / waves, w = place - k * waves;
  const Column l = column_of(a, w);
  const int32_t t0 = k * a.chunk;
  const int32_t t1 = (int32_t)min((int64_t)a.S, (int64_t)t0 + a.chunk);
  float A2[NT], h[NT], mu[NT], p[NT];
  load_decay<NT>(a, l, A2);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    h[n] = 0.0f, mu[n] = 0.0f, p[n] = 1.0f;
    A2[n] = l.active ? A2[n] : 0.0f;
  }
  const float bias = l.active ? step_bias(a, l.c) : 0.0f;
  const bool gated = a.z != nullptr;
  float sum = 0.0f;

  struct Raw {
    uint32_t x, dt, dy, z;
  };
  RowBuffer bx, bd, bg, bz;
  bx.open(a.x, t0, a.xs);
  bd.open(a.dt, t0, a.dts);
  bg.open(a.dy, t0, a.dys);
  bz.open(gated ? a.z : a.x, t0, gated ? a.zs : a.xs);  // without a gate nothing uses it
  const uint16_t* pB = a.B + t0 * a.Bs + l.group * a.bn;
  const uint16_t* pC = a.Cm + t0 * a.Cs + l.group * a.bn;
  // Past a group's channels a lane reads zeros (out of the buffers' range), and
  // its state and gradient, which the main pass reads, stay zero, as do those
  // past the last state.
  const uint32_t lane2 = l.active ? l.c * 2u : 0x80000000u;
  int32_t left = t1 - t0, left_bc = left;
  auto request = [&]() {
    Raw r;
    r.x = bx.get(lane2);
    r.dt = bd.get(lane2);
    r.dy = bg.get(lane2);
    r.z = bz.get(lane2);
    --left;
    bx.row += left > 0 ? bx.stride : 0u;
    bd.row += left > 0 ? bd.stride : 0u;
    bg.row += left > 0 ? bg.stride : 0u;
    bz.row += left > 0 ? bz.stride : 0u;
    return r;
  };
  struct Rows {
    Uniform<NT> B, C;
  };
  auto request_bc = [&]() {
    Rows r;
    r.B.load(pB);
    r.C.load(pC);
    --left_bc;
    pB += left_bc > 0 ? a.Bs : 0;
    pC += left_bc > 0 ? a.Cs : 0;
    return r;
  };
  auto token = [&](const Raw& r, const Rows& now, Rows& then) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), as in the forward
    then = request_bc();
    __builtin_amdgcn_sched_barrier(0);
    const float d = step_size(a, bf16_lo(r.dt), bias);
    const float dx = d * bf16_lo(r.x);
    sum += d;
    float g = bf16_lo(r.dy);
    if (gated) {
      const float z = bf16_lo(r.z);
      g *= z * sigmoid_f32(z);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float e = __builtin_amdgcn_exp2f(d * A2[n]);
      h[n] = __builtin_fmaf(e, h[n], dx * now.B.get(n));
      p[n] *= e;
      mu[n] = __builtin_fmaf(p[n], g * now.C.get(n), mu[n]);
      settled(h[n], p[n], mu[n]);
    }
  };
  // Past the first document mu is written and what it goes on to gather is
  // never used.
  bool in_first = true;
  auto write_mu = [&]() {
    const uint32_t col = here(l.col);
    const int32_t kk = here_uniform(k);
#pragma unroll
    for (int n = 0; n < NT; ++n) (a.mu + ((int64_t)kk * NT + n) * a.cols)[col] = mu[n];
  };

  Raw q[kAhead];
  Rows bc[2];
  bc[0] = request_bc();
#pragma unroll
  for (int i = 0; i < kAhead; ++i) q[i] = request();
  // The next document start behind t0.
  int32_t doc = first_at_least(a.cu, a.num_docs + 1, t0);
  int32_t flags = doc <= a.num_docs && uniform_at(a.cu, doc) == t0 ? 1 : 0;
  int32_t next = t0;
  auto advance = [&](int32_t t) {
    while (doc <= a.num_docs && uniform_at(a.cu, doc) <= t) ++doc;
    next = doc <= a.num_docs ? uniform_at(a.cu, doc) : INT32_MAX;
  };
  advance(t0);

  // The state before token t, every kScanKeep tokens.
  auto keep = [&](int32_t t) {
    if ((t - t0) % kScanKeep != 0 || t == t0) return;
    const uint32_t col = here(l.col);
    float* r = a.keep + (int64_t)(t / kScanKeep) * (NT + 1) * a.cols;
#pragma unroll
    for (int n = 0; n < NT; ++n) (r + (int64_t)n * a.cols)[col] = h[n];
    (r + (int64_t)NT * a.cols)[col] = sum;
  };

  int32_t t = t0;
#pragma unroll 1
  while (t < t1) {
    const int32_t end = min(next, t1);
#pragma unroll 1
    for (; t + kAhead <= end; t += kAhead) {
      pB = uniform(pB);
      pC = uniform(pC);
      bc[0].B.pin();
      bc[0].C.pin();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        keep(t + i);
        const Raw r = q[i];
        q[i] = request();
        token(r, bc[i % 2], bc[1 - i % 2]);
      }
    }
#pragma unroll 1
    for (; t < end; ++t) {
      keep(t);
      const Raw r = q[0];
#pragma unroll
      for (int j = 0; j + 1 < kAhead; ++j) q[j] = q[j + 1];
      q[kAhead - 1] = request();
      token(r, bc[0], bc[1]);
      bc[0] = bc[1];
    }
    if (t < t1) {  // a document starts
      flags |= 2;
      if (in_first) write_mu();
      in_first = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) h[n] = 0.0f;
      advance(t);
    }
  }
  const uint32_t col = here(l.col);
#pragma unroll
  for (int n = 0; n < NT; ++n) (a.hend + ((int64_t)k * NT + n) * a.cols)[col] = h[n];
  if (in_first) write_mu();
  (a.sum + (int64_t)k * a.cols)[col] = sum;
  if (w == 0 && (threadIdx.x & 63) == 0) a.flags[k] = flags;
}

// ---- the main pass
//
// Document starts of a chunk are a bitmask in LDS, one for each wave: bit i
// for token t0 + i, the token after the chunk's last included.
struct Starts {
  uint32_t bits[kScanMaxChunk / 32 + 2];
};

// Orders a wave's own LDS writes before its lanes' reads.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Returns the first start at or behind t0 as an offset from it.
__device__ __forceinline__ int32_t find_starts(const ScanArgs& a, Starts& m, int32_t t0, int32_t t1) {
  const int32_t lane = threadIdx.x & 63;
  const int32_t words = (t1 - t0) / 32 + 2;
  for (int32_t i = lane; i < words; i += 64) m.bits[i] = 0u;
  wave_sync();
  const int32_t at = first_at_least(a.cu, a.num_docs + 1, t0);
  for (int64_t i = (int64_t)at + lane; i <= a.num_docs; i += 64) {
    const int32_t v = a.cu[i];
    if (v > t1) break;
    if (v >= t0) atomicOr(&m.bits[(v - t0) >> 5], 1u << ((v - t0) & 31));
  }
  wave_sync();
  return at <= a.num_docs ? uniform_at(a.cu, at) - t0 : INT32_MAX;
}

// Bits i .. i + 31 of the mask, in a scalar register.
__device__ __forceinline__ uint32_t starts_from(const Starts& m, int32_t i) {
  return uniform(__builtin_amdgcn_alignbit(m.bits[(i >> 5) + 1], m.bits[i >> 5], (uint32_t)i & 31u));
}

// A lane's tile: RC channels x RN states.  P lanes share a channel set:
// lane = P * set + part, states RN * part .. of channels RC * set .. .  More
// states a lane make the sums over states cheap, more channels those over
// channels; two lanes a channel cost the fewest instructions of both (for 16
// states: 9 + 6 + 34 a token for the sums over states, the broadcasts within
// a set and the sums over channels; four lanes 27 + 12 + 16, one lane 70).
template <int NT>
struct Tile {
  static constexpr int P = NT <= 32 ? 2 : 4;
  static constexpr int RN = NT / P;
  static constexpr int RC = NT <= 16 ? 2 : 1;
  static constexpr int CB = 64 / P * RC;  // channels of a wave
};

// The value of a set's lane r.
template <int P, int R>
__device__ __forceinline__ float set_from(float v) {
  return dpp<(P == 2 ? 0xa0 : 0) + R * 0x55>(v);
}
template <int P, int RC>
__device__ __forceinline__ void set_spread(float v, float (&o)[RC]) {
  o[0] = set_from<P, 0>(v);
  if constexpr (RC > 1) o[1] = set_from<P, 1>(v);
}

// Sum over a set's lanes of the lane's own channel's value.
template <int P, int RC>
__device__ __forceinline__ float set_sum(const float (&v)[RC], bool odd) {
  if constexpr (RC == 2) {
    const float keep = odd ? v[1] : v[0], send = odd ? v[0] : v[1];
    return keep + dpp<kXor1>(send);
  } else {
    float s = v[0] + dpp<kXor1>(v[0]);
    if constexpr (P == 4) s += dpp<kXor2>(s);
    return s;
  }
}

// Sums RN values over the sets of a wave.  The upper half of the wave takes
// over half of the values from the lower and gives up the other half, the odd
// rows of 16 lanes likewise (each value then costs half an exchange and half
// an addition), and the rest is added within rows.  Value
// (lane / 32) * RN / 2 + (lane / 16 % 2) * RN / 4 + i is left in v[i], i < RN / 4.
template <int P, int RN>
__device__ __forceinline__ void sets_sum(float (&v)[RN]) {
#pragma unroll
  for (int i = 0; i < RN / 2; ++i) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + RN / 2]),
                                                    false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
#pragma unroll
  for (int i = 0; i < RN / 4; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[i + RN / 4]),
                                                    false, false);
    float x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    x += dpp<kRor8>(x);
    x += dpp<kRor4>(x);
    if constexpr (P == 2) x += dpp<kXor2>(x);
    v[i] = x;
  }
}

// a b + c where c is needed afterwards: written out, as the compiler copies c
// and adds to the copy.  No operand may come straight from an exponential, a
// reciprocal or a root, whose results take a cycle more.
__device__ __forceinline__ float fma_apart(float a, float b, float c) {
  float r;
  asm("v_fma_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Sets eight values to zero where the uniform `bit` is set, which it hardly
// ever is.  As control flow of the compiler's own this would cost a copy of
// the values on the usual path, to bring both into the same registers.
__device__ __forceinline__ void zero_if(uint32_t bit, float& a, float& b, float& c, float& d, float& e,
                                        float& f, float& g, float& h) {
  asm volatile(
      "s_cmp_eq_u32 %8, 0\n\t"
      "s_cbranch_scc1 .Lkeep%=\n\t"
      "v_mov_b32 %0, 0\n\tv_mov_b32 %1, 0\n\tv_mov_b32 %2, 0\n\tv_mov_b32 %3, 0\n\t"
      "v_mov_b32 %4, 0\n\tv_mov_b32 %5, 0\n\tv_mov_b32 %6, 0\n\tv_mov_b32 %7, 0\n"
      ".Lkeep%=:"
      : "+v"(a), "+v"(b), "+v"(c), "+v"(d), "+v"(e), "+v"(f), "+v"(g), "+v"(h)
      : "s"(bit)
      : "scc");
}

// Runs a chunk backwards in blocks of kScanKeep tokens.  A block's states are
// computed forward from its kept start twice: once for the starts of its
// sub-blocks of kSub tokens (to LDS, each lane its own), then for each
// sub-block, whose decays a and decayed states ah = a h[t-1] stay in registers
// for the way back.  h itself is ah + d x B: its part in y and in dC needs only
// sum_n C B and sum_c g d x, one number a token each.
//
// States kept every 8 tokens are 1/8 of all of them: 0.55 GB written and read at
// 16384 tokens, C = 4096, 16 states, behind the arithmetic.  Kept every 2 they
// would save the first of the two ways forward, 14% of this kernel, and move 2.1
// GB each way, which takes as long.  That size takes 936 us: 424 VALU instructions
// a token and 64 channels, of which the formulas above are 240, VALU busy 88% of
// the time.
//
// Two waves a SIMD up to 32 states; 64 states need one wave's registers.
constexpr int kSub = 2;

template <int NT, bool kGate>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(NT <= 32 ? 2 : 1)))
void scan_bwd_main_kernel(ScanArgs a, int32_t work) {
  typedef Tile<NT> T;
  constexpr int P = T::P, RN = T::RN, RC = T::RC, CB = T::CB, kSubs = kScanKeep / kSub;
  struct Lds {
    Starts starts;
    f32x4_t h[kSubs - 1][RC * RN / 4][64];  // states before the sub-blocks but the last
    f32x4_t in[RC * RN / 4][64];            // what came into the chunk
    float step[kScanKeep - kSub][64];       // step sizes of the tokens but the last sub-block's
    float bc[kScanKeep][2][NT];       // B and C of the block's tokens
    float cb[kScanKeep];              // sum_n C B
  };
  __shared__ __align__(16) Lds lds[kWaves];
  const int32_t place = place_of(work);
  if (place < 0) return;
  Lds& m = lds[threadIdx.x / 64u];
  const int32_t lane = threadIdx.x & 63, part = lane % P, set = lane / P;
  const int32_t bpg = (a.per + CB - 1) / CB, blocks = a.G * bpg;
  const int32_t k = place / blocks, wb = place - k * blocks;
  const int32_t g = wb / bpg, i0 = (wb - g * bpg) * CB;
  const int32_t t0 = k * a.chunk;
  const int32_t t1 = (int32_t)min((int64_t)a.S, (int64_t)t0 + a.chunk);
  // The channel whose loads and per-channel terms are this lane's.  A channel
  // past the group reads zeros (out of the buffers' range): its x, g, h and
  // lambda stay zero and add nothing.
  const int32_t mine = part % RC;
  const bool odd = part & 1;
  const bool active = i0 + RC * set + mine < a.per;
  const uint32_t c = (uint32_t)(g * a.per + (active ? i0 + RC * set + mine : 0));
  const float Dc = active && a.D ? param_at(a.D, a.D_bf16, c) : 0.0f;
  float bias = step_bias(a, c);
  if (!active) bias = 0.0f;
  const uint32_t col = (uint32_t)(g * a.wpg * 64 + i0 + RC * set);
  const int32_t n0 = RN * part;

  // The lane's tile of NT rows of the workspace, whose states past the last and
  // columns past a group hold zeros; the host keeps the rows below 2^31 bytes.
  const uint32_t stride4 = (uint32_t)a.cols * 4u;
  auto tile = [&](const float* rows, uint32_t at4, float (&o)[RC][RN]) {
    const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(rows), (short)0, 0x7fffffff, 0x00020000);
    const uint32_t lane4 = (uint32_t)n0 * stride4 + at4;
#pragma unroll
    for (int j = 0; j < RN; ++j) {
      if constexpr (RC == 2) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b64(b, (int)lane4, (int)(j * stride4), 0);
        o[0][j] = __uint_as_float(v[0]);
        o[1][j] = __uint_as_float(v[1]);
      } else {
        o[0][j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)lane4, (int)(j * stride4), 0));
      }
    }
  };
  const int64_t chunk_rows = (int64_t)NT * a.cols;
  float dD = 0.0f, dbias = 0.0f;
  constexpr float kLn2 = 0.6931471805599453f;

  RowBuffer bx, bd, bg, bz, ox, od, oz;
  bx.open(a.x, t0, a.xs);
  bd.open(a.dt, t0, a.dts);
  bg.open(a.dy, t0, a.dys);
  bz.open(kGate ? a.z : a.x, t0, kGate ? a.zs : a.xs);
  ox.open(a.dx, t0, a.C);
  od.open(a.ddt, t0, a.C);
  oz.open(kGate ? a.dz : a.dx, t0, a.C);
  const uint32_t get2 = active ? c * 2u : 0x80000000u, put2 = part < RC ? get2 : 0x80000000u;
  const int32_t last = t1 - t0 - 1;  // tokens are counted from t0 from here on
  auto get = [&](const RowBuffer& b, int32_t i) {
    return (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b.r, (int)get2, (int)((uint32_t)min(i, last) * b.stride), 0);
  };
  auto put = [&](const RowBuffer& b, int32_t i, float v) {  // past the end: out of range, dropped
    const uint32_t row = i <= last ? (uint32_t)i * b.stride : 0x7fffffffu;
    __builtin_amdgcn_raw_buffer_store_b16(bf16_of(v), b.r, (int)put2, (int)row, 0);
  };
  // The activations of a sub-block's tokens, requested one sub-block ahead.
  struct Raw {
    uint32_t x, dt, dy, z;
  };
  Raw q[kSub];
  auto request = [&](int32_t i, bool back) {
#pragma unroll
    for (int j = 0; j < kSub; ++j) {
      q[j].x = get(bx, i + j);
      q[j].dt = get(bd, i + j);
    }
    if (back) {
#pragma unroll
      for (int j = 0; j < kSub; ++j) {
        q[j].dy = get(bg, i + j);
        if (kGate) q[j].z = get(bz, i + j);
      }
    }
  };
  float h[RC][RN];
  auto reset_if = [&](uint32_t bit, float (&v)[RC][RN]) {
#pragma unroll
    for (int e = 0; e < RC * RN; e += 8)
      zero_if(bit, v[e / RN][e % RN], v[(e + 1) / RN][(e + 1) % RN], v[(e + 2) / RN][(e + 2) % RN],
              v[(e + 3) / RN][(e + 3) % RN], v[(e + 4) / RN][(e + 4) % RN], v[(e + 5) / RN][(e + 5) % RN],
              v[(e + 6) / RN][(e + 6) % RN], v[(e + 7) / RN][(e + 7) % RN]);
  };
  auto states = [&](const float* row, float (&o)[RN]) {
#pragma unroll
    for (int j = 0; j < RN; j += 4) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(row + n0 + j);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e < RN) o[j + e] = v[e];
    }
  };

  // What a block starts from, requested while the block behind it is at work:
  // its B and C, its kept state (to h, which is free then) and the sum of the
  // step sizes before it.
  constexpr int kRaw = kScanKeep * 2 * NT / 64;
  uint32_t raw_bc[kRaw];
  float sum[RC];
  // Lane e of 2 NT: state e of B, state e - NT of C.
  const bool is_c = lane / NT % 2;
  const uint32_t bc_stride = (uint32_t)(is_c ? a.Cs : a.Bs);
  const uint16_t* const bc = (is_c ? a.Cm + t0 * a.Cs : a.B + t0 * a.Bs) + g * a.N + min(lane % NT, a.N - 1);
  auto request_block = [&](int32_t ib) {
    const int32_t i_first = ib * kScanKeep;
    const uint32_t at = here(col);
    const uint32_t stride = here(bc_stride);
#pragma unroll
    for (int u = 0; u < kRaw; ++u) {
      if constexpr (NT < 64) {
        const uint32_t i = (uint32_t)min(i_first + (lane + 64 * u) / (2 * NT), last);
        raw_bc[u] = bc[(uint64_t)i * stride];
      } else {  // a row of B or of C a wave
        const int64_t i = t0 + min(i_first + u / 2, last);
        raw_bc[u] = ((u % 2 ? a.Cm + i * a.Cs : a.B + i * a.Bs) + g * a.N)[min(lane, a.N - 1)];
      }
    }
    if (ib > 0) {
      const float* kept = a.keep + (int64_t)((t0 + i_first) / kScanKeep) * (NT + 1) * a.cols;
      tile(kept, at * 4u, h);
#pragma unroll
      for (int r = 0; r < RC; ++r) sum[r] = (kept + chunk_rows)[at + r];
    }
  };

  // The first block's loads before all the others that a wave begins with.
  request(last / kScanKeep * kScanKeep, last % kScanKeep < kSub);
  request_block(last / kScanKeep);
  const int32_t first_start = find_starts(a, m.starts, t0, t1);
  // A times log2(e); the sums with A are taken with it and scaled at their end.
  // Loads without a condition, all under way at once: what is past the group or
  // the states is read at the last of them and not used.
  float A2[RC][RN], mu[RC][RN], dA[RC][RN];
  auto decays = [&](auto* A) {
#pragma unroll
    for (int r = 0; r < RC; ++r) {
      const uint32_t row = (uint32_t)(g * a.per + min(i0 + RC * set + r, a.per - 1)) * (uint32_t)a.N;
#pragma unroll
      for (int j = 0; j < RN; ++j) {
        const auto v = A[row + (uint32_t)min(n0 + j, a.N - 1)];
        if constexpr (sizeof(v) == 2) A2[r][j] = bf16_f32(v);
        else A2[r][j] = v;
      }
    }
  };
  if (a.A_bf16) decays(static_cast<const uint16_t*>(a.A));
  else decays(static_cast<const float*>(a.A));
#pragma unroll
  for (int r = 0; r < RC; ++r)
#pragma unroll
    for (int j = 0; j < RN; ++j) {
      A2[r][j] = i0 + RC * set + r < a.per && n0 + j < a.N ? A2[r][j] * kLog2E : kNoState;
      mu[r][j] = dA[r][j] = 0.0f;
    }
  // What the chunk to the right sends; nothing where a document starts with it.
  // (The join clears such a chunk's rows, but for states past the last and
  // columns past the group, where 0 times an infinity may have left a NaN.)
  if (k + 1 < a.chunks && !(starts_from(m.starts, t1 - t0) & 1u)) tile(a.mu + (k + 1) * chunk_rows, col * 4u, mu);
  if (k > 0) {
    float in[RC][RN];
    tile(a.hend + (k - 1) * chunk_rows, col * 4u, in);
#pragma unroll
    for (int e = 0; e < RC * RN; e += 4)
      m.in[e / 4][lane] = (f32x4_t){in[e / RN][e % RN], in[e / RN][e % RN + 1], in[e / RN][e % RN + 2],
                                    in[e / RN][e % RN + 3]};
  }
#pragma unroll 1
  for (int32_t ib = last / kScanKeep; ib >= 0; --ib) {
    const int32_t i_first = ib * kScanKeep;
    const int32_t subs = min(kSubs, (last - i_first) / kSub + 1);  // sub-blocks that have tokens
    // Bit i: a document starts at the block's token i.
    const uint32_t starts = starts_from(m.starts, i_first);
    wave_sync();
#pragma unroll
    for (int u = 0; u < kRaw; ++u) {
      const int32_t e = lane + 64 * u;
      (&m.bc[0][0][0])[e] = e % NT < a.N ? bf16_lo(raw_bc[u]) : 0.0f;
    }
    wave_sync();
    {
      static_assert(kScanKeep == 8, "eight lanes a token");
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < NT / 8; ++j)
        s = __builtin_fmaf(m.bc[lane / 8][0][lane % 8 + 8 * j], m.bc[lane / 8][1][lane % 8 + 8 * j], s);
      s += dpp<kXor1>(s);
      s += dpp<kXor2>(s);
      s += dpp<kHalfMirror>(s);
      if (lane % 8 == 0) m.cb[lane / 8] = s;
    }
    wave_sync();
    // The state before the block: kept from zero history, plus what came into
    // the chunk, decayed, if no document has started since.
    {
      if (ib == 0) {
#pragma unroll
        for (int r = 0; r < RC; ++r) {
          sum[r] = 0.0f;
#pragma unroll
          for (int j = 0; j < RN; ++j) h[r][j] = 0.0f;
        }
      }
      if (k > 0 && first_start >= i_first) {
#pragma unroll
        for (int e = 0; e < RC * RN; e += 4) {
          const f32x4_t in = m.in[e / 4][lane];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = (e + q) / RN, j = (e + q) % RN;
            // Finite, so that nothing that came in stays nothing.
            const float decay = __builtin_fminf(__builtin_amdgcn_exp2f(A2[r][j] * sum[r]), FLT_MAX);
            h[r][j] = __builtin_fmaf(decay, in[q], h[r][j]);
          }
        }
      }
    }
    // Forward over sub-block s, for the state behind it.
    auto forward = [&](int32_t s) {
      Raw v[kSub];
#pragma unroll
      for (int i = 0; i < kSub; ++i) v[i] = q[i];
      request(i_first + (s + 1) * kSub, s + 2 == subs);
#pragma unroll
      for (int e = 0; e < RC * RN; e += 4)
        m.h[s][e / 4][lane] = (f32x4_t){h[e / RN][e % RN], h[e / RN][e % RN + 1], h[e / RN][e % RN + 2],
                                        h[e / RN][e % RN + 3]};
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        const int32_t at = s * kSub + i;
        reset_if((starts >> at) & 1u, h);
        const float own = step_size(a, bf16_lo(v[i].dt), bias);
        m.step[at][lane] = own;
        float B[RN], d[RC], dx[RC];
        states(m.bc[at][0], B);
        set_spread<P, RC>(own, d);
        set_spread<P, RC>(own * bf16_lo(v[i].x), dx);
#pragma unroll
        for (int r = 0; r < RC; ++r)
#pragma unroll
          for (int j = 0; j < RN; ++j)
            h[r][j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[r] * A2[r][j]), h[r][j], dx[r] * B[j]);
      }
    };
    // Sub-block s forward once more from the state before it, then backward.
    auto backward = [&](int32_t s) {
      const int32_t at0 = s * kSub;
      Raw v[kSub];
#pragma unroll
      for (int i = 0; i < kSub; ++i) v[i] = q[i];
      request(s > 0 ? i_first + (s - 1) * kSub : max(i_first - kScanKeep, 0), s > 0);
      float aw[kSub][RC][RN], hw[kSub][RC][RN];
      float own[kSub];  // step sizes, of all but the last sub-block as the way forward left them
      if (s + 1 < subs) {
#pragma unroll
        for (int i = 0; i < kSub; ++i) own[i] = m.step[at0 + i][lane];
      } else {
#pragma unroll
        for (int i = 0; i < kSub; ++i) own[i] = step_size(a, bf16_lo(v[i].dt), bias);
      }
#pragma unroll
      for (int i = 0; i < kSub; ++i) {
        reset_if((starts >> (at0 + i)) & 1u, h);
        // A token past the end does nothing: no step, and no gradient below.
        own[i] = i_first + at0 + i <= last ? own[i] : 0.0f;
        float B[RN], d[RC], dx[RC];
        states(m.bc[at0 + i][0], B);
        set_spread<P, RC>(own[i], d);
        set_spread<P, RC>(own[i] * bf16_lo(v[i].x), dx);
#pragma unroll
        for (int r = 0; r < RC; ++r)
#pragma unroll
          for (int j = 0; j < RN; ++j) {
            aw[i][r][j] = __builtin_amdgcn_exp2f(d[r] * A2[r][j]);
            hw[i][r][j] = aw[i][r][j] * h[r][j];
            h[r][j] = fma_apart(dx[r], B[j], hw[i][r][j]);
          }
      }
      if (s == 0 && ib > 0) request_block(ib - 1);
#pragma unroll
      for (int i = kSub - 1; i >= 0; --i) {
        const int32_t at = at0 + i, tok = i_first + at;
        const bool real = tok <= last;
        const float x = bf16_lo(v[i].x), dy = real ? bf16_lo(v[i].dy) : 0.0f;
        float gy = dy, z = 0.0f, sz = 0.0f;
        if (kGate) {
          z = bf16_lo(v[i].z);
          sz = sigmoid_f32(z);
          gy *= z * sz;
        }
        const float own_dx = own[i] * x;
        float B[RN], Cm[RN], d[RC], dx[RC], gr[RC];
        states(m.bc[at][0], B);
        states(m.bc[at][1], Cm);
        set_spread<P, RC>(own[i], d);
        set_spread<P, RC>(own_dx, dx);
        set_spread<P, RC>(gy, gr);
        float dB[RN], dC[RN], lb[RC], va[RC], y0[RC];
        auto add = [](bool first, float a, float b, float& sum) {
          sum = first ? a * b : __builtin_fmaf(a, b, sum);
        };
#pragma unroll
        for (int r = 0; r < RC; ++r) {
#pragma unroll
          for (int j = 0; j < RN; ++j) {
            const float lam = __builtin_fmaf(gr[r], Cm[j], mu[r][j]);
            const float w = lam * hw[i][r][j];
            if (kGate) add(j == 0, Cm[j], hw[i][r][j], y0[r]);
            add(j == 0, lam, B[j], lb[r]);
            add(j == 0, w, A2[r][j], va[r]);
            dA[r][j] = __builtin_fmaf(w, d[r], dA[r][j]);
            add(r == 0, lam, dx[r], dB[j]);
            add(r == 0, gr[r], hw[i][r][j], dC[j]);
            mu[r][j] = aw[i][r][j] * lam;
          }
        }
        reset_if((starts >> at) & 1u, mu);
        const float slb = set_sum<P, RC>(lb, odd), sva = set_sum<P, RC>(va, odd) * kLn2;
        float ddt = __builtin_fmaf(x, slb, sva);
        if (a.softplus) ddt *= sigmoid_f32(bf16_lo(v[i].dt) + bias);
        dD = __builtin_fmaf(gy, x, dD);
        dbias += real ? ddt : 0.0f;
        put(ox, tok, __builtin_fmaf(Dc, gy, own[i] * slb));
        put(od, tok, ddt);
        if (kGate) {
          const float y = __builtin_fmaf(own_dx, m.cb[at], set_sum<P, RC>(y0, odd));
          put(oz, tok, dy * __builtin_fmaf(Dc, x, y) * dsilu_f32(z, sz));
        }
        const float gdx = lanes_sum<64>(part < RC ? gy * own_dx : 0.0f);
        sets_sum<P, RN>(dB);
        sets_sum<P, RN>(dC);
        if ((lane & 15) < P && real) {
          const int32_t n = n0 + (lane >> 5) * (RN / 2) + ((lane >> 4) & 1) * (RN / 4);
          float* out = a.pbc + ((int64_t)wb * a.S + t0 + tok) * (2 * NT);
#pragma unroll
          for (int e = 0; e < RN / 4; ++e) {
            out[n + e] = dB[e];
            out[NT + n + e] = __builtin_fmaf(gdx, m.bc[at][0][n + e], dC[e]);
          }
        }
      }
    };
#pragma unroll 1
    for (int32_t s = 0; s + 1 < subs; ++s) forward(s);
#pragma unroll 1
    for (int32_t s = subs - 1; s >= 0; --s) {
      if (s + 1 < subs) {
#pragma unroll
        for (int e = 0; e < RC * RN; e += 4) {
          const f32x4_t v = m.h[s][e / 4][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[e / RN][e % RN + i] = v[i];
        }
      }
      backward(s);
    }
  }
  float* pp = a.pparam + (int64_t)k * (NT + 2) * a.cols;
#pragma unroll
  for (int r = 0; r < RC; ++r)
#pragma unroll
    for (int j = 0; j < RN; ++j) (pp + (int64_t)j * a.cols)[(uint32_t)n0 * (uint32_t)a.cols + here(col) + r] = dA[r][j];
  if (part < RC) {
    (pp + (int64_t)NT * a.cols)[col + mine] = dD;
    (pp + (int64_t)(NT + 1) * a.cols)[col + mine] = dbias;
  }
}

// dA, dD and ddt_bias: the chunks' partial rows in order, summed in FP64.
__device__ __forceinline__ void param_sum(const ScanArgs& a, int32_t col, int32_t n) {
  const int32_t g = col / (a.wpg * 64), i = col - g * a.wpg * 64;
  if (col >= a.cols || i >= a.per) return;
  // Rows: the states, then D and the bias behind the states that there is room for.
  const float* p = a.pparam + (int64_t)(n < a.N ? n : a.rows + n - a.N) * a.cols + col;
  const int64_t row = (int64_t)(a.rows + 2) * a.cols;
  double sum = 0.0;
  int32_t k = 0;
  for (; k + 16 <= a.chunks; k += 16) {  // 16 loads at once
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = p[(k + j) * row];
#pragma unroll
    for (int j = 0; j < 16; ++j) sum += v[j];
  }
  for (; k < a.chunks; ++k) sum += p[k * row];
  const int64_t c = (int64_t)g * a.per + i;
  if (n < a.N) param_put(a.dA, a.A_bf16, c * a.N + n, (float)sum);
  else if (n == a.N) {
    if (a.dD) param_put(a.dD, a.D_bf16, c, (float)sum);
  } else if (a.dbias) {
    param_put(a.dbias, a.bias_bf16, c, (float)sum);
  }
}

// dB and dC: the partial rows of a group's channel blocks, in order.  A lane
// has four values of a token's row, so that a wave reads 1 KiB of each block.
// Bound by HBM: 134 MB at 16384 tokens, 64 blocks and 16 states in 25 us.
__device__ __forceinline__ void bc_sum(const ScanArgs& a, int64_t block, int32_t bpg, int32_t NT) {
  const int64_t rows = (int64_t)a.S * 2 * NT;  // of one block
  const int64_t per = (rows / 4 + 255) / 256;  // workgroups of one group
  const int64_t g = block / per;
  const int64_t e = ((block - g * per) * 256 + threadIdx.x) * 4;
  if (e >= rows) return;
  const float* p = a.pbc + g * bpg * rows + e;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  int32_t b = 0;
  for (; b + 8 <= bpg; b += 8) {  // 8 loads at once
    f32x4_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4_t*>(p + (b + j) * rows);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[q] += v[j][q];
  }
  for (; b < bpg; ++b) {
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + b * rows);
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[q] += v[q];
  }
  const int64_t t = e / (2 * NT);
  const int32_t i = (int32_t)(e - t * 2 * NT), half = i / NT, n = i - half * NT;
  uint16_t* o = (half ? a.dC : a.dB) + (t * a.G + g) * a.N + n;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (n + q < a.N) o[q] = bf16_of(sum[q]);
}

// Both in one launch, the parameters' workgroups first.
__global__ __launch_bounds__(256) void scan_sum_kernel(ScanArgs a, int32_t bpg, int32_t NT) {
  const uint32_t cb = (uint32_t)(a.cols + 255) / 256, params = cb * (a.N + 2);
  if (blockIdx.x < params)
    param_sum(a, (int32_t)(blockIdx.x % cb * 256 + threadIdx.x), (int32_t)(blockIdx.x / cb));
  else
    bc_sum(a, blockIdx.x - params, bpg, NT);
}

// --------------------------------------------------------- single tokens --

// One token a row.  NL lanes hold a channel's states, four each, so that a
// wave reads and writes 1 KiB of states in a row; it keeps its channels' A, D
// and bias and takes `rows` rows one after another, the next row's loads
// requested before the current is computed.  kVec: N is a multiple of 4 and
// the states are 16-byte aligned.
//
// Bound by HBM: 8 bytes a state.  States are loaded and stored past the caches:
// a model's layers take turns, and by its next token a layer's states are gone
// from them.  Layers of 4096 channels and 16 states in turn: 512 rows 57 us (4.7
// TB/s) against 66 through the caches, 64 rows 10.8 against 12.8; a layer on its
// own, whose states the caches would hold, 57 against 47.
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

template <int NL, bool kVec, bool kGate>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a, int32_t rows) {
  constexpr int kChannels = 64 / NL;
  const int32_t cblocks = (a.C + kChannels - 1) / kChannels;
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
  const int64_t rb = wave / cblocks;
  const int32_t lane = threadIdx.x & 63, part = lane % NL;
  const int32_t c0 = (int32_t)(wave - rb * cblocks) * kChannels + lane / NL;
  const bool there = c0 < a.C;
  const uint32_t c = there ? c0 : 0;
  const int32_t row0 = (int32_t)min(rb * rows, (int64_t)a.S), row1 = (int32_t)min((rb + 1) * rows, (int64_t)a.S);
  const int32_t n0 = 4 * part;
  float A2[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    A2[j] = n0 + j < a.N ? param_at(a.A, a.A_bf16, (int64_t)c * a.N + n0 + j) * kLog2E : 0.0f;
  const float bias = step_bias(a, c);
  const float Dc = a.D ? param_at(a.D, a.D_bf16, c) : 0.0f;
  const uint32_t bc0 = c / (uint32_t)a.per * (uint32_t)a.N + n0;
  const uint32_t h0 = c * (uint32_t)a.N + n0;

  struct Row {
    int64_t slot;
    float h[4], b[4], c[4];
    uint16_t x, dt, z;
  };
  auto states = [&](const uint16_t* p, float (&o)[4]) {
    if (kVec) {
      const u32x2_any v = *reinterpret_cast<const u32x2_any*>(p);
      o[0] = bf16_lo(v.x), o[1] = bf16_hi(v.x), o[2] = bf16_lo(v.y), o[3] = bf16_hi(v.y);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = n0 + j < a.N ? bf16_f32(p[j]) : 0.0f;
    }
  };
  const bool some = kVec ? n0 < a.N : true;  // NL lanes may hold more than N states
  auto load = [&](int32_t row) {
    Row r;
    r.slot = slot_of(a.index, row, a.slots);
    r.x = (a.x + row * a.xs)[c];
    r.dt = (a.dt + row * a.dts)[c];
    r.z = kGate ? (a.z + row * a.zs)[c] : (uint16_t)0;
#pragma unroll
    for (int j = 0; j < 4; ++j) r.h[j] = r.b[j] = r.c[j] = 0.0f;
    if (r.slot >= 0 && some) {
      states(a.B + row * a.Bs + bc0, r.b);
      states(a.Cm + row * a.Cs + bc0, r.c);
      const float* h = a.state + r.slot * a.C * a.N + h0;
      if (kVec) {
        const f32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(h));
#pragma unroll
        for (int j = 0; j < 4; ++j) r.h[j] = v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.h[j] = n0 + j < a.N ? h[j] : 0.0f;
      }
    }
    return r;
  };
  if (row0 >= row1) return;
  Row next = load(row0);
#pragma unroll 1
  for (int32_t row = row0; row < row1; ++row) {
    Row r = next;
    if (row + 1 < row1) next = load(row + 1);
    float y = 0.0f;
    if (r.slot >= 0) {
      const float x = bf16_f32(r.x), d = step_size(a, bf16_f32(r.dt), bias), dx = d * x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d * A2[j]), r.h[j], dx * r.b[j]);
        y = __builtin_fmaf(r.c[j], r.h[j], y);
      }
      y = __builtin_fmaf(Dc, x, lanes_sum<NL>(y));
      if (kGate) {
        const float z = bf16_f32(r.z);
        y *= z * sigmoid_f32(z);
      }
      if (there && some) {
        float* h = a.state + r.slot * a.C * a.N + h0;
        if (kVec) {
          __builtin_nontemporal_store((f32x4_t){r.h[0], r.h[1], r.h[2], r.h[3]}, reinterpret_cast<f32x4_t*>(h));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n0 + j < a.N) h[j] = r.h[j];
        }
      }
    }
    if (there && part == 0) (a.y + (int64_t)row * a.C)[c] = bf16_of(y);
  }
}

template <int NL>
void step_nl(const ScanArgs& a, hipStream_t s) {
  const int64_t rows = scan_step_rows(a.S, a.C, a.N);
  const dim3 grid((uint32_t)(scan_step_threads(a.S, a.C, a.N) / 256)), block(256);
  const bool vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0;
  if (a.z) {
    if (vec) hipLaunchKernelGGL((scan_step_kernel<NL, true, true>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((scan_step_kernel<NL, false, true>), grid, block, 0, s, a, (int32_t)rows);
  } else {
    if (vec) hipLaunchKernelGGL((scan_step_kernel<NL, true, false>), grid, block, 0, s, a, (int32_t)rows);
    else hipLaunchKernelGGL((scan_step_kernel<NL, false, false>), grid, block, 0, s, a, (int32_t)rows);
  }
}

// ----------------------------------------------------------- short prompts --
//
// The forward of a row of tokens that is short: the lanes of the single-token
// form, walking the row.  A token takes a wave a third of the instructions that
// it takes with all states in a lane, and the row one launch instead of three.
// The waves of a workgroup have the same channels and a part of the row each:
// they find the state behind their part from zero history, join these through
// LDS, and go over their part again for the outputs.  kVec: N a multiple of 4.
//
// Bound by the instructions of the two or so waves a SIMD has.  C = 2048, 16
// states, 77 tokens: 10.5 us; one wave for the whole row 20.6, three launches 22.
// Groups of 4 tokens: of 2 take 10.0 us there but 12.2 against 8.6 at 16 tokens
// of 16384 channels, of 8 12.0.  16 waves a workgroup are slower from C = 6144 on
// (77 tokens 19.0 against 15.4) and not faster below.

constexpr int kShortWaves = 8, kShortAhead = 4;

template <int NL, bool kVec, bool kGate>
__global__ __launch_bounds__(64 * kShortWaves) void scan_short_kernel(ScanArgs a, int32_t each) {
  constexpr int kChannels = 64 / NL;
  struct Piece {
    float h[4][64], sum[64];
    int32_t apart;  // a document starts in the part
  };
  __shared__ Piece pieces[kShortWaves - 1];
  // The outputs wait here for the end: loads and stores share one counter of
  // outstanding accesses, and a store among the loads would be waited for with
  // every group of them.
  __shared__ uint16_t out[scan_short(4 * NL)][kChannels];
  const int32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
  const int32_t lane = threadIdx.x & 63, part = lane % NL, n0 = 4 * part;
  const int32_t c0 = (int32_t)blockIdx.x * kChannels + lane / NL;
  const bool there = c0 < a.C, some = n0 < a.N;
  const uint32_t c = there ? c0 : 0;
  const int32_t t0 = w * each, t1 = min(a.S, t0 + each);
  float A2[4], h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    A2[j] = n0 + j < a.N ? param_at(a.A, a.A_bf16, (int64_t)c * a.N + n0 + j) * kLog2E : 0.0f;
    h[j] = 0.0f;
  }
  const float bias = step_bias(a, c);
  const float Dc = a.D ? param_at(a.D, a.D_bf16, c) : 0.0f;
  const uint32_t bc0 = c / (uint32_t)a.per * (uint32_t)a.N + (some ? n0 : 0);
  const uint32_t h0 = c * (uint32_t)a.N + n0;
  auto four = [&](const uint16_t* p) {
    if (kVec) return *reinterpret_cast<const u32x2_any*>(p);
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n0 + j < a.N ? (uint32_t)p[j] : 0u;
    return (u32x2_any){v[0] | v[1] << 16, v[2] | v[3] << 16};
  };
  // The document that starts at t0 or before it, and whether it starts there.
  const int32_t at = first_at_least(a.cu, a.num_docs + 1, t0);
  const bool starts = at <= a.num_docs && uniform_at(a.cu, at) == t0;
  float first[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // what a document that runs past the part resumed with
  float sum = 0.0f;
  int32_t apart = 0;

  // One pass over the part: from zero history for the state behind it and the
  // sum of the step sizes, or from h for the outputs.
  auto pass = [&](auto outputs) {
    constexpr bool kOut = decltype(outputs)::value;
    struct Raw {
      uint32_t x, dt, z;
      u32x2_any B, C;  // four states
    };
    // The next token's; past the end the last token's again.  A wave is bound by
    // the instructions it issues, addresses among them.
    RowBuffer bx, bd, bz;
    bx.open(a.x, t0, a.xs);
    bd.open(a.dt, t0, a.dts);
    bz.open(kGate ? a.z : a.x, t0, kGate ? a.zs : a.xs);
    const uint16_t *pB = a.B + t0 * a.Bs, *pC = a.Cm + t0 * a.Cs;
    const uint32_t lane2 = c * 2u;
    int32_t left = t1 - t0;
    auto request = [&]() {
      Raw r;
      r.x = bx.get(lane2);
      r.dt = bd.get(lane2);
      r.z = kOut && kGate ? bz.get(lane2) : 0u;
      r.B = four(pB + bc0);
      if (kOut) r.C = four(pC + bc0);
      --left;
      const bool more = left > 0;
      bx.row += more ? bx.stride : 0u;
      bd.row += more ? bd.stride : 0u;
      if (kOut && kGate) bz.row += more ? bz.stride : 0u;
      pB += more ? a.Bs : 0;
      if (kOut) pC += more ? a.Cs : 0;
      return r;
    };
    int32_t doc = at - 1, t = t0;
    int32_t next = doc >= 0 && doc < a.num_docs ? uniform_at(a.cu, doc + 1) : INT32_MAX;
    auto write = [&](int32_t d) {
      const int64_t slot = kOut && a.state ? slot_of(a.index, d, a.slots) : -1;
      if (slot < 0 || !there) return;
      float* s = a.state + slot * a.C * a.N + h0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + j < a.N) s[j] = h[j];
    };
    // The document that starts at t, past the empty ones before it.
    auto open = [&](int32_t d) {
      apart = 1;
      while (true) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = 0.0f;
        if (d >= a.num_docs || uniform_at(a.cu, d + 1) > t) break;
        if (kOut && !resumes(a, d)) write(d);
        ++d;
      }
      doc = d;
      next = d < a.num_docs ? uniform_at(a.cu, d + 1) : INT32_MAX;
      if (!a.state || d >= a.num_docs || !resumes(a, d)) return;
      const int64_t slot = slot_of(a.index, d, a.slots);
      if (slot < 0) return;
      // The wave that ends the document writes its slot while this one is at
      // its second pass: that pass has the state from the first, which the
      // row's last part does not make.
      const bool past = next > t1 && t1 < a.S;
      const float* s = a.state + slot * a.C * a.N + h0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v = 0.0f;
        if (n0 + j < a.N && !(kOut && past)) v = s[j];
        h[j] = kOut && past ? first[j] : v;
        if (!kOut) first[j] = v;
      }
    };
    // kTokens tokens from t on.  What does not wait for the states, and the sums
    // over the lanes, stand side by side for all of them: a wave alone on its
    // SIMD would otherwise wait for most of its own results.
    auto tokens = [&](auto count, const Raw* r) {
      constexpr int kTokens = decltype(count)::value;
      float x[kTokens], d[kTokens], y[kTokens];
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        x[i] = bf16_lo(r[i].x);
        d[i] = step_size(a, bf16_lo(r[i].dt), bias);
        if (!kOut) sum += d[i];
      }
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        const float dx = d[i] * x[i];
        const float b[4] = {bf16_lo(r[i].B.x), bf16_hi(r[i].B.x), bf16_lo(r[i].B.y), bf16_hi(r[i].B.y)};
        y[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = __builtin_fmaf(__builtin_amdgcn_exp2f(d[i] * A2[j]), h[j], dx * b[j]);
        if (kOut) {
          const float cm[4] = {bf16_lo(r[i].C.x), bf16_hi(r[i].C.x), bf16_lo(r[i].C.y), bf16_hi(r[i].C.y)};
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i] = __builtin_fmaf(cm[j], h[j], y[i]);
          if (!some) y[i] = 0.0f;
        }
      }
      if (!kOut) return;
#pragma unroll
      for (int i = 0; i < kTokens; ++i) {
        float v = __builtin_fmaf(Dc, x[i], lanes_sum<NL>(y[i]));
        if (kGate) {
          const float z = bf16_lo(r[i].z);
          v *= z * sigmoid_f32(z);
        }
        if (part == 0) out[t + i][lane / NL] = bf16_of(v);
      }
    };
    Raw q[kShortAhead];
    if (t0 < t1) {
#pragma unroll
      for (int i = 0; i < kShortAhead; ++i) q[i] = request();
    }
    if (starts) open(at);
#pragma unroll 1
    while (t < t1) {
      const int32_t end = next > t && next < t1 ? next : t1;
#pragma unroll 1
      for (; t + kShortAhead <= end; t += kShortAhead) {
        Raw r[kShortAhead];
#pragma unroll
        for (int i = 0; i < kShortAhead; ++i) {
          r[i] = q[i];
          q[i] = request();
        }
        tokens(std::integral_constant<int, kShortAhead>(), r);
      }
#pragma unroll 1
      for (; t < end; ++t) {
        const Raw r = q[0];
#pragma unroll
        for (int i = 0; i + 1 < kShortAhead; ++i) q[i] = q[i + 1];
        q[kShortAhead - 1] = request();
        tokens(std::integral_constant<int, 1>(), &r);
      }
      if (t == next && doc >= 0 && doc < a.num_docs) {
        write(doc);
        if (t < t1 || t == a.S) open(doc + 1);
      }
    }
  };

  if (t1 < a.S) {
    pass(std::false_type());
#pragma unroll
    for (int j = 0; j < 4; ++j) pieces[w].h[j][lane] = h[j];
    pieces[w].sum[lane] = sum;
    if (lane == 0) pieces[w].apart = apart;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = 0.0f;
#pragma unroll 1
  for (int32_t u = 0; u < w; ++u) {
    const float s = pieces[u].sum[lane];
    const bool cut = pieces[u].apart != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // 0 times an infinite decay is 0
      const float own = pieces[u].h[j][lane];
      h[j] = !cut && h[j] != 0.0f ? __builtin_fmaf(__builtin_amdgcn_exp2f(A2[j] * s), h[j], own) : own;
    }
  }
  pass(std::true_type());
  __syncthreads();
  const int32_t k = (int32_t)blockIdx.x * kChannels + threadIdx.x % kChannels;
  for (int32_t i = threadIdx.x / kChannels; i < a.S; i += blockDim.x / kChannels)
    if (k < a.C) a.y[(int64_t)i * a.C + k] = out[i][threadIdx.x % kChannels];
}

template <int NL>
void short_nl(const ScanArgs& a, hipStream_t s) {
  // Parts of whole groups of tokens, as even as they get.
  int32_t each = (a.S + kShortWaves - 1) / kShortWaves;
  each = (each + kShortAhead - 1) / kShortAhead * kShortAhead;
  const int32_t waves = a.S > 0 ? (a.S + each - 1) / each : 1;
  const dim3 grid((uint32_t)((a.C + 64 / NL - 1) / (64 / NL))), block(64 * waves);
  if (a.z) {
    if (a.N % 4 == 0) hipLaunchKernelGGL((scan_short_kernel<NL, true, true>), grid, block, 0, s, a, each);
    else hipLaunchKernelGGL((scan_short_kernel<NL, false, true>), grid, block, 0, s, a, each);
  } else {
    if (a.N % 4 == 0) hipLaunchKernelGGL((scan_short_kernel<NL, true, false>), grid, block, 0, s, a, each);
    else hipLaunchKernelGGL((scan_short_kernel<NL, false, false>), grid, block, 0, s, a, each);
  }
}

template <int NT, bool kOut>
void fwd_nt(const ScanArgs& a, int32_t work, hipStream_t s) {
  hipLaunchKernelGGL((scan_fwd_kernel<NT, kOut>), dim3(place_grid(work)), dim3(64 * kWaves), 0, s, a, work);
}

template <bool kOut>
hipError_t fwd(const ScanArgs& a, int32_t chunks, hipStream_t s) {
  const int32_t work = a.G * a.wpg * chunks;
  switch (scan_states(a.N)) {
    case 8: fwd_nt<8, kOut>(a, work, s); break;
    case 16: fwd_nt<16, kOut>(a, work, s); break;
    case 32: fwd_nt<32, kOut>(a, work, s); break;
    default: fwd_nt<64, kOut>(a, work, s); break;
  }
  return hipGetLastError();
}

template <int NT>
void bwd_main_nt(const ScanArgs& a, hipStream_t s) {
  const int32_t cb = scan_bwd_channels(a.N), work = a.G * ((a.per + cb - 1) / cb) * a.chunks;
  const dim3 grid(place_grid(work)), block(64 * kWaves);
  if (a.z) hipLaunchKernelGGL((scan_bwd_main_kernel<NT, true>), grid, block, 0, s, a, work);
  else hipLaunchKernelGGL((scan_bwd_main_kernel<NT, false>), grid, block, 0, s, a, work);
}

template <int NT>
void bwd_local_nt(const ScanArgs& a, hipStream_t s) {
  static_assert(Tile<NT>::CB == (NT <= 16 ? 64 : NT == 32 ? 32 : 16), "scan_bwd_channels");
  const int32_t work = a.G * a.wpg * a.chunks;
  hipLaunchKernelGGL((scan_bwd_local_kernel<NT>), dim3(place_grid(work)), dim3(64 * kWaves), 0, s, a, work);
}

}  // namespace

bool scan_rows_fit(const ScanArgs& a) {
  const auto even = [](const uint16_t* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && stride % 2 == 0;
  };
  return a.N == scan_states(a.N) && even(a.B, a.Bs) && even(a.Cm, a.Cs);
}

hipError_t launch_scan_pad(ScanArgs* a, hipStream_t s) {
  const int32_t NT = scan_states(a->N);
  const int64_t each = (int64_t)a->S * a->G * (NT / 2);
  const int64_t blocks = std::min((2 * each + 255) / 256, kPadBlocks);
  hipLaunchKernelGGL(scan_pad_kernel, dim3((uint32_t)blocks), dim3(256), 0, s, *a, NT);
  a->B = reinterpret_cast<const uint16_t*>(a->pad);
  a->Cm = reinterpret_cast<const uint16_t*>(a->pad + each);
  a->Bs = a->Cs = (int64_t)a->G * NT;
  a->bn = NT;
  return hipGetLastError();
}

hipError_t launch_scan_local(const ScanArgs& a, hipStream_t s) { return fwd<false>(a, a.chunks - 1, s); }
hipError_t launch_scan_out(const ScanArgs& a, hipStream_t s) { return fwd<true>(a, a.chunks, s); }

hipError_t launch_scan_join(const ScanArgs& a, bool backward, hipStream_t s) {
  hipLaunchKernelGGL(scan_join_kernel, dim3(a.cols / 64, a.N, backward ? 2 : 1),
                     dim3(64 * kJoinWaves), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_scan_bwd_local(const ScanArgs& a, hipStream_t s) {
  switch (scan_states(a.N)) {
    case 8: bwd_local_nt<8>(a, s); break;
    case 16: bwd_local_nt<16>(a, s); break;
    case 32: bwd_local_nt<32>(a, s); break;
    default: bwd_local_nt<64>(a, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_scan_bwd_main(const ScanArgs& a, hipStream_t s) {
  switch (scan_states(a.N)) {
    case 8: bwd_main_nt<8>(a, s); break;
    case 16: bwd_main_nt<16>(a, s); break;
    case 32: bwd_main_nt<32>(a, s); break;
    default: bwd_main_nt<64>(a, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_scan_bwd_sum(const ScanArgs& a, hipStream_t s) {
  const int32_t cb = scan_bwd_channels(a.N), bpg = (a.per + cb - 1) / cb;
  const int32_t NT = scan_states(a.N);
  const int64_t params = (int64_t)((a.cols + 255) / 256) * (a.N + 2);
  const int64_t quads = (int64_t)a.S * NT / 2;
  hipLaunchKernelGGL(scan_sum_kernel, dim3((uint32_t)(params + (quads + 255) / 256 * a.G)), dim3(256), 0, s, a,
                     bpg, NT);
  return hipGetLastError();
}

hipError_t launch_scan_short(const ScanArgs& a, hipStream_t s) {
  if (a.N <= 4) short_nl<1>(a, s);
  else if (a.N <= 8) short_nl<2>(a, s);
  else if (a.N <= 16) short_nl<4>(a, s);
  else if (a.N <= 32) short_nl<8>(a, s);
  else short_nl<16>(a, s);
  return hipGetLastError();
}

hipError_t launch_scan_step(const ScanArgs& a, hipStream_t s) {
  switch (scan_step_lanes(a.N)) {
    case 1: step_nl<1>(a, s); break;
    case 2: step_nl<2>(a, s); break;
    case 4: step_nl<4>(a, s); break;
    case 8: step_nl<8>(a, s); break;
    default: step_nl<16>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace vdc
