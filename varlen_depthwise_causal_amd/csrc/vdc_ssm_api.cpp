// Host side of the state space layer's entry points declared in
// include/vdc.h: argument validation, launch planning, workspace layout.
// Nothing here allocates device memory, synchronizes or reads it.

#include "vdc.h"

#include <algorithm>
#include <climits>
#include <stdint.h>

#include "vdc_check.h"
#include "vdc_ssm.h"

namespace vdc {
namespace {

int conv_state_check(int64_t rows, int64_t C, const void* weight, int w_dtype, const void* bias,
                     int b_dtype, const void* state, int64_t slots, const int32_t* index,
                     int64_t seqs) {
  if (C <= 0 || C % 8 != 0 || C > kMaxC || rows < 0 || rows > kMaxS) return VDC_EINVAL;
  if (slots < 0 || slots > kMaxS || (!index && seqs > slots)) return VDC_EINVAL;
  if (!valid_dtype(w_dtype) || (bias && !valid_dtype(b_dtype))) return VDC_EDTYPE;
  if (seqs == 0) return VDC_OK;
  if (!weight || (!state && slots > 0)) return VDC_EINVAL;
  if (!aligned(weight, 16) || (bias && !aligned(bias, 16)) || !aligned(state, 16) ||
      !aligned(index, 4))
    return VDC_EALIGN;
  return VDC_OK;
}

}  // namespace
}  // namespace vdc

using namespace vdc;

extern "C" int conv1d_prefill(const void* x, const void* weight, int w_dtype, const void* bias,
                              int b_dtype, const int32_t* cu_seqlens, int64_t num_docs, int64_t S,
                              int64_t C, void* state, int64_t slots, const int32_t* state_index,
                              const uint8_t* resume, void* y, hipStream_t stream) {
  if (num_docs < 0 || num_docs > kMaxS - 1 || (S > 0 && num_docs < 1)) return VDC_EINVAL;
  int rc = conv_state_check(S, C, weight, w_dtype, bias, b_dtype, state, slots, state_index, num_docs);
  if (rc || num_docs == 0) return rc;
  if (!cu_seqlens) return VDC_EINVAL;
  const int64_t per = ceil_div(C / 8, 64);
  if (num_docs * per * 64 > kMaxThreads) return VDC_EINVAL;
  const size_t act = (size_t)S * C * 2;
  if (clash({{state, (size_t)slots * 3 * C * 2}, {y, act}},
            {{x, act}, {weight, (size_t)C * 4 * dtype_bytes(w_dtype)},
             {bias, bias ? (size_t)C * dtype_bytes(b_dtype) : 0},
             {cu_seqlens, (size_t)(num_docs + 1) * 4},
             {state_index, (size_t)num_docs * 4}, {resume, (size_t)num_docs}}))
    return VDC_EINVAL;
  rc = conv1d_fwd(x, weight, w_dtype, bias, b_dtype, cu_seqlens, num_docs, S, C, y, nullptr, 0, stream);
  if (rc || slots == 0) return rc;
  ConvStateArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.w = weight;
  a.b = bias;
  a.state = static_cast<uint16_t*>(state);
  a.index = state_index;
  a.cu = cu_seqlens;
  a.resume = resume;
  a.rows = S;
  a.C = C;
  a.x_stride = C;
  a.slots = slots;
  a.w_bf16 = w_dtype == VDC_BF16;
  a.b_bf16 = b_dtype == VDC_BF16;
  return done(launch_conv_edges(a, num_docs, stream));
}

extern "C" int conv1d_update(const void* x, int64_t x_stride, const void* weight, int w_dtype,
                             const void* bias, int b_dtype, int64_t rows, int64_t C, void* state,
                             int64_t slots, const int32_t* state_index, void* y,
                             hipStream_t stream) {
  int rc = conv_state_check(rows, C, weight, w_dtype, bias, b_dtype, state, slots, state_index, rows);
  if (rc) return rc;
  if (x_stride < C || x_stride > kMaxStride || x_stride % 8 != 0) return VDC_EINVAL;
  if (rows == 0) return VDC_OK;
  if (!x || !y) return VDC_EINVAL;
  if (!aligned(x, 16) || !aligned(y, 16)) return VDC_EALIGN;
  if (rows * ceil_div(C / 8, 64) * 64 > kMaxThreads) return VDC_EINVAL;
  if (clash({{y, (size_t)rows * C * 2}, {state, (size_t)slots * 3 * C * 2}},
            {{x, rows_bytes(rows, C, x_stride)}, {weight, (size_t)C * 4 * dtype_bytes(w_dtype)},
             {bias, bias ? (size_t)C * dtype_bytes(b_dtype) : 0}, {state_index, (size_t)rows * 4}}))
    return VDC_EINVAL;
  ConvStateArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.w = weight;
  a.b = bias;
  a.state = static_cast<uint16_t*>(state);
  a.index = state_index;
  a.rows = rows;
  a.C = C;
  a.x_stride = x_stride;
  a.slots = slots;
  a.w_bf16 = w_dtype == VDC_BF16;
  a.b_bf16 = b_dtype == VDC_BF16;
  return done(launch_conv_step(a, stream));
}

// ============================================================= the scan ==

namespace vdc {
namespace {

// The kernels count tokens, and a few past the last, in 32 bits.
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;

int scan_sizes(int64_t S, int64_t C, int64_t N, int64_t G) {
  if (S < 0 || S > kMaxTokens || C < 1 || C > kMaxC || N < 1 || N > kMaxStates) return VDC_EINVAL;
  if (G < 1 || C % G != 0) return VDC_EINVAL;
  return VDC_OK;
}

// Chunks of time: the waves of 64 channels alone fill the machine's 1024
// SIMDs only at C = 65536 and more, so a row of tokens is cut, into at most as
// many chunks as make kScanWaves waves.  A function of the sizes only.
constexpr int64_t kScanWaves = 4096, kScanSimds = 1024;
// Rows that do not fill the machine are cut as far as the chunks save more
// than joining them costs: to about a wave for each SIMD, into 24 (backward
// 64, a token takes five times as long) to 192 chunks, but not below 8 tokens,
// and no further than to 32.  Forward, C = 4096 and 300 tokens: 19 chunks 41
// us, 38 chunks 44.  Backward, C = 512: 300 tokens in 38 chunks 42 us, in 19
// 54; 2048 tokens in 128 chunks 65 us, in 86 77; 4096 tokens in chunks of 32
// 93 us and of 16 87, but at C = 1024 122 and 137.
constexpr int64_t kScanMinCut[2] = {24, 64}, kScanMaxCut = 192;
constexpr int64_t kScanMinChunk = 8, kScanCutChunk = 32;
static_assert(VDC_FWD == 0 && VDC_BWD == 1, "both are indexed by the direction");

// Largest row stride of x, dt, z and dy: a chunk of it stays below 2^31 bytes.
int64_t scan_stride_limit(int64_t C) { return std::max<int64_t>(int64_t(1) << 19, 4 * C) - 1; }

struct ScanPlan {
  bool brief;  // forward by launch_scan_short
  int32_t wpg, cols, chunk, chunks, blocks;  // blocks: channel blocks of the backward's main kernel
};

bool scan_plan(int dir, int64_t S, int64_t C, int64_t N, int64_t G, ScanPlan* out) {
  const int64_t per = C / G, wpg = ceil_div(per, 64), waves = G * wpg;
  // Rows of states of a chunk are addressed by 32-bit offsets in bytes.
  if (waves * 64 * scan_states(N) > INT32_MAX / 4) return false;
  const int64_t blocks = dir == VDC_BWD ? G * ceil_div(per, scan_bwd_channels(N)) : waves;
  const int64_t want = std::max<int64_t>(1, kScanWaves / blocks);
  int64_t low = ceil_div(std::max<int64_t>(S, 1), want);
  const int64_t cuts = std::min(std::max(kScanSimds / blocks, kScanMinCut[dir]), kScanMaxCut);
  const int64_t least = std::min(std::max(ceil_div(S, cuts), kScanMinChunk), kScanCutChunk);
  low = ceil_div(std::max(low, least), 8) * 8;
  // The kernels end with the fullest SIMD: of the chunks up to twice that long,
  // the one that gives it the fewest tokens.  C = 1500, 7000 tokens, forward
  // and backward: 125 chunks of 56 (2.9 waves a SIMD) 100 and 266 us, 146 of
  // 48 (3.4) 111 and 286.  Fewer than two waves save nothing, they wait.
  int64_t chunk = low, least_load = INT64_MAX;
  for (int64_t c = low; c <= 2 * low && c <= kScanMaxChunk; c += 8) {
    const int64_t load = std::max<int64_t>(ceil_div(ceil_div(S, c) * blocks, kScanSimds), 2) * c;
    if (load < least_load) least_load = load, chunk = c;
  }
  // A chunk's rows are addressed by 32-bit offsets from its first: with at
  // most 2^28 / C tokens, row strides up to scan_stride_limit fit.
  chunk = std::min<int64_t>(chunk, std::min<int64_t>(kScanMaxChunk, (int64_t(1) << 28) / C / 8 * 8));
  out->brief = dir == VDC_FWD && S <= scan_short(N);
  if (out->brief) chunk = scan_short(N);
  const int64_t chunks = std::max<int64_t>(1, ceil_div(S, chunk));
  if (chunk > INT32_MAX || (chunks * std::max(blocks, waves) + 64) * 64 > kMaxThreads) return false;
  const int64_t params = ceil_div(waves * 64, 256) * (N + 2);
  if (dir == VDC_BWD && (G * ceil_div(S * scan_states(N) / 2, 256) + params) * 256 > kMaxThreads) return false;
  out->wpg = (int32_t)wpg;
  out->cols = (int32_t)(waves * 64);
  out->chunk = (int32_t)chunk;
  out->chunks = (int32_t)chunks;
  out->blocks = (int32_t)blocks;
  return true;
}

// Places the workspace's arrays (base may be null: the size alone).
size_t scan_layout(int dir, int64_t S, int64_t N, int64_t G, const ScanPlan& p, char* base, ScanArgs* a) {
  size_t at = 0;
  auto take = [&](size_t elems) {
    char* r = base ? base + at : nullptr;
    at += (elems * 4 + 255) / 256 * 256;
    return reinterpret_cast<float*>(r);
  };
  // The backward's kernels read and write whole vectors of states.
  a->rows = (int32_t)(dir == VDC_BWD ? scan_states(N) : N);
  const size_t cols = p.cols, rows = (size_t)p.chunks * a->rows * cols;
  if (p.brief) return 0;
  a->pad = reinterpret_cast<uint32_t*>(take(S * G * scan_states(N)));
  if (dir == VDC_FWD && p.chunks == 1) return at;
  a->hend = take(rows);
  a->sum = take((size_t)p.chunks * cols);
  a->flags = reinterpret_cast<int32_t*>(take(p.chunks));
  if (dir == VDC_FWD) {
    a->snap = take(rows);
    return at;
  }
  a->mu = take(rows);
  a->keep = take((size_t)p.chunks * (p.chunk / kScanKeep) * (a->rows + 1) * cols);
  a->pparam = take((size_t)p.chunks * (a->rows + 2) * cols);
  a->pbc = take((size_t)p.blocks * S * 2 * scan_states(N));
  return at;
}

// The checks that fwd, bwd and update share, and the kernels' arguments.
int scan_common(const vdc_scan* v, bool prompt, ScanArgs* a) {
  if (!v) return VDC_EINVAL;
  int rc = scan_sizes(v->S, v->C, v->N, v->groups);
  if (rc) return rc;
  if (!valid_dtype(v->A_dtype) || (v->D && !valid_dtype(v->D_dtype)) ||
      (v->dt_bias && !valid_dtype(v->dt_bias_dtype)))
    return VDC_EDTYPE;
  const int64_t bc = v->groups * v->N;
  const int64_t strides[5] = {v->x_stride, v->dt_stride, v->z ? v->z_stride : v->C, v->B_stride,
                              v->C_stride};
  for (int i = 0; i < 5; ++i)
    if (strides[i] < (i < 3 ? v->C : bc) || strides[i] > (i < 3 ? scan_stride_limit(v->C) : kMaxStride))
      return VDC_EINVAL;
  if (prompt) {
    if (v->num_docs < 0 || v->num_docs > kMaxS - 1 || (v->S > 0 && v->num_docs < 1)) return VDC_EINVAL;
    if (v->num_docs > 0 && !v->cu_seqlens) return VDC_EINVAL;
  }
  const int64_t seqs = prompt ? v->num_docs : v->S;
  if (v->slots < 0 || v->slots > kMaxS) return VDC_EINVAL;
  if (v->state && !v->state_index && seqs > v->slots) return VDC_EINVAL;
  if (!v->A) return VDC_EINVAL;
  if (v->S > 0 && (!v->x || !v->dt || !v->B || !v->Cm)) return VDC_EINVAL;
  if (!aligned(v->x, 2) || !aligned(v->dt, 2) || !aligned(v->z, 2) || !aligned(v->B, 2) ||
      !aligned(v->Cm, 2) || !aligned(v->A, dtype_bytes(v->A_dtype)) ||
      (v->D && !aligned(v->D, dtype_bytes(v->D_dtype))) ||
      (v->dt_bias && !aligned(v->dt_bias, dtype_bytes(v->dt_bias_dtype))) ||
      !aligned(v->state, 4) || !aligned(v->state_index, 4) || !aligned(v->cu_seqlens, 4))
    return VDC_EALIGN;
  a->x = static_cast<const uint16_t*>(v->x);
  a->dt = static_cast<const uint16_t*>(v->dt);
  a->z = static_cast<const uint16_t*>(v->z);
  a->B = static_cast<const uint16_t*>(v->B);
  a->Cm = static_cast<const uint16_t*>(v->Cm);
  a->xs = v->x_stride;
  a->dts = v->dt_stride;
  a->zs = v->z_stride;
  a->Bs = v->B_stride;
  a->Cs = v->C_stride;
  a->A = v->A;
  a->D = v->D;
  a->bias = v->dt_bias;
  a->A_bf16 = v->A_dtype == VDC_BF16;
  a->D_bf16 = v->D_dtype == VDC_BF16;
  a->bias_bf16 = v->dt_bias_dtype == VDC_BF16;
  a->softplus = v->dt_softplus != 0;
  a->cu = v->cu_seqlens;
  a->num_docs = (int32_t)v->num_docs;
  a->S = (int32_t)v->S;
  a->C = (int32_t)v->C;
  a->N = (int32_t)v->N;
  a->G = (int32_t)v->groups;
  a->bn = (int32_t)v->N;
  a->per = (int32_t)(v->C / v->groups);
  a->state = v->state;
  a->slots = v->slots;
  a->index = v->state_index;
  a->resume = v->resume;
  return VDC_OK;
}

Span scan_in(const vdc_scan* v, int i) {
  const int64_t bc = v->groups * v->N;
  switch (i) {
    case 0: return {v->x, rows_bytes(v->S, v->C, v->x_stride)};
    case 1: return {v->dt, rows_bytes(v->S, v->C, v->dt_stride)};
    case 2: return {v->z, v->z ? rows_bytes(v->S, v->C, v->z_stride) : 0};
    case 3: return {v->B, rows_bytes(v->S, bc, v->B_stride)};
    case 4: return {v->Cm, rows_bytes(v->S, bc, v->C_stride)};
    case 5: return {v->A, (size_t)v->C * v->N * dtype_bytes(v->A_dtype)};
    case 6: return {v->D, v->D ? (size_t)v->C * dtype_bytes(v->D_dtype) : 0};
    case 7: return {v->dt_bias, v->dt_bias ? (size_t)v->C * dtype_bytes(v->dt_bias_dtype) : 0};
    default: return {nullptr, 0};
  }
}

// Whether `o` shares memory with an input of the call.
bool hits_input(const vdc_scan* v, const Span& o, bool prompt) {
  for (int i = 0; i < 8; ++i)
    if (overlaps(o, scan_in(v, i))) return true;
  const int64_t seqs = prompt ? v->num_docs : v->S;
  return (prompt && overlaps(o, {v->cu_seqlens, (size_t)(v->num_docs + 1) * 4})) ||
         overlaps(o, {v->state_index, (size_t)seqs * 4}) ||
         (prompt && overlaps(o, {v->resume, (size_t)seqs}));
}

Span state_span(const vdc_scan* v) {
  return {v->state, v->state ? (size_t)v->slots * v->C * v->N * 4 : 0};
}

}  // namespace
}  // namespace vdc

extern "C" size_t selective_scan_workspace_bytes(int direction, int64_t S, int64_t C, int64_t N,
                                                 int64_t groups) {
  ScanPlan p{};
  ScanArgs a{};
  if ((direction != VDC_FWD && direction != VDC_BWD) || scan_sizes(S, C, N, groups) != VDC_OK ||
      S == 0 || !scan_plan(direction, S, C, N, groups, &p))
    return 0;
  return scan_layout(direction, S, N, groups, p, nullptr, &a);
}

extern "C" int selective_scan_fwd(const vdc_scan* v, void* y, void* workspace, size_t ws_bytes,
                                  hipStream_t stream) {
  ScanArgs a{};
  ScanPlan p{};
  int rc = scan_common(v, true, &a);
  if (rc) return rc;
  if (!scan_plan(VDC_FWD, v->S, v->C, v->N, v->groups, &p)) return VDC_EINVAL;
  if (v->S == 0 && (!v->state || v->num_docs == 0)) return VDC_OK;
  if (v->S > 0 && !y) return VDC_EINVAL;
  if (!aligned(y, 2)) return VDC_EALIGN;
  const Span out{y, (size_t)v->S * v->C * 2}, st = state_span(v);
  if (hits_input(v, out, true) || hits_input(v, st, true) || overlaps(out, st)) return VDC_EINVAL;
  const size_t need = scan_layout(VDC_FWD, v->S, v->N, v->groups, p, static_cast<char*>(workspace), &a);
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
    const Span ws{workspace, need};
    if (hits_input(v, ws, true) || overlaps(ws, out) || overlaps(ws, st)) return VDC_EINVAL;
  }
  a.y = static_cast<uint16_t*>(y);
  a.wpg = p.wpg;
  a.cols = p.cols;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  if (!p.brief && !scan_rows_fit(a) && (rc = done(launch_scan_pad(&a, stream)))) return rc;
  if (p.chunks > 1) {
    if ((rc = done(launch_scan_local(a, stream)))) return rc;
    if ((rc = done(launch_scan_join(a, false, stream)))) return rc;
  }
  return done(p.brief ? launch_scan_short(a, stream) : launch_scan_out(a, stream));
}

extern "C" int selective_scan_bwd(const vdc_scan* v, const void* dy, int64_t dy_stride, void* dx,
                                  void* ddt, void* dz, void* dB, void* dC, void* dA, void* dD,
                                  void* ddt_bias, void* workspace, size_t ws_bytes,
                                  hipStream_t stream) {
  ScanArgs a{};
  ScanPlan p{};
  int rc = scan_common(v, true, &a);
  if (rc) return rc;
  if (v->state) return VDC_EINVAL;
  if (!scan_plan(VDC_BWD, v->S, v->C, v->N, v->groups, &p)) return VDC_EINVAL;
  if (dy_stride < v->C || dy_stride > scan_stride_limit(v->C)) return VDC_EINVAL;
  if (!dA || (dD == nullptr) != (v->D == nullptr) || (ddt_bias == nullptr) != (v->dt_bias == nullptr))
    return VDC_EINVAL;
  if (v->S > 0 && (!dy || !dx || !ddt || !dB || !dC || (dz == nullptr) != (v->z == nullptr)))
    return VDC_EINVAL;
  if (!aligned(dy, 2) || !aligned(dx, 2) || !aligned(ddt, 2) || !aligned(dz, 2) || !aligned(dB, 2) ||
      !aligned(dC, 2) || !aligned(dA, dtype_bytes(v->A_dtype)) ||
      (dD && !aligned(dD, dtype_bytes(v->D_dtype))) ||
      (ddt_bias && !aligned(ddt_bias, dtype_bytes(v->dt_bias_dtype))))
    return VDC_EALIGN;
  const size_t act = (size_t)v->S * v->C * 2, bc = (size_t)v->S * v->groups * v->N * 2;
  const size_t need = v->S ? scan_layout(VDC_BWD, v->S, v->N, v->groups, p, static_cast<char*>(workspace), &a) : 0;
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
  }
  const Span outs[9] = {{dx, act}, {ddt, act}, {dz, dz ? act : 0}, {dB, bc}, {dC, bc},
                        {dA, scan_in(v, 5).n}, {dD, scan_in(v, 6).n}, {ddt_bias, scan_in(v, 7).n},
                        {workspace, need}};
  for (int i = 0; i < 9; ++i) {
    if (hits_input(v, outs[i], true) || overlaps(outs[i], {dy, rows_bytes(v->S, v->C, dy_stride)}))
      return VDC_EINVAL;
    for (int j = i + 1; j < 9; ++j)
      if (overlaps(outs[i], outs[j])) return VDC_EINVAL;
  }
  a.dy = static_cast<const uint16_t*>(dy);
  a.dys = dy_stride;
  a.dx = static_cast<uint16_t*>(dx);
  a.ddt = static_cast<uint16_t*>(ddt);
  a.dz = static_cast<uint16_t*>(dz);
  a.dB = static_cast<uint16_t*>(dB);
  a.dC = static_cast<uint16_t*>(dC);
  a.dA = dA;
  a.dD = dD;
  a.dbias = ddt_bias;
  a.wpg = p.wpg;
  a.cols = p.cols;
  a.chunk = p.chunk;
  a.chunks = v->S ? p.chunks : 0;  // no tokens: sums over no partial rows
  if (v->S > 0) {
    ScanArgs first = a;
    if (!scan_rows_fit(a) && (rc = done(launch_scan_pad(&first, stream)))) return rc;
    if ((rc = done(launch_scan_bwd_local(first, stream)))) return rc;
    if (p.chunks > 1 && (rc = done(launch_scan_join(a, true, stream)))) return rc;
    if ((rc = done(launch_scan_bwd_main(a, stream)))) return rc;
  }
  return done(launch_scan_bwd_sum(a, stream));
}

extern "C" int selective_update(const vdc_scan* v, void* y, hipStream_t stream) {
  ScanArgs a{};
  int rc = scan_common(v, false, &a);
  if (rc) return rc;
  if (v->S == 0) return VDC_OK;
  if (!y || (!v->state && v->slots > 0)) return VDC_EINVAL;
  if (!v->state_index && v->S > v->slots) return VDC_EINVAL;
  if (!aligned(y, 2)) return VDC_EALIGN;
  if (scan_step_threads(v->S, v->C, v->N) > kMaxThreads) return VDC_EINVAL;
  const Span out{y, (size_t)v->S * v->C * 2}, st = state_span(v);
  if (hits_input(v, out, false) || hits_input(v, st, false) || overlaps(out, st)) return VDC_EINVAL;
  a.y = static_cast<uint16_t*>(y);
  return done(launch_scan_step(a, stream));
}

// =========================================================== group norm ==

namespace vdc {
namespace {

int norm_common(const void* x, int64_t xs, const void* w, int w_dtype, const void* b, int b_dtype,
                const void* z, int64_t zs, int64_t S, int64_t C, int64_t G, float eps, NormArgs* a) {
  if (S < 0 || S > kMaxS || C < 1 || C > kMaxC || G < 1 || C % G != 0 || C / G > kNormMaxGroup)
    return VDC_EINVAL;
  if (!(eps >= 0.0f)) return VDC_EINVAL;
  if (xs < C || xs > kMaxStride || (z && (zs < C || zs > kMaxStride))) return VDC_EINVAL;
  if (!valid_dtype(w_dtype) || (b && !valid_dtype(b_dtype))) return VDC_EDTYPE;
  if (!w || (S > 0 && !x)) return VDC_EINVAL;
  if (!aligned(x, 2) || !aligned(z, 2) || !aligned(w, dtype_bytes(w_dtype)) ||
      (b && !aligned(b, dtype_bytes(b_dtype))))
    return VDC_EALIGN;
  a->x = static_cast<const uint16_t*>(x);
  a->z = static_cast<const uint16_t*>(z);
  a->xs = xs;
  a->zs = zs;
  a->w = w;
  a->b = b;
  a->w_bf16 = w_dtype == VDC_BF16;
  a->b_bf16 = b_dtype == VDC_BF16;
  a->G = (int32_t)G;
  a->per = (int32_t)(C / G);
  a->S = S;
  a->C = C;
  a->eps = eps;
  return VDC_OK;
}

}  // namespace
}  // namespace vdc

extern "C" int group_norm_silu_fwd(const void* x, int64_t x_stride, const void* weight, int w_dtype,
                                   const void* bias, int b_dtype, const void* z, int64_t z_stride,
                                   int64_t S, int64_t C, int64_t groups, float eps, void* y,
                                   hipStream_t stream) {
  NormArgs a{};
  int rc = norm_common(x, x_stride, weight, w_dtype, bias, b_dtype, z, z_stride, S, C, groups, eps, &a);
  if (rc || S == 0) return rc;
  if (!y) return VDC_EINVAL;
  if (!aligned(y, 2)) return VDC_EALIGN;
  if (clash({{y, (size_t)S * C * 2}},
            {{x, rows_bytes(S, C, x_stride)}, {z, z ? rows_bytes(S, C, z_stride) : 0},
             {weight, (size_t)C * dtype_bytes(w_dtype)}, {bias, bias ? (size_t)C * dtype_bytes(b_dtype) : 0}}))
    return VDC_EINVAL;
  a.y = static_cast<uint16_t*>(y);
  return done(launch_norm_fwd(a, stream));
}

extern "C" size_t group_norm_silu_workspace_bytes(int64_t S, int64_t C, int64_t groups) {
  if (S < 1 || S > kMaxS || C < 1 || C > kMaxC || groups < 1 || C % groups != 0 ||
      C / groups > kNormMaxGroup)
    return 0;
  return (size_t)norm_bwd_rows(S, C, groups) * 2 * C * 4;
}

extern "C" int group_norm_silu_bwd(const void* x, int64_t x_stride, const void* weight, int w_dtype,
                                   const void* bias, int b_dtype, const void* z, int64_t z_stride,
                                   const void* dy, int64_t dy_stride, int64_t S, int64_t C,
                                   int64_t groups, float eps, void* dx, void* dweight, void* dbias,
                                   void* dz, void* workspace, size_t ws_bytes, hipStream_t stream) {
  NormArgs a{};
  int rc = norm_common(x, x_stride, weight, w_dtype, bias, b_dtype, z, z_stride, S, C, groups, eps, &a);
  if (rc) return rc;
  if (dy_stride < C || dy_stride > kMaxStride) return VDC_EINVAL;
  if (!dweight || (dbias == nullptr) != (bias == nullptr)) return VDC_EINVAL;
  if (S > 0 && (!dy || !dx || (dz == nullptr) != (z == nullptr))) return VDC_EINVAL;
  if (!aligned(dy, 2) || !aligned(dx, 2) || !aligned(dz, 2) || !aligned(dweight, dtype_bytes(w_dtype)) ||
      (dbias && !aligned(dbias, dtype_bytes(b_dtype))))
    return VDC_EALIGN;
  const size_t act = (size_t)S * C * 2, wn = (size_t)C * dtype_bytes(w_dtype);
  const size_t bn = bias ? (size_t)C * dtype_bytes(b_dtype) : 0;
  const size_t need = S ? group_norm_silu_workspace_bytes(S, C, groups) : 0;
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
  }
  if (clash({{dx, act}, {dz, dz ? act : 0}, {dweight, wn}, {dbias, bn}, {workspace, need}},
            {{x, rows_bytes(S, C, x_stride)}, {z, z ? rows_bytes(S, C, z_stride) : 0},
             {dy, rows_bytes(S, C, dy_stride)}, {weight, wn}, {bias, bn}}))
    return VDC_EINVAL;
  a.dy = static_cast<const uint16_t*>(dy);
  a.dys = dy_stride;
  a.dx = static_cast<uint16_t*>(dx);
  a.dz = static_cast<uint16_t*>(dz);
  a.dw = dweight;
  a.db = dbias;
  a.part = static_cast<float*>(workspace);
  a.prows = S ? norm_bwd_rows(S, C, groups) : 0;
  if (S > 0 && (rc = done(launch_norm_bwd(a, stream)))) return rc;
  return done(launch_norm_bwd_sum(a, stream));
}
