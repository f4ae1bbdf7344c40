// Host side of the recurrent layer's entry points declared in include/vdc.h:
// argument validation, workspace layout.  Nothing here allocates device memory,
// synchronizes or reads it.

#include "vdc.h"

#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "vdc_check.h"
#include "vdc_layer.h"

// ==================================================== the recurrence ==

namespace vdc {
namespace {

// The kernels count tokens, and entries of cu_seqlens, and a few past the last of
// them, in 32 bits.
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;

// Largest row stride of x, r, i, z and dy: a run of tokens stays below 2^31 bytes.
constexpr int64_t kRecurMaxStride = int64_t(1) << 25;

int recur_sizes(int64_t S, int64_t C) {
  if (S < 0 || S > kMaxTokens || C < 1 || C > kMaxC) return VDC_EINVAL;
  return ceil_div(S, kRecurBwdTile) * ceil_div(C, 64) >= (int64_t(1) << 23) ? VDC_EINVAL : VDC_OK;
}

// The checks that fwd, bwd and update share, and the kernels' arguments.
int recur_common(const vdc_recurrence* v, bool prompt, RecurArgs* a) {
  if (!v) return VDC_EINVAL;
  const int rc = recur_sizes(v->S, v->C);
  if (rc) return rc;
  if (!valid_dtype(v->decay_dtype)) return VDC_EDTYPE;
  if (!(v->scale >= 0.0f) || std::isinf(v->scale)) return VDC_EINVAL;
  const int64_t strides[4] = {v->x_stride, v->r_stride, v->i_stride, v->z ? v->z_stride : v->C};
  for (int64_t s : strides)
    if (s < v->C || s > kRecurMaxStride) return VDC_EINVAL;
  if (prompt) {
    if (v->num_docs < 0 || v->num_docs > kMaxTokens || (v->S > 0 && v->num_docs < 1)) return VDC_EINVAL;
    if (v->num_docs > 0 && !v->cu_seqlens) return VDC_EINVAL;
  }
  const int64_t seqs = prompt ? v->num_docs : v->S;
  if (v->slots < 0 || v->slots > kMaxS) return VDC_EINVAL;
  if (v->state && !v->state_index && seqs > v->slots) return VDC_EINVAL;
  if (!v->decay || (v->S > 0 && (!v->x || !v->r || !v->i))) return VDC_EINVAL;
  if (!aligned(v->x, 2) || !aligned(v->r, 2) || !aligned(v->i, 2) || !aligned(v->z, 2) ||
      !aligned(v->decay, dtype_bytes(v->decay_dtype)) || !aligned(v->state, 4) ||
      !aligned(v->state_index, 4) || !aligned(v->cu_seqlens, 4))
    return VDC_EALIGN;
  a->x = static_cast<const uint16_t*>(v->x);
  a->r = static_cast<const uint16_t*>(v->r);
  a->i = static_cast<const uint16_t*>(v->i);
  a->z = static_cast<const uint16_t*>(v->z);
  a->xs = v->x_stride;
  a->rs = v->r_stride;
  a->is = v->i_stride;
  a->zs = v->z_stride;
  a->decay = v->decay;
  a->decay_bf16 = v->decay_dtype == VDC_BF16;
  a->scale = v->scale;
  a->cu = v->cu_seqlens;
  a->num_docs = (int32_t)v->num_docs;
  a->S = (int32_t)v->S;
  a->C = (int32_t)v->C;
  a->state = v->state;
  a->slots = v->slots;
  a->index = v->state_index;
  a->resume = v->resume;
  return VDC_OK;
}

Span recur_in(const vdc_recurrence* v, int i) {
  switch (i) {
    case 0: return {v->x, rows_bytes(v->S, v->C, v->x_stride)};
    case 1: return {v->r, rows_bytes(v->S, v->C, v->r_stride)};
    case 2: return {v->i, rows_bytes(v->S, v->C, v->i_stride)};
    case 3: return {v->z, v->z ? rows_bytes(v->S, v->C, v->z_stride) : 0};
    default: return {v->decay, (size_t)v->C * dtype_bytes(v->decay_dtype)};
  }
}

// Whether `o` shares memory with an input of the call.
bool hits_input(const vdc_recurrence* v, const Span& o, bool prompt) {
  for (int i = 0; i < 5; ++i)
    if (overlaps(o, recur_in(v, i))) return true;
  const int64_t seqs = prompt ? v->num_docs : v->S;
  return (prompt && overlaps(o, {v->cu_seqlens, (size_t)(v->num_docs + 1) * 4})) ||
         overlaps(o, {v->state_index, (size_t)seqs * 4}) ||
         (prompt && overlaps(o, {v->resume, (size_t)seqs}));
}

Span state_span(const vdc_recurrence* v) {
  return {v->state, v->state ? (size_t)v->slots * v->C * 4 : 0};
}

// Places the workspace's arrays (base may be null: the size alone): the tickets
// and the words, which one tile does without, then the backward's partial sums.
size_t recur_layout(int dir, int64_t S, int64_t C, char* base, RecurArgs* a) {
  const int tile = dir == VDC_FWD ? recur_fwd_tile(S, C) : kRecurBwdTile;
  const int64_t tiles = ceil_div(S, tile);
  const int64_t cols = ceil_div(C, 64) * 64;
  const size_t row = (size_t)tiles * cols * 8, words = tiles > 1 ? cols * 8 + row : 0;
  const bool few = recur_few(S);
  a->tiles = (int32_t)tiles;
  a->tile = tile;
  a->cols = (int32_t)cols;
  a->tickets = reinterpret_cast<uint64_t*>(base);
  a->words = a->tickets + cols;
  a->part = reinterpret_cast<float*>(base + words);
  a->sums = dir == VDC_BWD && few ? reinterpret_cast<uint64_t*>(base + words) : nullptr;
  if (dir == VDC_FWD) return words;
  return few ? words + std::max<size_t>(row, 256) : words + (size_t)tiles * C * 4;
}

}  // namespace
}  // namespace vdc

using namespace vdc;

extern "C" int64_t gated_recurrence_keep_rows(int64_t S) {
  return S < 0 || S > kMaxTokens ? 0 : ceil_div(S, kRecurKeep);
}

extern "C" size_t gated_recurrence_workspace_bytes(int direction, int64_t S, int64_t C) {
  RecurArgs a{};
  if ((direction != VDC_FWD && direction != VDC_BWD) || recur_sizes(S, C) != VDC_OK || S == 0) return 0;
  return recur_layout(direction, S, C, nullptr, &a);
}

extern "C" int gated_recurrence_fwd(const vdc_recurrence* v, void* y, float* keep, void* workspace,
                                    size_t ws_bytes, hipStream_t stream) {
  RecurArgs a{};
  int rc = recur_common(v, true, &a);
  if (rc) return rc;
  if (keep && v->state) return VDC_EINVAL;
  if (v->S == 0 && (!v->state || v->num_docs == 0)) return VDC_OK;
  if (v->S > 0 && !y) return VDC_EINVAL;
  if (!aligned(y, 2) || !aligned(keep, 4)) return VDC_EALIGN;
  const size_t need = recur_layout(VDC_FWD, v->S, v->C, static_cast<char*>(workspace), &a);
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
  }
  const Span outs[4] = {{y, (size_t)v->S * v->C * 2}, state_span(v),
                        {keep, keep ? (size_t)ceil_div(v->S, kRecurKeep) * v->C * 4 : 0}, {workspace, need}};
  for (int i = 0; i < 4; ++i) {
    if (hits_input(v, outs[i], true)) return VDC_EINVAL;
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(outs[i], outs[j])) return VDC_EINVAL;
  }
  a.y = static_cast<uint16_t*>(y);
  a.keep = keep;
  a.docs_each = (int32_t)ceil_div(v->num_docs, std::max(a.tiles, 1));
  if (a.tiles > 1 && (rc = done(launch_recur_clear(a, stream)))) return rc;
  return done(launch_recur_fwd(a, stream));
}

extern "C" int gated_recurrence_bwd(const vdc_recurrence* v, const void* dy, int64_t dy_stride,
                                    const float* keep, void* dx, void* dr, void* di, void* ddecay,
                                    void* dz, void* workspace, size_t ws_bytes, hipStream_t stream) {
  RecurArgs a{};
  int rc = recur_common(v, true, &a);
  if (rc) return rc;
  if (v->state || !ddecay || dy_stride < v->C || dy_stride > kRecurMaxStride) return VDC_EINVAL;
  if (v->S > 0 && (!dy || !keep || !dx || !dr || !di || (dz == nullptr) != (v->z == nullptr)))
    return VDC_EINVAL;
  if (!aligned(dy, 2) || !aligned(keep, 4) || !aligned(dx, 2) || !aligned(dr, 2) || !aligned(di, 2) ||
      !aligned(dz, 2) || !aligned(ddecay, dtype_bytes(v->decay_dtype)))
    return VDC_EALIGN;
  const size_t need = v->S ? recur_layout(VDC_BWD, v->S, v->C, static_cast<char*>(workspace), &a) : 0;
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
  }
  const size_t act = (size_t)v->S * v->C * 2, kept = (size_t)ceil_div(v->S, kRecurKeep) * v->C * 4;
  const Span outs[6] = {{dx, act}, {dr, act}, {di, act}, {dz, dz ? act : 0}, {ddecay, recur_in(v, 4).n},
                        {workspace, need}};
  for (int i = 0; i < 6; ++i) {
    if (hits_input(v, outs[i], true) || overlaps(outs[i], {dy, rows_bytes(v->S, v->C, dy_stride)}) ||
        overlaps(outs[i], {keep, kept}))
      return VDC_EINVAL;
    for (int j = i + 1; j < 6; ++j)
      if (overlaps(outs[i], outs[j])) return VDC_EINVAL;
  }
  a.dy = static_cast<const uint16_t*>(dy);
  a.dys = dy_stride;
  a.keep = const_cast<float*>(keep);
  a.dx = static_cast<uint16_t*>(dx);
  a.dr = static_cast<uint16_t*>(dr);
  a.di = static_cast<uint16_t*>(di);
  a.dz = static_cast<uint16_t*>(dz);
  a.ddecay = ddecay;
  if (a.tiles > 1 && (rc = done(launch_recur_clear(a, stream)))) return rc;
  if (v->S > 0 && (rc = done(launch_recur_bwd(a, stream)))) return rc;
  return a.sums ? VDC_OK : done(launch_recur_bwd_sum(a, stream));
}

extern "C" int gated_recurrence_update(const vdc_recurrence* v, void* y, hipStream_t stream) {
  RecurArgs a{};
  int rc = recur_common(v, false, &a);
  if (rc) return rc;
  if (v->S == 0) return VDC_OK;
  if (!y || (!v->state && v->slots > 0)) return VDC_EINVAL;
  if (!v->state_index && v->S > v->slots) return VDC_EINVAL;
  if (!aligned(y, 2)) return VDC_EALIGN;
  const Span out{y, (size_t)v->S * v->C * 2}, st = state_span(v);
  if (hits_input(v, out, false) || hits_input(v, st, false) || overlaps(out, st)) return VDC_EINVAL;
  a.y = static_cast<uint16_t*>(y);
  return done(launch_recur_step(a, stream));
}

// ======================================================== layer norm ==

namespace vdc {
namespace {

int layer_norm_common(const void* x, int64_t xs, const void* w, int w_dtype, int b_dtype, bool bias,
                      int64_t S, int64_t C, float eps, LayerNormArgs* a) {
  if (S < 0 || S > kMaxS || C < 1 || C > kLayerNormMaxC || !(eps >= 0.0f)) return VDC_EINVAL;
  if (xs < C || xs > kMaxStride) return VDC_EINVAL;
  if (!valid_dtype(w_dtype) || (bias && !valid_dtype(b_dtype))) return VDC_EDTYPE;
  if (!w || (S > 0 && !x)) return VDC_EINVAL;
  if (!aligned(x, 2) || !aligned(w, dtype_bytes(w_dtype))) return VDC_EALIGN;
  a->x = static_cast<const uint16_t*>(x);
  a->xs = xs;
  a->w = w;
  a->w_bf16 = w_dtype == VDC_BF16;
  a->b_bf16 = b_dtype == VDC_BF16;
  a->S = S;
  a->C = (int32_t)C;
  a->eps = eps;
  return VDC_OK;
}

}  // namespace
}  // namespace vdc

extern "C" int layer_norm_fwd(const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, const void* weight, int w_dtype, const void* bias,
                              int b_dtype, int64_t S, int64_t C, float eps, void* y, void* stream_out,
                              hipStream_t stream) {
  LayerNormArgs a{};
  const int rc = layer_norm_common(x, x_stride, weight, w_dtype, b_dtype, bias != nullptr, S, C, eps, &a);
  if (rc) return rc;
  if (residual && (residual_stride < C || residual_stride > kMaxStride)) return VDC_EINVAL;
  if (S == 0) return VDC_OK;
  if (!y || (stream_out == nullptr) != (residual == nullptr)) return VDC_EINVAL;
  if (!aligned(y, 2) || !aligned(residual, 2) || !aligned(stream_out, 2) ||
      (bias && !aligned(bias, dtype_bytes(b_dtype))))
    return VDC_EALIGN;
  const size_t act = (size_t)S * C * 2;
  if (clash({{y, act}, {stream_out, stream_out ? act : 0}},
            {{x, rows_bytes(S, C, x_stride)}, {residual, residual ? rows_bytes(S, C, residual_stride) : 0},
             {weight, (size_t)C * dtype_bytes(w_dtype)}, {bias, bias ? (size_t)C * dtype_bytes(b_dtype) : 0}}))
    return VDC_EINVAL;
  a.res = static_cast<const uint16_t*>(residual);
  a.ress = residual_stride;
  a.b = bias;
  a.y = static_cast<uint16_t*>(y);
  a.stream = static_cast<uint16_t*>(stream_out);
  return done(launch_layer_norm_fwd(a, stream));
}

extern "C" size_t layer_norm_workspace_bytes(int64_t S, int64_t C) {
  if (S < 1 || S > kMaxS || C < 1 || C > kLayerNormMaxC) return 0;
  return (size_t)layer_norm_bwd_rows(S, C) * 2 * C * 4;
}

extern "C" int layer_norm_bwd(const void* s, int64_t s_stride, const void* weight, int w_dtype,
                              const void* dy, int64_t dy_stride, const void* dstream,
                              int64_t dstream_stride, int64_t S, int64_t C, float eps, void* dx,
                              void* dweight, void* dbias, int b_dtype, void* workspace, size_t ws_bytes,
                              hipStream_t stream) {
  LayerNormArgs a{};
  int rc = layer_norm_common(s, s_stride, weight, w_dtype, b_dtype, dbias != nullptr, S, C, eps, &a);
  if (rc) return rc;
  if (dy_stride < C || dy_stride > kMaxStride || !dweight) return VDC_EINVAL;
  if (dstream && (dstream_stride < C || dstream_stride > kMaxStride)) return VDC_EINVAL;
  if (S > 0 && (!dy || !dx)) return VDC_EINVAL;
  if (!aligned(dy, 2) || !aligned(dstream, 2) || !aligned(dx, 2) || !aligned(dweight, dtype_bytes(w_dtype)) ||
      (dbias && !aligned(dbias, dtype_bytes(b_dtype))))
    return VDC_EALIGN;
  const size_t act = (size_t)S * C * 2, wn = (size_t)C * dtype_bytes(w_dtype);
  const size_t need = layer_norm_workspace_bytes(S, C);
  if (need) {
    if (!workspace || ws_bytes < need) return VDC_EWORKSPACE;
    if (!aligned(workspace, 16)) return VDC_EALIGN;
  }
  if (clash({{dx, act}, {dweight, wn}, {dbias, dbias ? (size_t)C * dtype_bytes(b_dtype) : 0}, {workspace, need}},
            {{s, rows_bytes(S, C, s_stride)}, {dy, rows_bytes(S, C, dy_stride)},
             {dstream, dstream ? rows_bytes(S, C, dstream_stride) : 0}, {weight, wn}}))
    return VDC_EINVAL;
  a.dy = static_cast<const uint16_t*>(dy);
  a.dys = dy_stride;
  a.dstream = static_cast<const uint16_t*>(dstream);
  a.dss = dstream_stride;
  a.dx = static_cast<uint16_t*>(dx);
  a.dw = dweight;
  a.db = dbias;
  a.part = static_cast<float*>(workspace);
  a.prows = S ? layer_norm_bwd_rows(S, C) : 0;
  if (S > 0 && (rc = done(launch_layer_norm_bwd(a, stream)))) return rc;
  return done(launch_layer_norm_bwd_sum(a, stream));
}

// ================================================== states put aside ==

namespace vdc {
namespace {

int pool_common(const void* state, int dtype, int64_t slots, int64_t E, const int32_t* state_index,
                const void* codes, int code, const float* scales, int64_t pool, const int32_t* pool_index,
                int64_t rows, PoolArgs* a) {
  if (slots < 0 || slots > kMaxS || pool < 0 || pool > kMaxS || rows < 0 || rows > kMaxS) return VDC_EINVAL;
  if (E < 1 || E > (int64_t(1) << 28) || rows * ceil_div(E, 4096) >= (int64_t(1) << 24)) return VDC_EINVAL;
  if (!valid_dtype(dtype) || (code != VDC_INT8 && code != VDC_E4M3)) return VDC_EDTYPE;
  if ((!state_index && rows > slots) || (!pool_index && rows > pool)) return VDC_EINVAL;
  if ((slots > 0 && !state) || (pool > 0 && (!codes || !scales))) return VDC_EINVAL;
  if (!aligned(state, dtype_bytes(dtype)) || !aligned(scales, 4) || !aligned(state_index, 4) ||
      !aligned(pool_index, 4))
    return VDC_EALIGN;
  const Span s{state, (size_t)slots * E * dtype_bytes(dtype)}, c{codes, (size_t)pool * E},
      f{scales, (size_t)pool * ceil_div(E, kPoolBlock) * 4};
  if (clash({s, c, f}, {{state_index, (size_t)rows * 4}, {pool_index, (size_t)rows * 4}})) return VDC_EINVAL;
  a->state = const_cast<void*>(state);
  a->codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  a->scales = const_cast<float*>(scales);
  a->state_index = state_index;
  a->pool_index = pool_index;
  a->slots = slots;
  a->pool = pool;
  a->rows = rows;
  a->E = E;
  a->bf16 = dtype == VDC_BF16;
  a->e4m3 = code == VDC_E4M3;
  return VDC_OK;
}

}  // namespace
}  // namespace vdc

extern "C" int state_quantize(const void* state, int dtype, int64_t slots, int64_t E,
                              const int32_t* state_index, void* codes, int code, float* scales,
                              int64_t pool, const int32_t* pool_index, int64_t rows, hipStream_t stream) {
  PoolArgs a{};
  const int rc = pool_common(state, dtype, slots, E, state_index, codes, code, scales, pool, pool_index, rows, &a);
  if (rc || rows == 0 || slots == 0 || pool == 0) return rc;
  return done(launch_pool_quantize(a, stream));
}

extern "C" int state_dequantize(const void* codes, int code, const float* scales, int64_t pool,
                                const int32_t* pool_index, void* state, int dtype, int64_t slots, int64_t E,
                                const int32_t* state_index, int64_t rows, hipStream_t stream) {
  PoolArgs a{};
  const int rc = pool_common(state, dtype, slots, E, state_index, codes, code, scales, pool, pool_index, rows, &a);
  if (rc || rows == 0 || slots == 0 || pool == 0) return rc;
  return done(launch_pool_dequantize(a, stream));
}
