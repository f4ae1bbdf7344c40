// Internal interface between the host entry points (vdc_layer_api.cpp) and the
// kernels of the recurrent layer (vdc_recurrence.hip, vdc_layer_norm.hip,
// vdc_pool.hip).  Not installed; include/vdc.h is the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace vdc {

// ---------------------------------------------- gated linear recurrence --

// Tokens of the tiles that a row is cut into: 128 forward and 64 backward, and 64
// forward where that leaves a CU one tile or none (1543 tokens, C = 520, 225 tiles of
// 64: 8.8 against 10.6 us; 8000 tokens, C = 256, 500 of them: 14.4 against 12.5), but
// one tile as far as it goes, which needs no words (77 tokens, C = 2048: 7.5 us against
// 2.0 for the words and 7.9).
constexpr int kRecurFwdTile = 128, kRecurBwdTile = 64;
inline int64_t recur_tiles_of_64(int64_t S, int64_t C) { return (S + 63) / 64 * ((C + 63) / 64); }
inline int recur_fwd_tile(int64_t S, int64_t C) {
  return S > kRecurFwdTile && recur_tiles_of_64(S, C) <= 256 ? 64 : kRecurFwdTile;
}
// Tokens between two states that a training forward keeps.
constexpr int kRecurKeep = kRecurBwdTile;

struct RecurArgs {
  const uint16_t *x, *r, *i, *z, *dy;
  int64_t xs, rs, is, zs, dys;  // elements between rows
  const void* decay;            // [C]
  int32_t decay_bf16;
  float scale;
  const int32_t* cu;
  int32_t num_docs;
  int32_t S, C;
  int32_t tiles, tile;          // of tokens, and how many each has
  int32_t blocks;               // workgroups that share a tile of tokens
  int32_t cols;                 // words of a tile: C rounded up to 64
  int32_t docs_each;            // documents that a tile looks through for empty ones
  float* state;                 // [slots][C]
  const int32_t* index;
  const uint8_t* resume;
  int64_t slots;
  uint16_t* y;
  float* keep;                  // [ceil(S / kRecurKeep)][C] or null; backward: read
  uint16_t *dx, *dr, *di, *dz;
  void* ddecay;
  // workspace
  uint64_t* tickets;            // [cols] every 64th counts the tiles of its channels that have begun; the words follow
  uint64_t* words;              // [tiles][cols] what a tile hands on
  float* part;                  // backward of many tiles: [tiles][C] partial ddecay
  uint64_t* sums;               // backward of few: [tiles][cols] of them as words, behind the others; else null
};

// Whether a backward's tiles add their partial sums of ddecay in the same launch.  25
// tiles, C = 520, with their forward: 22.6 against 23.9 us; 125 tiles, C = 1024, whose
// last one has more words to read than its neighbours: 81 against 75.
inline bool recur_few(int64_t S) { return S <= 32 * kRecurBwdTile; }

// The tickets and the words as a call finds them.
hipError_t launch_recur_clear(const RecurArgs& a, hipStream_t s);
hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s);
hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s);
hipError_t launch_recur_bwd_sum(const RecurArgs& a, hipStream_t s);
hipError_t launch_recur_step(const RecurArgs& a, hipStream_t s);

// ------------------------------------------------------------ layer norm --

// Widest row, in channels.
constexpr int kLayerNormMaxC = 16384;

struct LayerNormArgs {
  const uint16_t *x, *res, *dy, *dstream;  // backward: x is the stream
  int64_t xs, ress, dys, dss;
  const void *w, *b;
  int32_t w_bf16, b_bf16;
  int64_t S;
  int32_t C;
  float eps;
  uint16_t *y, *stream, *dx;
  void *dw, *db;
  float* part;                             // [prows][2][C]
  int32_t prows;
};

hipError_t launch_layer_norm_fwd(const LayerNormArgs& a, hipStream_t s);
hipError_t launch_layer_norm_bwd(const LayerNormArgs& a, hipStream_t s);
hipError_t launch_layer_norm_bwd_sum(const LayerNormArgs& a, hipStream_t s);
// Partial rows of dweight and dbias, one or more for each workgroup of the backward.
int layer_norm_bwd_rows(int64_t S, int64_t C);

// ------------------------------------------------------ states put aside --

// Values that share a scale.
constexpr int kPoolBlock = 64;

struct PoolArgs {
  void* state;            // [slots][E]
  uint8_t* codes;         // [pool][E]
  float* scales;          // [pool][blocks]
  const int32_t *state_index, *pool_index;
  int64_t slots, pool, rows, E;
  int32_t bf16, e4m3;     // the state's dtype, the code
};

hipError_t launch_pool_quantize(const PoolArgs& a, hipStream_t s);
hipError_t launch_pool_dequantize(const PoolArgs& a, hipStream_t s);

}  // namespace vdc
