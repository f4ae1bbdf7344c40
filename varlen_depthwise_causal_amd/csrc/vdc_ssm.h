// Internal interface between the host entry points (vdc_ssm_api.cpp) and the
// kernels of the state space layer (vdc_conv_state.hip, vdc_scan.hip,
// vdc_norm.hip).  Not installed; include/vdc.h is the ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace vdc {

// ------------------------------------------- convolution, carried state --

struct ConvStateArgs {
  const uint16_t* x;      // [rows][C], x_stride elements between rows
  uint16_t* y;            // [rows][C] dense
  const void* w;          // [C][4]
  const void* b;          // [C] or null
  uint16_t* state;        // [slots][3][C]
  const int32_t* index;   // slot of each sequence, or null: its own number
  const int32_t* cu;      // prompts: prefix sums
  const uint8_t* resume;  // prompts: documents that go on from their slot
  int64_t rows;
  int64_t C;
  int64_t x_stride;
  int64_t slots;
  int32_t w_bf16;
  int32_t b_bf16;
};

hipError_t launch_conv_step(const ConvStateArgs& a, hipStream_t s);
hipError_t launch_conv_edges(const ConvStateArgs& a, int64_t docs, hipStream_t s);

// -------------------------------------------------------- selective scan --

// Largest number of states a channel may have.
constexpr int kMaxStates = 64;
// Backward: tokens between two kept states, and the longest chunk (its
// document starts are a bitmask in LDS).
constexpr int kScanKeep = 8;
constexpr int kScanMaxChunk = 2048;
// Forward rows of at most this many tokens take one launch instead of three.
// With 16 states 224 tokens take 20 us against 29 at C = 4096 and 20 against 18
// at C = 512; with 8 states and C = 2048 160 tokens 16 against 16; with 64
// states and C = 2048 512 tokens 60 against 102.
constexpr int scan_short(int64_t N) { return N <= 8 ? 160 : N <= 16 ? 224 : N <= 32 ? 320 : 512; }

struct ScanArgs {
  const uint16_t *x, *dt, *z, *B, *Cm, *dy;
  int64_t xs, dts, zs, Bs, Cs, dys;  // elements between rows
  const void *A, *D, *bias;          // [C][N], [C], [C]
  int32_t A_bf16, D_bf16, bias_bf16;
  int32_t softplus;
  const int32_t* cu;
  int32_t num_docs;
  int32_t S, C, N, G;
  int32_t bn;              // elements between the groups of a row of B or C
  // Channels by waves of 64 within a group: column (g, i) of the workspace
  // rows is g * wpg * 64 + i, for channel g * per + i.
  int32_t per;             // C / G
  int32_t wpg;             // waves of 64 channels a group takes
  int32_t cols;            // G * wpg * 64
  int32_t chunk, chunks;   // tokens a chunk holds, chunks of the packed row
  int32_t rows;            // states the workspace has room for: forward N, backward scan_states(N)
  float* state;            // [slots][C][N]
  const int32_t* index;
  const uint8_t* resume;
  int64_t slots;
  uint16_t* y;
  uint16_t *dx, *ddt, *dz, *dB, *dC;
  void *dA, *dD, *dbias;
  // workspace
  float* hend;             // [chunks][rows][cols] state after each chunk
  float* mu;               // [chunks][rows][cols] gradient that leaves each chunk to its left
  float* sum;              // [chunks][cols] sum of the step sizes of each chunk
  uint32_t* pad;           // [2][S][G][scan_states(N)] BF16: B and C, where their rows do not fit
  float* snap;             // [chunks][rows][cols] state a resumed document began with
  int32_t* flags;          // [chunks] bit 0: a document starts at the chunk's first token, 1: inside
  float* keep;             // [chunks * chunk / kScanKeep][rows + 1][cols]
  float* pparam;           // [chunks][rows + 2][cols] partial dA, dD, ddt_bias
  float* pbc;              // [G * bpg][S][2][NT] partial dB, dC
};

// States rounded up to what the kernels are built for.
inline int scan_states(int64_t N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
// Channels one wave of the backward's main kernel covers.
inline int scan_bwd_channels(int64_t N) {
  const int nt = scan_states(N);
  return nt <= 16 ? 64 : nt == 32 ? 32 : 16;
}

// Single tokens: lanes that hold a channel's states, four each, and the rows that
// a wave takes one after another, as many as leave eight waves a SIMD, at most 16.
inline int scan_step_lanes(int64_t N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline int64_t scan_step_blocks(int64_t C, int64_t N) { return (C * scan_step_lanes(N) + 63) / 64; }
inline int64_t scan_step_rows(int64_t S, int64_t C, int64_t N) {
  const int64_t rows = scan_step_blocks(C, N) * S / 8192;
  return rows < 1 ? 1 : rows > 16 ? 16 : rows;
}
inline int64_t scan_step_threads(int64_t S, int64_t C, int64_t N) {
  const int64_t rows = scan_step_rows(S, C, N), waves = scan_step_blocks(C, N) * ((S + rows - 1) / rows);
  return (waves + 3) / 4 * 256;
}

// Whether the forward and the backward's first pass can read B's and C's rows as
// they are; launch_scan_pad copies them to the workspace and points `a` there.
bool scan_rows_fit(const ScanArgs& a);
hipError_t launch_scan_pad(ScanArgs* a, hipStream_t s);
hipError_t launch_scan_local(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_join(const ScanArgs& a, bool backward, hipStream_t s);
hipError_t launch_scan_out(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd_local(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd_main(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_bwd_sum(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_step(const ScanArgs& a, hipStream_t s);
hipError_t launch_scan_short(const ScanArgs& a, hipStream_t s);

// ------------------------------------------------------------ group norm --

struct NormArgs {
  const uint16_t *x, *z, *dy;
  int64_t xs, zs, dys;
  const void *w, *b;
  int32_t w_bf16, b_bf16;
  int32_t G, per;          // groups, channels of a group
  int64_t S, C;
  float eps;
  uint16_t *y, *dx, *dz;
  void *dw, *db;
  float* part;             // [prows][2][C]
  int32_t prows;
};

// Largest group, in channels.
constexpr int kNormMaxGroup = 16384;

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_bwd_sum(const NormArgs& a, hipStream_t s);
int norm_bwd_rows(int64_t S, int64_t C, int64_t G);

}  // namespace vdc
