// The launch interface of what a DiT block does around the attention: rotary positions, the qk norm and the gated
// feed-forward.  Apart from dsv_internal.h, so that a change here leaves the attention's own sources as they were
// measured (the bench counts a kernel's captured DRAM traffic only for the sources it was captured on).
#pragma once

#include "dsv_internal.h"

namespace dsv {

// Bit of the device status word: a kernel met a token position outside its axis' table.
constexpr unsigned int kStatusBadPosition = 4u;

// ---------------------------------------------------------------- rotary positions, qk norm (dsv_rope.cu)
// A [B][H][N][d] view: element strides of sample, head and token (features are contiguous).
struct RopeView {
  bf16* p = nullptr;
  int64_t sb = 0, sh = 0, sn = 0;
};
struct RopeGeom {
  int64_t B, H, N;
  int64_t pos_batch;        // rows of pos between samples (0: shared)
  int pairs;                // rotated pairs of a row
  int axis_pairs[3];        // of them, each axis'
  int64_t len[3];           // positions of each axis' table
  int64_t table_off[3];     // first (cos, sin) of each axis
  // launch plan (rope_plan)
  int64_t tiles_per_b, heads_per_chunk, chunks, units;
};
struct RopeParams {
  RopeGeom g;
  int d;
  bool half, backward;      // pairs (j, j + R/2) instead of (2j, 2j + 1); rope3d's direction
  float eps;
  RopeView q, k, v;         // inputs (rope3d: q alone)
  RopeView qo, ko, vo;      // outputs of the forward; their gradients in the backward
  RopeView dq, dk, dv;      // gradients of the inputs (backward)
  const bf16 *wq, *wk;      // [d] or null (ones)
  float *dwq, *dwk;         // [d] or null (backward)
  float* partial;           // [rope_bwd_ctas][2][d] (backward)
  const int32_t* pos;       // [N][3] or [B][N][3]
  const float* table;
  unsigned int* status;
};
constexpr int64_t kRopeWantCtas = 8 * 152;   // CTAs below which the heads of a token are split
RopeGeom rope_plan(const RopeGeom& in, int d, bool backward);
int64_t rope_bwd_ctas(const RopeGeom& plan);
cudaError_t launch_rope3d_table(const RopeGeom& g, const double (&theta)[3], float* table, cudaStream_t stream);
cudaError_t launch_rope3d(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_fwd(const RopeParams& p, cudaStream_t stream);
cudaError_t launch_qk_norm_rope_bwd(const RopeParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- gated feed-forward (dsv_ffn.cu)
struct FfnParams {
  int64_t M, D, F;
  int act;                              // 0 silu, 1 gelu (tanh form)
  const bf16 *x, *w_gate, *w_up;        // [M][D], [F][D], [F][D]
  bf16* h;                              // [M][F] (forward)
  const bf16* dh;                       // [M][F] (backward)
  bf16 *dx, *dw_gate, *dw_up;           // [M][D], [F][D], [F][D] (backward)
  void* ws;                             // ffn_fwd_workspace / ffn_bwd_workspace bytes
  unsigned int* status;
};
size_t ffn_fwd_workspace(int64_t M, int64_t D, int64_t F);
size_t ffn_bwd_workspace(int64_t M, int64_t D, int64_t F);
cudaError_t launch_ffn_gated_fwd(const FfnParams& p, cudaStream_t stream);
cudaError_t launch_ffn_gated_bwd(const FfnParams& p, cudaStream_t stream);

}  // namespace dsv
