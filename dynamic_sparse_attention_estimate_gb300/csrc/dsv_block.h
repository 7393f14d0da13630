// The launch interface of what a DiT block does around the attention: rotary positions, the qk norm, the gated
// feed-forward, the branches' way back into the residual stream and the modulation's projection.  Apart from dsv_internal.h, so that a change here leaves the attention's own sources as they were
// measured (the bench counts a kernel's captured DRAM traffic only for the sources it was captured on).
#pragma once

#include <atomic>

#include "dsv_internal.h"

namespace dsv {

// Lets a kernel have `bytes` of dynamic shared memory on the current device: asked of the runtime once per kernel and device (the
// question costs the host about 0.7 us).
template <auto Kernel>
cudaError_t allow_shared(int bytes) {
  static std::atomic<uint64_t> allowed{0};   // a bit per device
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (allowed.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_release);
  return e;
}

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

// ---------------------------------------------------------------- gated residual with its norms (dsv_residual.cu)
enum { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };
struct ResidualParams {
  int64_t B, N, D;
  int post, pre;                        // norm of the branch (none, rms), of the new stream (none, rms, layer)
  bool f32;                             // x, r, dr, dx are fp32 instead of bf16
  float alpha, eps;
  const bf16 *z;                        // [B][N][D]
  const bf16 *gate, *scale, *shift;     // [B] rows of D, the strides apart; null: gate 1, scale and shift 0
  int64_t gate_stride, scale_stride, shift_stride;
  const bf16 *w_post, *w_pre;           // [D] or null (ones)
  const void* x;                        // [B][N][D] (forward)
  void* r;                              // [B][N][D]: the forward's output, the backward's input
  bf16* y;                              // [B][N][D] (forward)
  const void* dr;                       // [B][N][D] or null (backward)
  const bf16* dy;                       // [B][N][D] (backward)
  void* dx;                             // [B][N][D] (backward)
  bf16* dz;                             // [B][N][D] (backward)
  float *d_gate, *d_scale, *d_shift;    // [B] rows of D, d_stride apart, or null (backward)
  int64_t d_stride;
  float *dw_post, *dw_pre;              // [D] or null (backward)
  float* partial;                       // residual_bwd_workspace bytes (backward)
};
size_t residual_bwd_workspace(int64_t B, int64_t N, int64_t D, int pre, bool f32);
cudaError_t launch_residual_norm_fwd(const ResidualParams& p, cudaStream_t stream);
cudaError_t launch_residual_norm_bwd(const ResidualParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- 4-bit weights (dsv_w4.cu)
struct W4Params {
  int64_t M, D, F;
  int group;                            // columns to a scale: 32, 64 or 128
  uint8_t* data;                        // [F][D / 2]: column 2 i in the low bits of byte i
  bf16* scale;                          // [F][D / group]
  uint8_t* zero;                        // [F][D / group] or null (8)
  const bf16* w;                        // [F][D] (quantize)
  const bf16 *x, *bias;                 // [M][D], [F] or null (forward)
  bf16* y;                              // [M][F] (forward)
  const void* dy;                       // [M][F], bf16 or fp32 (backward)
  bool dy_f32;
  bf16* dx;                             // [M][D] (backward)
  float* partial;                       // w4_bwd_workspace bytes (backward)
};
size_t w4_bwd_workspace(int64_t M, int64_t D, int64_t F, int group, bool dy_f32);
cudaError_t launch_w4_quantize(const W4Params& p, cudaStream_t stream);
cudaError_t launch_w4_fwd(const W4Params& p, cudaStream_t stream);
cudaError_t launch_w4_bwd(const W4Params& p, cudaStream_t stream);

}  // namespace dsv
