/*
 * dsv.h -- C ABI of libdsv.so: DSV's dynamic sparse 3D attention on one GB300 (sm_103a).
 *
 * Source of the method: "DSV: Exploiting Dynamic Sparsity to Accelerate Large-Scale
 * Video DiT Training" (German and Spanish technical summaries).  Per attention head
 * a low-rank pair (Q_lr, K_lr) estimates Q K^T (section 2A); one fused kernel forms
 * that estimate and selects the top-k keys without materialising the N x N scores
 * (section 2B, "Fused MM & Top-K"), once per group of 3D-neighbouring queries
 * (section 2B, "Query Grouping"); softmax attention forward and backward then run
 * over the selected keys only (Spanish summary section 3, custom fused kernels for
 * estimation and sparse attention; training needs the backward).
 *
 * Conventions shared by every call
 *   - Layout: contiguous [B][H][N][d] (bf16) for Q, K, V, dO, O, dQ, dK, dV;
 *     [B][H][N][r] (bf16) for Q_lr, K_lr; [B][H][N] fp32 for LSE;
 *     [B][H][N/block][k] int32 for idx.  Tokens are in block-major order: query
 *     block b of a head is rows [block*b, block*b + block).  The caller permutes
 *     tokens (3D cubes of neighbours) before the call; the kernels do not care how.
 *   - Every pointer is a DEVICE pointer owned by the caller, 16-byte aligned.  The
 *     library allocates nothing and frees nothing; it keeps no state between calls
 *     except the device status word read by dsv_last_device_status().
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Calls enqueue work and return at once; none synchronises except
 *     dsv_last_device_status().
 *   - Arguments are validated on the host before anything is launched; an invalid
 *     call returns an error code, launches nothing and writes nothing.
 *     dsv_last_error_message() then holds a one-line reason (per host thread).
 *   - Identical inputs give bitwise-identical outputs (no floating-point atomics).
 */
#ifndef DSV_H
#define DSV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DSV_OK = 0,
    DSV_ERR_INVALID_ARG = 1,   /* bad shape, null or misaligned pointer */
    DSV_ERR_UNSUPPORTED = 2,   /* valid but not built (e.g. d not in {64,128}) */
    DSV_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    DSV_ERR_CUDA = 4,          /* a CUDA runtime call failed (launch, attribute) */
    DSV_ERR_DEVICE_CHECK = 5   /* a kernel found an out-of-range key index */
} dsv_status;

/* Problem sizes.  block must be 64; N % block == 0; 1 <= k <= N;
 * d in {64, 128}; r in {16, 32, 48, 64} (only the estimate reads r);
 * scale <= 0 selects 1/sqrt(d) (the usual softmax scale; the pages give none). */
typedef struct {
    int64_t B, H, N;
    int64_t d, r;
    int64_t block;
    int64_t k;
    float scale;
} dsv_dims;

/* Bytes of device workspace dsv_estimate_topk needs (0: it needs none). */
size_t dsv_estimate_topk_workspace(const dsv_dims* dims);

/*
 * Low-rank estimate + top-k per query block (DSV section 2A/2B: fused MM & top-k
 * with query grouping).
 *   q_hat[b]  = sum of Q_lr over the `block` tokens of query block b;
 *   s[b, j]   = q_hat[b] . K_lr[j]   for every key j of the same head (never stored);
 *   idx[b, :] = the k keys of largest s[b, j], ties to the lower j, ascending order.
 * q_lr, k_lr: bf16 [B][H][N][r].  idx: int32 [B][H][N/block][k] (output).
 * Scores are formed in fp32 from q_hat held as an exact two-term bf16 sum; with
 * integer-valued factors (|q_hat| < 2^16, |s| < 2^24) every score is exact, so the
 * selection equals the exact-arithmetic one.  ws may be NULL when the workspace
 * size is 0.
 */
dsv_status dsv_estimate_topk(const dsv_dims* dims, const void* q_lr, const void* k_lr,
                             int32_t* idx, void* ws, size_t ws_bytes, void* stream);

/*
 * Mass-based adaptive k per query block (DSV German summary section 2A, stage 2, and
 * Spanish summary "Fase 2": the critical KV pairs are those that make up ~90 % of the
 * attention score).  A block's estimated attention distribution over keys is
 * softmax_j(tau s[b, j]) with s the block logits above; k_row[b] is the length of the
 * shortest prefix of its keys, in (s desc, key asc) order, whose mass reaches the fraction
 * mass_num / 2^16 of the total.  The mass is counted in integer weights
 *   w_j = floor(2^24 * 2^x_j),  x_j = tau_log2 * (s[b, j] - max_j s[b, j])  (fp32),
 * 2^x by a fixed fp32 recipe (x = n + f, n = floor(x); 2^f from its Taylor series to degree
 * 6 with coefficients (ln 2)^i / i! rounded to fp32, evaluated in Horner form with every
 * product and sum rounded separately; then scaled by 2^n), w_j = 0 when x_j < -30, and the
 * target is ceil(W * mass_num / 2^16) with W = sum_j w_j.  So the selection is exactly
 * reproducible (for integer-valued factors, as for dsv_estimate_topk).
 *   tau_log2: tau * log2(e) as fp32, > 0 (tau: the estimate's inverse temperature; for a
 *             block-summed logit of 64 queries, 1/64 takes the mean);
 *   mass_num: the mass fraction times 2^16, 1 .. 65536 (0.9 -> 58982);
 *   dense_num: the per-block sparse/dense switch (the pages decide per block, from its
 *             sparsity, whether sparse attention is used): 0 = off, else a block whose k
 *             exceeds the fraction dense_num / 2^16 of the keys (k * 2^16 > dense_num * N)
 *             attends to all N keys (k_row = N);
 *   k_row:    int32 [B][H][N/block] (output), 1 <= k_row[b] <= N;
 *   rowptr:   int64 [B*H*N/block + 1] (output), the CSR offsets: rowptr[0] = 0,
 *             rowptr[i + 1] = rowptr[i] + k_row[i] (rows in [B][H][N/block] order);
 *   order:    int32 [B*H*N/block] (output, may be NULL): the rows by descending
 *             ceil(k_row / 128), a launch order for the CSR attention calls below (the
 *             longest blocks start first); needs N <= 523,904.
 * dims->k is not used (it must still pass validation).  All buffers are device memory
 * owned by the caller; the call only enqueues work on `stream`.
 */
dsv_status dsv_estimate_mass_k(const dsv_dims* dims, const void* q_lr, const void* k_lr, float tau_log2,
                               uint32_t mass_num, uint32_t dense_num, int32_t* k_row, int64_t* rowptr, int32_t* order,
                               void* stream);

/*
 * A longest-first launch order for CSR rows with any per-block k (e.g. a different k per
 * head, all heads in one launch): order (int32 [B*H*N/block], output) lists the rows by
 * descending ceil(k / 128), where k = rowptr[i + 1] - rowptr[i].  Pass it to the CSR
 * attention calls below so the longest blocks start first.  Needs N <= 523,904.
 */
dsv_status dsv_csr_launch_order(const dsv_dims* dims, const int64_t* rowptr, int32_t* order, void* stream);

/*
 * The selected keys of every query block for per-block k (e.g. from dsv_estimate_mass_k),
 * in CSR form: row i's k_row[i] keys of largest s (ties to the lower key, ascending) at
 * cols[rowptr[i] .. rowptr[i + 1]).  k_row[i] must be in [1, N]; cols has rowptr[last]
 * entries (int32, device, caller-owned).  The same selection rule and exactness as
 * dsv_estimate_topk.
 */
dsv_status dsv_estimate_topk_csr(const dsv_dims* dims, const void* q_lr, const void* k_lr, const int32_t* k_row,
                                 const int64_t* rowptr, int32_t* cols, void* stream);

/* Bytes of device workspace dsv_sparse_attn_fwd needs: 0 for every shape at present (the
 * workspace arguments are reserved, so that a future forward may take scratch without an ABI
 * change). */
size_t dsv_sparse_attn_fwd_workspace(const dsv_dims* dims);

/*
 * Sparse attention forward over the selected keys (DSV Spanish summary section 3:
 * sparse attention kernels; page 1 section 2A: only the critical KV pairs are used).
 * For query i of block b:  l_ij = scale * Q_i . K_j for j in idx[b];
 *   LSE_i = max_j l_ij + ln sum_j exp(l_ij - max_j l_ij);  O_i = sum_j exp(l_ij - LSE_i) V_j.
 * q, k, v: bf16 [B][H][N][d].  idx: int32 [B][H][N/block][k], entries in [0, N)
 * (need not be sorted here).  With k = N every key is selected and idx is not read (the
 * dense path; idx may then be NULL).  o: bf16 [B][H][N][d] (output).  lse: fp32 [B][H][N] (output, natural log).
 * Accumulation in fp32.  ws, ws_bytes: a device workspace of at least
 * dsv_sparse_attn_fwd_workspace(dims) bytes (NULL and 0 while that is 0), 16-byte aligned.
 */
dsv_status dsv_sparse_attn_fwd(const dsv_dims* dims, const void* q, const void* k, const void* v,
                               const int32_t* idx, void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Recommended / minimum device workspace for dsv_sparse_attn_bwd.  With more
 * workspace the backward processes more query blocks per wave (fewer launches). */
size_t dsv_sparse_attn_bwd_workspace(const dsv_dims* dims);
size_t dsv_sparse_attn_bwd_workspace_min(const dsv_dims* dims);

/*
 * Sparse attention backward (needed for training, DSV page 1 section 2A stage 2).
 * Recomputes P_ij = exp(scale Q_i.K_j - LSE_i) from the stored LSE, then
 *   D_i = dO_i . O_i;  dS_ij = P_ij (dO_i . V_j - D_i);
 *   dQ_i = scale sum_j dS_ij K_j;
 *   dK_j = scale sum_{i: j in idx[block(i)]} dS_ij Q_i;  dV_j = sum_{same i} P_ij dO_i.
 * Keys no block selected get dK = dV = 0.  No gradient flows to Q_lr / K_lr.
 * The entries of one idx row must be distinct (dsv_estimate_topk writes them strictly
 * ascending); a repeated or out-of-range entry sets the device status word.
 * dK/dV are reduced per key in ascending query-block order from per-(block, key)
 * partial rows held in the workspace: deterministic, no float atomics.  With k = N (every key
 * selected: the pages' dense case) idx is not read and no partial rows exist: dK and dV of each
 * tile of 128 keys accumulate on chip over all query blocks in block order, dQ per query block
 * (idx may then be NULL);
 * the workspace then holds only D = rowsum(dO o O) (4 bytes per query row).
 * d_o, q, k, v, o: bf16 [B][H][N][d]; lse fp32 [B][H][N]; idx int32 [B][H][N/block][k];
 * dq, dk, dv: bf16 [B][H][N][d] (outputs).  ws: device workspace of ws_bytes >=
 * dsv_sparse_attn_bwd_workspace_min(dims), 256-byte aligned.
 */
dsv_status dsv_sparse_attn_bwd(const dsv_dims* dims, const void* d_o, const void* q, const void* k,
                               const void* v, const void* o, const float* lse, const int32_t* idx,
                               void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);

/*
 * The backward in two calls, so that its first part can run beside the forward.  The first part
 * (dsv_sparse_attn_bwd_prepare) builds the backward's key-major rank structure of idx in the
 * workspace -- which query blocks selected each key, and where each key's partial rows go -- and
 * reads nothing but idx; the second (dsv_sparse_attn_bwd_prepared) runs the rest of
 * dsv_sparse_attn_bwd on that workspace and gives bitwise the same dQ, dK, dV.  A training step
 * can call prepare on a second stream as soon as idx exists, after the forward is enqueued, so
 * that it fills the SMs the forward leaves idle, and order prepared after it with an event.
 *   - Both calls take the same dims, idx, ws and ws_bytes; ws must hold every head in one wave
 *     (dsv_sparse_attn_bwd_workspace(dims) does when it fits; otherwise DSV_ERR_WORKSPACE).
 *   - prepared must run after prepare has finished (same stream, or an event), and nothing may
 *     write the workspace in between.  Arguments as dsv_sparse_attn_bwd.
 */
dsv_status dsv_sparse_attn_bwd_prepare(const dsv_dims* dims, const int32_t* idx, void* ws, size_t ws_bytes,
                                       void* stream);
dsv_status dsv_sparse_attn_bwd_prepared(const dsv_dims* dims, const void* d_o, const void* q, const void* k,
                                        const void* v, const void* o, const float* lse, const int32_t* idx, void* dq,
                                        void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);

/*
 * Backward without a caller workspace.  Some callers cannot allocate device memory
 * themselves: a host framework that owns every byte of the GPU through its own pool and
 * forbids outside allocations during a step, a plug-in whose memory budget is fixed when
 * its process starts, or a latency-critical loop where cudaMalloc/cudaFree would stall the
 * device.  This entry point computes exactly what dsv_sparse_attn_bwd computes, with the
 * library's own scratch: a fixed array of DSV_NOALLOC_SCRATCH_BYTES (32 MiB) in device
 * memory, held by every GPU that loads the library until the process exits.  It allocates
 * nothing.  (The DSV pages have no counterpart: this is a deployment convenience.)
 *   - Problems whose smallest backward workspace (dsv_sparse_attn_bwd_workspace_min) is
 *     above DSV_NOALLOC_SCRATCH_BYTES are rejected with DSV_ERR_WORKSPACE before anything
 *     runs; larger problems that fit are processed in several waves.  The smallest plan takes
 *     one query block per wave and chains a head's waves through an fp32 accumulator of
 *     8 d N bytes, next to k bf16 partial rows of 4 d bytes, so at d = 128 and the largest
 *     sparse k (N - 1) the limit is about N = 21,000 tokens per head (about N = 43,000 at
 *     d = 64); a head whose partial rows all fit (N/64 * k * 4 d bytes plus its rank structure)
 *     needs no accumulator, and k = N (the dense backward) needs only 4 bytes per query row.
 *     The long-video
 *     shape (N = 520,192, k = 52,019) is rejected: use dsv_sparse_attn_bwd there.
 *   - The first call on a device looks up that device's address of the array (with the
 *     device current); make that first call before any stream capture.
 *   - All calls share the one array, which keeps whatever the last call left there (every
 *     call rebuilds what it reads, so stale contents are never used); calls whose work
 *     overlaps on the GPU (other streams, other host threads) race on it and must be
 *     ordered by the caller.
 * Arguments and outputs are those of dsv_sparse_attn_bwd without ws / ws_bytes.
 */
#define DSV_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
dsv_status dsv_sparse_attn_bwd_noalloc(const dsv_dims* dims, const void* d_o, const void* q, const void* k,
                                       const void* v, const void* o, const float* lse, const int32_t* idx,
                                       void* dq, void* dk, void* dv, void* stream);

/*
 * Sparse attention over per-block key lists in CSR form (e.g. from dsv_estimate_mass_k and
 * dsv_estimate_topk_csr): query block i (rows in [B][H][N/block] order) attends to the keys
 * cols[rowptr[i] .. rowptr[i + 1]) (distinct, within [0, N); ascending order is not needed).
 * The same computation, layouts and outputs as dsv_sparse_attn_fwd / dsv_sparse_attn_bwd;
 * dims->k is not used (it must still pass validation).  A block with no keys gets O = 0,
 * LSE = -inf, dQ = 0.  rowptr: int64 [B*H*N/block + 1], cols: int32 [total_pairs], both
 * device memory owned by the caller.  order (may be NULL): a permutation of the rows in which
 * to launch them (e.g. dsv_estimate_mass_k's, longest first); results do not depend on it.
 * The backward runs as one wave over every head: its workspace must hold
 * dsv_sparse_attn_bwd_csr_workspace(dims, total_pairs) bytes (256-byte aligned), where
 * total_pairs = rowptr[B*H*N/block] (the caller knows it: it sized cols); otherwise
 * DSV_ERR_WORKSPACE.  total_pairs must fit int32.
 */
dsv_status dsv_sparse_attn_fwd_csr(const dsv_dims* dims, const void* q, const void* k, const void* v,
                                   const int64_t* rowptr, const int32_t* cols, const int32_t* order, void* o,
                                   float* lse, void* stream);
size_t dsv_sparse_attn_bwd_csr_workspace(const dsv_dims* dims, int64_t total_pairs);
dsv_status dsv_sparse_attn_bwd_csr(const dsv_dims* dims, const void* d_o, const void* q, const void* k, const void* v,
                                   const void* o, const float* lse, const int64_t* rowptr, const int32_t* cols,
                                   const int32_t* order, int64_t total_pairs, void* dq, void* dk, void* dv, void* ws,
                                   size_t ws_bytes, void* stream);

/* Human-readable name of a status code (static string). */
const char* dsv_status_string(dsv_status status);

/* One-line reason for the last non-OK status returned on this host thread. */
const char* dsv_last_error_message(void);

/* Synchronises `stream`, then reads and clears the current device's status word.
 * Returns DSV_ERR_DEVICE_CHECK if a kernel met a key index outside [0, N), or a token
 * position outside its axis' table, since the last read (the offending entry is skipped,
 * never dereferenced), DSV_ERR_CUDA if the synchronisation failed, DSV_OK otherwise. */
dsv_status dsv_last_device_status(void* stream);

/*
 * Optional per-kernel device timing, for measurement tools (not needed for use).
 * While enabled, every kernel launch the library makes is bracketed by two CUDA events
 * recorded on the launch's own stream (events come from a pool created at enable time;
 * no device memory is allocated).  dsv_profile_read() waits for the recorded events and
 * writes one line per kernel, "name launches total_ms\n", summed since the previous read,
 * into buf (NUL-terminated, truncated to buf_bytes); it returns the bytes needed.  With
 * buf == NULL it only reports the size and keeps the records.  Disabling drops unread
 * records.  Not thread-safe against concurrent launches from several host threads.
 */
dsv_status dsv_profile_enable(int on);
size_t dsv_profile_read(char* buf, size_t buf_bytes);

/* ---------------------------------------------------------------- fused AdaLN
 * LayerNorm + modulation in one pass over HBM, forward and backward (AdaptiveLoad page,
 * "AdaptiveLoad: Towards Efficient Video Diffusion Transformer Training", technical summary
 * section 2B: normalisation and modulation fused into one launch, statistics kept on chip,
 * and the modulation gradients reduced in (D tile, N tile) blocks so that reads stay
 * coalesced along D).  Per token n of sample b, over its D features:
 *   mean = sum_d x / D,  var = sum_d (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps),
 *   xhat = (x - mean) * rstd,   y = xhat * (1 + scale[b]) + shift[b].
 * The backward recomputes mean and rstd from x (nothing is saved by the forward) and returns
 *   dx = rstd * (g - mean_d(g) - xhat * mean_d(g * xhat)),  g = dy * (1 + scale[b]),
 *   d_scale[b] = sum_n dy * xhat,   d_shift[b] = sum_n dy.
 * Arithmetic: bf16 inputs, fp32 statistics and sums, bf16 y / dx, fp32 d_scale / d_shift;
 * bitwise reproducible (fixed summation order, no float atomics).
 * Layouts (contiguous, device memory owned by the caller, 16-byte aligned):
 *   x, y, dy, dx: bf16 [B][N][D];  scale, shift: bf16 [B][D];  d_scale, d_shift: fp32 [B][D].
 * Validation before any launch: B, N >= 1; D a multiple of 8 in [8, 8192]; eps >= 0 and
 * finite; no NULL or misaligned pointer (DSV_ERR_INVALID_ARG).  With eps = 0 a constant row
 * has var = 0 and its y / dx are NaN, as the definition gives.  Asynchronous on `stream`.
 */
typedef struct {
  int64_t B;   /* samples */
  int64_t N;   /* tokens per sample */
  int64_t D;   /* features per token */
  float eps;   /* added to the variance inside the square root */
} dsv_adaln_dims;

dsv_status dsv_adaln_fwd(const dsv_adaln_dims* dims, const void* x, const void* scale, const void* shift,
                         void* y, void* stream);
/* Bytes of workspace dsv_adaln_bwd needs (per-tile partial sums of the modulation gradients). */
size_t dsv_adaln_bwd_workspace(const dsv_adaln_dims* dims);
/* ws: at least dsv_adaln_bwd_workspace(dims) bytes, 256-byte aligned (DSV_ERR_WORKSPACE otherwise).
 * It holds per-tile partial sums and the tickets that order their final sum, so one workspace
 * must not serve two backward calls that can run at the same time (other streams); calls in
 * order on one stream may share it.  The call runs two kernels, the second launched as a
 * programmatic dependent of the first (it waits for the first to finish before reading). */
dsv_status dsv_adaln_bwd(const dsv_adaln_dims* dims, const void* x, const void* scale, const void* dy, void* dx,
                         float* d_scale, float* d_shift, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------- rotary positions with several axes, qk norm
 * What a video DiT block does between its Q/K/V projection and the attention above: the norm of
 * queries and keys for each head, the rotation by the token's (time, height, width) position, and
 * the move from the projection's layout to [B][H][N][d].  (The DSV pages take Q and K as given;
 * these calls produce them.)
 *
 * Rotation.  Axis a (0 time, 1 height, 2 width) turns rot[a] features (even; 0: axis unused): its
 * pair i < rot[a] / 2 by the angle p * theta[a]^(-2 i / rot[a]) at position p.  The R / 2 pairs
 * (R = rot[0] + rot[1] + rot[2] <= d) are numbered through the axes in order; pair j is
 *   DSV_PAIRS_INTERLEAVED: features (2 j, 2 j + 1);   DSV_PAIRS_HALVES: features (j, j + R / 2),
 * and turns  y0 = x0 cos - x1 sin,  y1 = x0 sin + x1 cos  (the backward by the negative angle).
 * Features from R on pass unchanged.  Angles separate over the axes, so the table holds one small
 * part per axis instead of a row per token:
 *   table: fp32 (cos, sin) pairs; axis a's part is [len[a]][rot[a] / 2][2], the parts one after
 *     another (dsv_rope3d_table fills it from theta, angles in fp64; a caller with scaled
 *     positions or frequencies fills its own);
 *   pos: int32 [N][3] (pos_batched = 0, shared by the samples) or [B][N][3]: each token's
 *     (t, h, w), 0 <= pos < len of that axis.  Tokens may be in any order (e.g. block-major).  An
 *     axis whose position is outside its table turns by the angle 0 for that token (finite features
 *     stay as they are), and the device status word is set (dsv_last_device_status).  A list that
 *     starts at another list's row i is 16-byte aligned where 4 divides i.
 *   With R = 0 nothing is rotated (norm alone); pos and table may then be NULL.
 *
 * Views.  Tensors are bf16 [B][H][N][d] with contiguous features; dsv_view_strides gives the
 * element strides of sample, head and token (each >= 0 and a multiple of 8; NULL: contiguous
 * [B][H][N][d]).  A packed projection [B][N][3][H][d] is three such views.  Inputs may be broadcast
 * (stride 0).  An output's elements must be distinct (its strides are checked), and outputs must
 * not overlap inputs or each other, except that rope3d may run in place (the same pointer and
 * strides).  A memory range that overlaps an input's in any other way is refused, the weights', pos
 * and the table (where the call reads them) among the inputs; outputs of one call may interleave in
 * one range with the same strides (a packed gradient).
 *
 * Validation before any launch: B, H, N >= 1; B*H*N < 2^31 - 64; d in {64, 128}; rot even, >= 0, sum
 * <= d (a multiple of 16 for DSV_PAIRS_HALVES); len >= 1 for every axis in use, and at most 2^31
 * (cos, sin) pairs in all; eps >= 0 and finite.  Any N: it need not be a multiple of the
 * attention's block.
 */
typedef enum { DSV_PAIRS_INTERLEAVED = 0, DSV_PAIRS_HALVES = 1 } dsv_pairing;

typedef struct {
  int64_t B, H, N, d;
  int64_t rot[3];        /* rotated features of time, height, width */
  int64_t len[3];        /* positions of each axis' table */
  int32_t pairing;       /* dsv_pairing */
  int32_t pos_batched;   /* pos has a row per (sample, token) */
  float eps;             /* of the norm (the rope3d calls do not read it) */
} dsv_rope_dims;

typedef struct {
  int64_t b, h, n;       /* element strides of sample, head, token */
} dsv_view_strides;

/* Bytes of the table (0 for invalid dims, or with R = 0). */
size_t dsv_rope3d_table_bytes(const dsv_rope_dims* dims);
/* Fills the table; theta[a] > 0 and finite for every axis in use.  Once per model, not per step. */
dsv_status dsv_rope3d_table(const dsv_rope_dims* dims, const double theta[3], float* table, void* stream);

/* y = x rotated at each token's position. */
dsv_status dsv_rope3d_fwd(const dsv_rope_dims* dims, const void* x, const dsv_view_strides* x_strides,
                          const int32_t* pos, const float* table, void* y, const dsv_view_strides* y_strides,
                          void* stream);
/* dx for the loss gradient dy: the rotation by the negative angles. */
dsv_status dsv_rope3d_bwd(const dsv_rope_dims* dims, const void* dy, const dsv_view_strides* dy_strides,
                          const int32_t* pos, const float* table, void* dx, const dsv_view_strides* dx_strides,
                          void* stream);

/*
 * Norm of queries and keys for each head and the rotation in one pass, with the layout change:
 *   n = x / sqrt(mean_d(x^2) + eps) * w,  out = rotation(n)   for q (w = wq) and k (w = wk);
 *   v_out = v  (v and v_out both NULL: no values in this call).
 * wq, wk: bf16 [d] (NULL: ones).  strides: of q, k, v in this order (NULL: all contiguous).
 * q_out, k_out, v_out: contiguous [B][H][N][d], as the attention calls take them.
 * fp32 arithmetic, one rounding to bf16 at the end.  The mean square is an fp32 number too: a row whose
 * squares pass its range (features beyond about 1e18) comes out as 0, and with eps = 0 a row whose squares
 * vanish in it (all features below about 1e-23, zero rows among them) as NaN or infinite, in that row alone.
 */
dsv_status dsv_qk_norm_rope_fwd(const dsv_rope_dims* dims, const void* q, const void* k, const void* v,
                                const dsv_view_strides strides[3], const void* wq, const void* wk,
                                const int32_t* pos, const float* table, void* q_out, void* k_out, void* v_out,
                                void* stream);
/* Bytes of workspace dsv_qk_norm_rope_bwd needs (partial sums of the weights' gradients). */
size_t dsv_qk_norm_rope_bwd_workspace(const dsv_rope_dims* dims);
/*
 * Gradients of the call above: with g = rotation^T(d_out) and xhat = x / sqrt(mean_d(x^2) + eps),
 *   dx = rstd (g w - xhat mean_d(g w xhat)),   dw[d] = sum over B, H, N of g xhat,   dv = d_v_out.
 * d_q_out, d_k_out, d_v_out: contiguous bf16 [B][H][N][d] (d_v_out NULL with dv: no values).
 * q, k: the forward's inputs, strides[0], strides[1].  dq, dk, dv: bf16 views with d_strides[0..2]
 * (NULL: contiguous).  dwq, dwk: fp32 [d], NULL where not wanted; bitwise reproducible (fixed
 * summation order).  ws: at least dsv_qk_norm_rope_bwd_workspace(dims) bytes, 256-byte aligned
 * (not needed, and not read, with both dwq and dwk NULL); one workspace must not serve two calls
 * that can run at the same time.
 */
dsv_status dsv_qk_norm_rope_bwd(const dsv_rope_dims* dims, const void* d_q_out, const void* d_k_out,
                                const void* d_v_out, const void* q, const void* k, const dsv_view_strides strides[2],
                                const void* wq, const void* wk, const int32_t* pos, const float* table, void* dq,
                                void* dk, void* dv, const dsv_view_strides d_strides[3], float* dwq, float* dwk,
                                void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- gated feed-forward
 * The feed-forward of a DiT block up to its down projection: both projections, the activation and
 * the product in one kernel, and its backward.
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) * u
 *   act: DSV_ACT_SILU      g / (1 + exp(-g))
 *        DSV_ACT_GELU_TANH g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))
 * The backward recomputes g and u from x (the forward keeps nothing) and returns
 *   dg = dh u act'(g), du = dh act(g);  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
 * Layouts (contiguous, 16-byte aligned device memory): x, dx bf16 [M][D]; w_gate, w_up, dw_gate,
 * dw_up bf16 [F][D]; h, dh bf16 [M][F].  M is the token count (samples and tokens flattened).
 * Products accumulate in fp32; h and the gradients are rounded to bf16 once, and dg, du once between the
 * backward's kernels, where the tensor cores take them as operands: the gradients are then off by about
 * 2.3e-3 of their norm (1.7e-3 with their own rounding alone).  For one and two tokens, and up to four with
 * D * F <= 2^22, dg and du stay fp32.  Bitwise reproducible.  Outputs must not overlap inputs.
 * Validation before any launch: M, D, F >= 1; D and F multiples of 8; M < 2^31 - 256, D and F <=
 * 2^20; act as above; no NULL, misaligned or overlapping pointer.
 */
typedef enum { DSV_ACT_SILU = 0, DSV_ACT_GELU_TANH = 1 } dsv_activation;

typedef struct {
  int64_t M;     /* tokens */
  int64_t D;     /* features of x */
  int64_t F;     /* features of h */
  int32_t act;   /* dsv_activation */
} dsv_ffn_dims;

/* Bytes of workspace dsv_ffn_gated_fwd needs: 0 but for few tiles of output with a long D, whose
 * products are split over D (at most 20 MB of fp32 sums). */
size_t dsv_ffn_gated_fwd_workspace(const dsv_ffn_dims* dims);
/* ws: at least dsv_ffn_gated_fwd_workspace(dims) bytes, 256-byte aligned (NULL where that is 0); one
 * workspace must not serve two calls that can run at the same time (so too in the backward). */
dsv_status dsv_ffn_gated_fwd(const dsv_ffn_dims* dims, const void* x, const void* w_gate, const void* w_up, void* h,
                             void* ws, size_t ws_bytes, void* stream);
/* Bytes of workspace dsv_ffn_gated_bwd needs: dg and du (4 M F), and the sums of split products (a few
 * tokens: dg and du in fp32, and parts of dx). */
size_t dsv_ffn_gated_bwd_workspace(const dsv_ffn_dims* dims);
/* ws: at least dsv_ffn_gated_bwd_workspace(dims) bytes, 256-byte aligned. */
dsv_status dsv_ffn_gated_bwd(const dsv_ffn_dims* dims, const void* dh, const void* x, const void* w_gate,
                             const void* w_up, void* dx, void* dw_gate, void* dw_up, void* ws, size_t ws_bytes,
                             void* stream);

/* ------------------------------------------- gated residual with the norms around a block's branches
 * What happens where a branch of a DiT block (attention, feed-forward) returns to the residual stream,
 * with the norm and modulation in front of the next branch, in one pass over HBM, and its backward.
 * Per token n of sample b, over its D features:
 *   t = z (post DSV_NORM_NONE)  or  z / sqrt(mean z^2 + eps) * w_post (DSV_NORM_RMS);
 *   r = x + alpha * gate[b] * t;
 *   y = xhat * w_pre * (1 + scale[b]) + shift[b]  with  xhat = (r - mean r) / sqrt(var r + eps)
 *       (pre DSV_NORM_LAYER, var the biased one) or r / sqrt(mean r^2 + eps) (DSV_NORM_RMS);
 *       DSV_NORM_NONE: no y (the last branch of a model), and scale, shift, w_pre, y are NULL.
 * The backward takes the gradients dr (of r along the stream; NULL: none) and dy (of y) and returns, with
 * f = w_pre (1 + scale[b]), g = dr + rstd (dy f - mean(dy f) - xhat mean(dy f xhat)) (RMS: without mean(dy f)):
 *   dx = g,   dz = alpha gate[b] g  or, through the branch's norm, rz (u - zhat mean(u zhat)), u = alpha gate[b] w_post g;
 *   d_gate[b] = alpha sum_n g t,  dw_post = alpha sum_{b,n} gate[b] g zhat,
 *   d_scale[b] = sum_n dy xhat w_pre,  d_shift[b] = sum_n dy,  dw_pre = sum_{b,n} dy xhat (1 + scale[b]).
 * It reads r as the forward stored it (NULL without a norm behind it), recomputes the norms' sums, and keeps nothing.
 * Types: z, y, dy, dz bf16; x, r, dr, dx bf16 or, with stream_f32, fp32; gate, scale, shift, w_post, w_pre bf16, each NULL
 * where it is not there (1, 0, 0, 1, 1); the vectors' gradients fp32, each NULL where not wanted.  fp32 arithmetic and
 * sums, one rounding at each output (the forward's y comes from r before its rounding).  The mean squares are fp32
 * numbers too: features beyond about 1e18 leave their row 0 or NaN, and with eps = 0 a row of zeros becomes NaN and one of
 * features below about 1e-19 loses bits of its norm.
 * Layouts: x, z, r, y, dr, dy, dx, dz contiguous [B][N][D]; gate, scale, shift: rows of D, gate_stride, scale_stride,
 * shift_stride elements apart (multiples of 8; 0: one row for all samples), so that parts of one modulation projection
 * [B][6][D] are passed as they are; d_gate, d_scale, d_shift: rows of D, d_stride elements apart (a multiple of 4, >= D), which may
 * interleave in one [B][6][D] gradient.  With B = 1 no stride is read.
 * Outputs must not overlap inputs or each other, except that r may be x and dx may be dr (the same pointer).
 * Bitwise reproducible.  Validation before any launch: 1 <= B <= 65535, N >= 1, B * N < 2^31; D a multiple of 8 in
 * [8, 8192]; eps >= 0 and finite, alpha finite; pointers 16-byte aligned, NULL only as above.
 */
typedef enum { DSV_NORM_NONE = 0, DSV_NORM_RMS = 1, DSV_NORM_LAYER = 2 } dsv_norm;

typedef struct {
  int64_t B, N, D;
  int32_t post;          /* dsv_norm of the branch's result: none or RMS */
  int32_t pre;           /* dsv_norm in front of the next branch */
  int32_t stream_f32;    /* x, r, dr, dx are fp32 */
  float alpha, eps;
  int64_t gate_stride, scale_stride, shift_stride;   /* elements between samples */
  int64_t d_stride;      /* of d_gate, d_scale, d_shift (backward) */
} dsv_residual_dims;

dsv_status dsv_residual_norm_fwd(const dsv_residual_dims* dims, const void* x, const void* z, const void* gate,
                                 const void* w_post, const void* scale, const void* shift, const void* w_pre, void* r,
                                 void* y, void* stream);
/* Bytes of workspace dsv_residual_norm_bwd needs (partial sums of the vectors' gradients). */
size_t dsv_residual_norm_bwd_workspace(const dsv_residual_dims* dims);
/* ws: at least dsv_residual_norm_bwd_workspace(dims) bytes, 256-byte aligned; one workspace must not serve two calls that
 * can run at the same time. */
dsv_status dsv_residual_norm_bwd(const dsv_residual_dims* dims, const void* dr, const void* dy, const void* r, const void* z,
                                 const void* gate, const void* w_post, const void* scale, const void* w_pre, void* dx,
                                 void* dz, float* d_gate, float* dw_post, float* d_scale, float* d_shift, float* dw_pre,
                                 void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------- products of a few vectors with 4-bit weights
 * The projection that makes a block's modulation vectors from its condition (one vector a sample), and any other
 * product of a few vectors, with weights held in 4 bits:
 *   w[f, c] = scale[f, c / group] * (q[f, c] - zero[f, c / group]),   q in 0 .. 15,
 *   y = x W^T + bias   and, the weights being frozen,   dx = dy W.
 * data: uint8 [F][D / 2], q of column 2 i in the low four bits of byte i and of column 2 i + 1 in the high four;
 * scale: bf16 [F][D / group], finite; zero: uint8 [F][D / group], 0 .. 15 (its low four bits are read), or NULL: 8.
 * x, dx bf16 [M][D]; y bf16 [M][F]; bias bf16 [F] or NULL; dy [M][F], bf16 or, with dy_f32, fp32.  Contiguous.
 * Sums are fp32, with one rounding at the output.  Forward: products are exact, and a group's sum of
 * x (q - zero) / 64 is taken before its scale, so that it may overflow for |x| above 2^123.  Backward: dy * scale, rounded to fp32, enters
 * its products as two (dy in bf16) or three (fp32) bf16 numbers that add up to it.
 * Bitwise reproducible.  Outputs must not overlap inputs.
 * Validation before any launch: 1 <= M <= 64; F >= 1; group 32, 64 or 128; D a multiple of group, D <= 2^20, F * D <= 2^40.
 */
typedef struct {
  int64_t M;             /* vectors (dsv_w4_quantize does not read it) */
  int64_t D, F;          /* columns and rows of W */
  int32_t group;         /* columns to a scale */
  int32_t dy_f32;        /* dy is fp32 (backward) */
} dsv_w4_dims;

/* Weights of 4 bits from w bf16 [F][D] (finite), once per model: each group's scale is max |w| / 7 (zero NULL) or (max(w, 0) -
 * min(w, 0)) / 15 with the zero point -min(w, 0) / scale, rounded to bf16 and to a whole number; q is w / scale rounded to the
 * nearest whole number (ties to even) plus the zero point, held to 0 .. 15.  A group of zeros has the scale 0. */
dsv_status dsv_w4_quantize(const dsv_w4_dims* dims, const void* w, uint8_t* data, void* scale, uint8_t* zero, void* stream);
dsv_status dsv_w4_linear_fwd(const dsv_w4_dims* dims, const void* x, const uint8_t* data, const void* scale,
                             const uint8_t* zero, const void* bias, void* y, void* stream);
/* Bytes of workspace dsv_w4_linear_bwd needs (partial sums of dx). */
size_t dsv_w4_linear_bwd_workspace(const dsv_w4_dims* dims);
/* ws: at least dsv_w4_linear_bwd_workspace(dims) bytes, 256-byte aligned; one workspace must not serve two calls that can
 * run at the same time. */
dsv_status dsv_w4_linear_bwd(const dsv_w4_dims* dims, const void* dy, const uint8_t* data, const void* scale,
                             const uint8_t* zero, void* dx, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSV_H */
