// Products of a few vectors with weights of 4 bits:  w[f, c] = scale[f, c / G] (q[f, c] - zero[f, c / G]),
//   y = x W^T + bias  and  dx = dy W  (include/dsv.h), and the rounding of bf16 weights to that form.
//
// The weights' bytes are the work: F D / 2 of them and 2 F D / G of scales, against 2 M F D operations for M of 1 to 64.
// At HBM's rate an SM has to turn 46 weights a clock into products, where plain fp32 arithmetic (unpack, convert,
// multiply) takes about three instructions a weight of the 128 it can issue to its lanes: so the products run on the
// tensor cores through mma.sync (16 x 8 x 16), whose operands come straight from the registers that the weights
// were loaded into.  tcgen05 would want them as bf16 in shared memory, 128 rows at a time, for at most 64 columns.
//   A value is unpacked as the bf16 number 128 + q (its four bits or-ed into 0x4300) and 128 + zero is subtracted, both
// exact; the scale multiplies fp32 sums (forward) or the other operand (backward).  Sums are fp32, with one rounding at
// the output.
#include "dsv_block.h"
#include "dsv_common.cuh"

namespace dsv {
namespace {

constexpr uint32_t kMagic = 0x43004300u;   // bf16 128 in both halves: or-ing q into the low bits gives 128 + q

DSV_DEVICE uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// Values i and i + 4 of a word's eight, less the zero point (zz: 128 + zero in both halves).
DSV_DEVICE uint32_t unpack_pair(uint32_t word, int i, uint32_t zz) {
  return sub_bf16x2(((word >> (4 * i)) & 0x000f000fu) | kMagic, zz);
}
DSV_DEVICE uint32_t zero_pair(const uint8_t* zero, int64_t at) {
  return zero ? kMagic + (zero[at] & 15u) * 0x00010001u : kMagic + 0x00080008u;
}

// ---------------------------------------------------------------- forward
// A CTA takes 16 RS rows of W; its four warps share the columns in chunks of 128 (warp w: chunks w, w + 4, ..) and add up
// in the end.  In a chunk a lane (g = lane / 4, t = lane % 4) loads columns 32 t .. 32 t + 31 of rows g and g + 8 (16
// bytes each): eight products of 16 columns, each with columns of all four t.  With G < 128 these are of
// different groups, whose sums must stay apart until the scales: the 8 columns of the other operand are then 8 G / 128
// vectors for each group, which are zero in the lanes t of other groups.
constexpr int kFwdWarps = 4;

template <int G, int NT, int RS>
__global__ void __launch_bounds__(32 * kFwdWarps)
w4_fwd_kernel(W4Params p) {
  constexpr int GP = 128 / G, VT = 8 / GP;       // groups of a chunk, vectors of a tile of eight
  __shared__ float red[kFwdWarps][RS * 16][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * (16 * RS), m0 = static_cast<int64_t>(blockIdx.y) * (VT * NT);
  const int64_t row_bytes = p.D / 2, row_groups = p.D / G;
  const int chunks = static_cast<int>((p.D + 127) / 128);
  const int part = t * 32 / G;                   // group of this lane's columns in a chunk

  int64_t row[RS][2];                            // rows past the last read the last, and are not stored
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row[i][h] = f0 + i * 16 + h * 8 + g;
      if (row[i][h] >= p.F) row[i][h] = p.F - 1;
    }
  float acc[RS][NT][4];
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.f;

  for (int c = warp; c < chunks; c += kFwdWarps) {
    const int64_t col = static_cast<int64_t>(c) * 128 + t * 32;
    const bool inside = col < p.D;               // D is a multiple of 32
    uint4 a[RS][2];
    uint32_t zz[RS][2];
    float sc[RS][2];
    const int64_t group = min(static_cast<int64_t>(c) * GP + part, row_groups - 1);
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[i][h] = inside ? __ldcs(reinterpret_cast<const uint4*>(p.data + row[i][h] * row_bytes + col / 2)) : make_uint4(0, 0, 0, 0);
        zz[i][h] = zero_pair(p.zero, row[i][h] * row_groups + group);
        sc[i][h] = __bfloat162float(p.scale[row[i][h] * row_groups + group]);
      }
    uint32_t b[NT][16];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t m = m0 + n * VT + g % VT;
      const bool mine = inside && g / VT == part && m < p.M;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 x = mine ? __ldg(reinterpret_cast<const uint4*>(p.x + m * p.D + col) + w) : make_uint4(0, 0, 0, 0);
        b[n][4 * w] = __byte_perm(x.x, x.z, 0x5410);       // columns 0 and 4, as unpack_pair gives them
        b[n][4 * w + 1] = __byte_perm(x.x, x.z, 0x7632);   // 1 and 5
        b[n][4 * w + 2] = __byte_perm(x.y, x.w, 0x5410);   // 2 and 6
        b[n][4 * w + 3] = __byte_perm(x.y, x.w, 0x7632);   // 3 and 7
      }
    }
#pragma unroll
    for (int i = 0; i < RS; ++i) {
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
      const uint32_t w0[4] = {a[i][0].x, a[i][0].y, a[i][0].z, a[i][0].w}, w1[4] = {a[i][1].x, a[i][1].y, a[i][1].z, a[i][1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int w = k / 2, e = 2 * (k % 2);
        const uint32_t frag[4] = {unpack_pair(w0[w], e, zz[i][0]), unpack_pair(w1[w], e, zz[i][1]),
                                  unpack_pair(w0[w], e + 1, zz[i][0]), unpack_pair(w1[w], e + 1, zz[i][1])};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma_bf16_16816(s[n], frag, b[n][4 * w + e], b[n][4 * w + e + 1]);
      }
      // sums j = 0, 1: row g; 2, 3: row g + 8; both of tile columns 2 t, 2 t + 1, which are of group 2 t / VT = part
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][n][j] += sc[i][j / 2] * s[n][j];
    }
  }
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[warp][i * 16 + g + 8 * (j / 2)][n * 8 + 2 * t + j % 2] = acc[i][n][j];
  __syncthreads();
  for (int i = threadIdx.x; i < RS * 16 * VT * NT; i += 32 * kFwdWarps) {
    const int r = i % (RS * 16), v = i / (RS * 16);
    const int64_t f = f0 + r, m = m0 + v;
    if (f >= p.F || m >= p.M) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w)
#pragma unroll
      for (int q = 0; q < GP; ++q) s += red[w][r][v / VT * 8 + q * VT + v % VT];
    if (p.bias) s += __bfloat162float(p.bias[f]);
    p.y[m * p.F + f] = __float2bfloat16(s);
  }
}

// ---------------------------------------------------------------- backward
// dx[m, c] = sum_f (dy[m, f] scale[f, c / G]) (q[f, c] - zero): the contraction runs over the rows.  A warp takes 64 columns
// and steps of 16 rows: a lane (g, t) loads its eight columns 8 g .. 8 g + 7 of rows 4 t .. 4 t + 3 (4 bytes each), pairs the
// rows, and product j of four is of columns 8 g + 2 j and 8 g + 2 j + 1.  The other operand, dy times the scale, is held as
// two bf16 numbers, the rounded value and what it left (16 bits: exact for dy in bf16, 2^-16 of the value for fp32), in
// neighbouring columns of the tile, so that a lane's two sums of a row add up to one result.  Groups of 32: the 64 columns
// are of two groups, and a tile holds each vector once for each.
//   A CTA is two such column blocks by four runs of rows, whose sums it adds; the CTAs of one column block share the rows
// of W in `splits` runs, whose partial results w4_join_kernel adds in order.
constexpr int kBwdColWarps = 2, kBwdRowWarps = 4, kBwdWarps = kBwdColWarps * kBwdRowWarps;
constexpr int kBwdCols = 64 * kBwdColWarps;
constexpr int64_t kBwdWantCtas = 4 * 152;
struct W4BwdPlan {
  int64_t col_blocks, splits, rows;     // rows of W to a CTA, a multiple of 16 kBwdRowWarps
};
W4BwdPlan w4_bwd_plan(int64_t D, int64_t F) {
  W4BwdPlan q;
  const int64_t step = 16 * kBwdRowWarps;
  q.col_blocks = (D + kBwdCols - 1) / kBwdCols;
  q.splits = (kBwdWantCtas + q.col_blocks - 1) / q.col_blocks;
  const int64_t most = (F + step - 1) / step;
  if (q.splits > most) q.splits = most;
  q.rows = ((F + q.splits - 1) / q.splits + step - 1) / step * step;
  q.splits = (F + q.rows - 1) / q.rows;
  return q;
}

template <int G, int NT, bool F32>
__global__ void __launch_bounds__(32 * kBwdWarps)
w4_bwd_kernel(W4Params p, W4BwdPlan plan) {
  constexpr int GP = G < 64 ? 64 / G : 1, VT = 4 / GP;   // groups of a warp's columns, vectors of a tile
  __shared__ float red[kBwdRowWarps][VT * NT][kBwdCols];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cw = warp % kBwdColWarps, rw = warp / kBwdColWarps;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kBwdCols + cw * 64, m0 = static_cast<int64_t>(blockIdx.z) * (VT * NT);
  const int64_t f_lo = blockIdx.y * plan.rows, f_hi = min(f_lo + plan.rows, p.F);
  const int64_t row_bytes = p.D / 2, row_groups = p.D / G;
  const bool inside = c0 + 8 * g < p.D;
  const int64_t my_group = min((c0 + 8 * g) / G, row_groups - 1);   // of the lane's columns
  // of the lane's place in the other operand: tile column g is (group, vector, rounded value or rest)
  const int64_t b_group = min(c0 / G + g / (2 * VT), row_groups - 1);
  const int b_vec = g / 2 % VT;

  float acc[NT][4][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][j][i] = 0.f;

  for (int64_t f = f_lo + rw * 16; f < f_hi; f += 16 * kBwdRowWarps) {
    uint32_t w[4], z[4];
    float b[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = f + 4 * t + i;
      const bool in = row < f_hi;
      w[i] = in && inside ? __ldcs(reinterpret_cast<const uint32_t*>(p.data + row * row_bytes + (c0 + 8 * g) / 2)) : 0u;
      z[i] = in && p.zero ? p.zero[row * row_groups + my_group] & 15u : 8u;
      const float sc = in ? __bfloat162float(p.scale[row * row_groups + b_group]) : 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t m = m0 + n * VT + b_vec;
        float d = 0.f;
        if (in && m < p.M)
          d = F32 ? static_cast<const float*>(p.dy)[m * p.F + row]
                  : __bfloat162float(static_cast<const bf16*>(p.dy)[m * p.F + row]);
        b[n][i] = d * sc;
      }
    }
    uint32_t other[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t hi = pack_bf16x2(b[n][2 * h], b[n][2 * h + 1]);
        // an infinite value leaves no rest
        const float r0 = isinf(bf16_lo(hi)) ? 0.f : b[n][2 * h] - bf16_lo(hi), r1 = isinf(bf16_hi(hi)) ? 0.f : b[n][2 * h + 1] - bf16_hi(hi);
        other[n][h] = g % 2 ? pack_bf16x2(r0, r1) : hi;
      }
    const uint32_t z01 = kMagic + z[0] + (z[1] << 16), z23 = kMagic + z[2] + (z[3] << 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t pick = j * 0x0011u + (4 + j) * 0x1100u;
      const uint32_t p01 = __byte_perm(w[0], w[1], pick), p23 = __byte_perm(w[2], w[3], pick);
      const uint32_t frag[4] = {sub_bf16x2((p01 & 0x000f000fu) | kMagic, z01), sub_bf16x2(((p01 >> 4) & 0x000f000fu) | kMagic, z01),
                                sub_bf16x2((p23 & 0x000f000fu) | kMagic, z23), sub_bf16x2(((p23 >> 4) & 0x000f000fu) | kMagic, z23)};
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_bf16_16816(acc[n][j], frag, other[n][0], other[n][1]);
    }
  }
  // sums i = 0, 1 are column 8 g + 2 j, 2, 3 column 8 g + 2 j + 1; tile columns 2 t, 2 t + 1: value and rest of group t / VT,
  // vector t % VT, which counts for the columns of that group
  if (GP == 1 || (8 * g) / G == t / VT)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        red[rw][n * VT + t % VT][cw * 64 + 8 * g + 2 * j] = acc[n][j][0] + acc[n][j][1];
        red[rw][n * VT + t % VT][cw * 64 + 8 * g + 2 * j + 1] = acc[n][j][2] + acc[n][j][3];
      }
  __syncthreads();
  for (int i = threadIdx.x; i < VT * NT * kBwdCols; i += 32 * kBwdWarps) {
    const int v = i / kBwdCols, c = i % kBwdCols;
    const int64_t m = m0 + v, col = static_cast<int64_t>(blockIdx.x) * kBwdCols + c;
    if (m >= p.M || col >= p.D) continue;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kBwdRowWarps; ++r) s += red[r][v][c];
    p.partial[(blockIdx.y * p.M + m) * p.D + col] = s;
  }
}
__global__ void __launch_bounds__(128)
w4_join_kernel(W4Params p, int64_t splits) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x, n = p.M * p.D;
  if (i >= n) return;
  float s = 0.f;
  for (int64_t k = 0; k < splits; ++k) s += p.partial[k * n + i];
  p.dx[i] = __float2bfloat16(s);
}

// ---------------------------------------------------------------- from bf16
// G / 8 lanes hold a group, eight weights each.  Without zero points the scale is max |w| / 7, else the range of the
// group and 0 in 15 steps, both rounded to bf16; values are rounded to the nearest step (ties to even).
template <int G>
__global__ void __launch_bounds__(256)
w4_quantize_kernel(W4Params p) {
  constexpr int L = G / 8;
  const int64_t vec = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, vecs = p.F * p.D / 8;
  float v[8], lo = 0.f, hi = 0.f;
  const bool inside = vec < vecs;
  const uint4 raw = inside ? reinterpret_cast<const uint4*>(p.w)[vec] : make_uint4(0, 0, 0, 0);
  const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = j % 2 ? bf16_hi(words[j / 2]) : bf16_lo(words[j / 2]);
    lo = fminf(lo, v[j]);
    hi = fmaxf(hi, v[j]);
  }
#pragma unroll
  for (int o = L / 2; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!inside) return;
  const bf16 scale = __float2bfloat16(p.zero ? (hi - lo) / 15.f : fmaxf(-lo, hi) / 7.f);
  const float s = __bfloat162float(scale);
  const float zero = !p.zero ? 8.f : s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 0.f;
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q = s > 0.f ? fminf(fmaxf(rintf(v[j] / s) + zero, 0.f), 15.f) : zero;
    out |= static_cast<uint32_t>(q) << (4 * j);
  }
  reinterpret_cast<uint32_t*>(p.data)[vec] = out;
  if (vec % L == 0) {
    p.scale[vec / L] = scale;
    if (p.zero) p.zero[vec / L] = static_cast<uint8_t>(zero);
  }
}

template <int G, int NT>
cudaError_t fwd(const W4Params& p, cudaStream_t stream) {
  constexpr int VT = 8 * G / 128;
  const dim3 grid(static_cast<unsigned>((p.F + 31) / 32), static_cast<unsigned>((p.M + VT * NT - 1) / (VT * NT)));
  w4_fwd_kernel<G, NT, 2><<<grid, 32 * kFwdWarps, 0, stream>>>(p);
  return cudaGetLastError();
}
template <int G>
cudaError_t fwd_group(const W4Params& p, cudaStream_t stream) {
  constexpr int VT = 8 * G / 128;
  return p.M <= VT ? fwd<G, 1>(p, stream) : p.M <= 2 * VT ? fwd<G, 2>(p, stream) : fwd<G, 4>(p, stream);
}
template <int G, int NT>
cudaError_t bwd(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  constexpr int VT = G < 64 ? 2 : 4;
  const dim3 grid(static_cast<unsigned>(plan.col_blocks), static_cast<unsigned>(plan.splits),
                  static_cast<unsigned>((p.M + VT * NT - 1) / (VT * NT)));
  if (p.dy_f32)
    w4_bwd_kernel<G, NT, true><<<grid, 32 * kBwdWarps, 0, stream>>>(p, plan);
  else
    w4_bwd_kernel<G, NT, false><<<grid, 32 * kBwdWarps, 0, stream>>>(p, plan);
  return cudaGetLastError();
}
template <int G>
cudaError_t bwd_group(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  constexpr int VT = G < 64 ? 2 : 4;
  return p.M <= VT ? bwd<G, 1>(p, plan, stream) : p.M <= 2 * VT ? bwd<G, 2>(p, plan, stream) : bwd<G, 4>(p, plan, stream);
}

}  // namespace

size_t w4_bwd_workspace(int64_t M, int64_t D, int64_t F) {
  return static_cast<size_t>(w4_bwd_plan(D, F).splits * M * D) * sizeof(float);
}

cudaError_t launch_w4_fwd(const W4Params& p, cudaStream_t stream) {
  ProfScope prof("w4_linear_fwd", stream);
  return p.group == 32 ? fwd_group<32>(p, stream) : p.group == 64 ? fwd_group<64>(p, stream) : fwd_group<128>(p, stream);
}

cudaError_t launch_w4_bwd(const W4Params& p, cudaStream_t stream) {
  const W4BwdPlan plan = w4_bwd_plan(p.D, p.F);
  {
    ProfScope prof("w4_linear_bwd", stream);
    const cudaError_t e = p.group == 32 ? bwd_group<32>(p, plan, stream) : p.group == 64 ? bwd_group<64>(p, plan, stream)
                                                                                         : bwd_group<128>(p, plan, stream);
    if (e != cudaSuccess) return e;
  }
  ProfScope prof("w4_join", stream);
  w4_join_kernel<<<static_cast<unsigned>((p.M * p.D + 127) / 128), 128, 0, stream>>>(p, plan.splits);
  return cudaGetLastError();
}

cudaError_t launch_w4_quantize(const W4Params& p, cudaStream_t stream) {
  ProfScope prof("w4_quantize", stream);
  const unsigned ctas = static_cast<unsigned>((p.F * p.D / 8 + 255) / 256);
  if (p.group == 32) w4_quantize_kernel<32><<<ctas, 256, 0, stream>>>(p);
  else if (p.group == 64) w4_quantize_kernel<64><<<ctas, 256, 0, stream>>>(p);
  else w4_quantize_kernel<128><<<ctas, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dsv
