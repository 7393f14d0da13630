// Products of a few vectors with weights of 4 bits:  w[f, c] = scale[f, c / G] (q[f, c] - zero[f, c / G]),
//   y = x W^T + bias  and  dx = dy W  (include/dsv.h), and the rounding of bf16 weights to that form.
//
// The weights' bytes are the work: F D / 2 of them and 2 F D / G of scales, against 2 M F D operations for M of 1 to 64.
// At HBM's rate an SM has to turn 46 weights a clock into products, where plain fp32 arithmetic (unpack, convert,
// multiply) takes about three instructions a weight of the 128 it can issue to its lanes: so the products run on the
// tensor cores through mma.sync (16 x 8 x 16), whose operands come straight from the registers that the weights
// were loaded into.  tcgen05 would want them as bf16 in shared memory, 128 rows at a time, for at most 64 columns.
//   Four bits that a mask leaves at the foot of a bf16 number are q 2^-133, a subnormal one, and four bits above them 16 q 2^-133:
// the numbers up to 255 2^-133 are evenly spaced.  One fma (which keeps subnormal numbers) makes (q - zero) / 64 of either, with
// nothing lost and without a shift: the integer pipe, which unpacks at half the rate of the others, is the busiest here.  The scale multiplies fp32 sums (forward) or the other operand (backward); the 64
// comes back into the finished sums, a power of two.  Sums are fp32, with one rounding at the output.
//   Forward, 294,912 x 2048 and two vectors: 63 us, 5.1 TB/s (0.77 of the copy rate); two instructions in three clocks on every
// scheduler, 72 of 170 to unpack.  Backward, 98,304 x 2048 and four vectors: 38 us for dy in fp32, 2.8 TB/s, and 35 in bf16; it unpacks
// with one more permutation a pair and makes the other operand besides, behind two barriers a chunk: no unit is full (issue slots 60 %).
#include <type_traits>

#include "dsv_block.h"
#include "dsv_common.cuh"

namespace dsv {
namespace {

constexpr float kUnit = 64.f;
// -zero / 64 in both halves of a register.
DSV_DEVICE __nv_bfloat162 zero_pair(uint32_t zero) {
  return __float2bfloat162_rn(static_cast<int>(zero & 15u) * (-1.f / kUnit));
}
// (q - zero) / 64 of the halves' four bits 0 .. 3 (`high`: 4 .. 7).
template <bool HIGH>
DSV_DEVICE uint32_t unpack_pair(uint32_t pair, __nv_bfloat162 zero) {
  const uint32_t bits = pair & (HIGH ? 0x00f000f0u : 0x000f000fu);
  const __nv_bfloat162 unit = __float2bfloat162_rn(HIGH ? 0x1p123f : 0x1p127f);
  const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&bits), unit, zero);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// -zero / 64 of two bytes.
DSV_DEVICE uint32_t zero_of2(uint32_t zeros) {
  return pack_bf16x2(static_cast<int>(zeros & 15u) * (-1.f / kUnit), static_cast<int>(zeros >> 8 & 15u) * (-1.f / kUnit));
}
DSV_DEVICE uint32_t read_bytes2(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(at) : "memory");
  return v;
}

// One, two or four 16-bit numbers, as one load brings them.
template <int N>
struct Pack {
  using type = std::conditional_t<N == 2, unsigned short, std::conditional_t<N == 4, unsigned int, uint2>>;
  uint32_t v[N == 8 ? 2 : 1];
  DSV_DEVICE Pack& operator=(const type& a) {
    if constexpr (N == 8) v[0] = a.x, v[1] = a.y;
    else v[0] = a;
    return *this;
  }
  DSV_DEVICE uint32_t get(int q) const { return v[q / 2] >> (16 * (q % 2)) & 0xffffu; }
  DSV_DEVICE void set(int q, uint32_t a) { v[q / 2] |= a << (16 * (q % 2)); }
};

// ---------------------------------------------------------------- forward
// A CTA takes 16 RS rows of W; its four warps share the columns in chunks of 128 (warp w: chunks w, w + 4, ..) and add up
// in the end.  A warp's next chunks are on their way into shared memory (cp.async), from where a lane (g = lane / 4,
// t = lane % 4) takes four words (32 values) of rows g and g + 8, G / 32 of them next to each other: then the sixteen columns of a
// product are all of one group, and its fp32 sums are scaled once a group.
constexpr int kFwdWarps = 4;
constexpr int kStages = 2;                       // chunks of a warp on their way
// Bytes between the 64-byte rows of a chunk in shared memory, so that what a load reads at once (16 bytes of two rows, 8 of four or
// 4 of eight, times t) is in different banks.
template <int G>
constexpr int fwd_pitch() {
  return G == 128 ? 64 : G == 64 ? 96 : 80;
}
template <int G, int NT, int RS>
constexpr int fwd_smem() {
  constexpr int ring = kStages * RS * 16 * fwd_pitch<G>() * kFwdWarps, red = kFwdWarps * RS * 16 * (8 * NT + 1) * 4;
  return ring > red ? ring : red;
}
// Four, eight or sixteen bytes of shared memory.
template <int N>
DSV_DEVICE void read_words(uint32_t at, uint32_t* v) {
  if constexpr (N == 1) asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v[0]) : "r"(at) : "memory");
  if constexpr (N == 2) asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v[0]), "=r"(v[1]) : "r"(at) : "memory");
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
}

// A product onto zeros.
DSV_DEVICE void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

template <int G, int NT, int RS, bool ZERO>
__global__ void __launch_bounds__(32 * kFwdWarps, NT == 1 ? 5 : NT == 2 ? 4 : 2)
w4_fwd_kernel(W4Params p) {
  constexpr int GP = 128 / G, WG = G / 32, kPitch = fwd_pitch<G>();   // groups of a chunk, a lane's words of a group
  extern __shared__ __align__(16) unsigned char shared[];   // the weights on their way, then the warps' sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * (16 * RS);
  const int m0 = blockIdx.y * (8 * NT);
  const int D = static_cast<int>(p.D), M = static_cast<int>(p.M), row_groups = D / G, chunks = (D + 127) / 128;
  const int last = static_cast<int>(min(p.F - f0, static_cast<int64_t>(16 * RS))) - 1;

  // Rows past the last read the last, and are not stored.  Columns past the last read the last ones: the vectors are 0 there.
  uint32_t scale_at[RS][2];                      // element of the scales (and zero points) of the lane's rows
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) scale_at[i][h] = min(i * 16 + h * 8 + g, last) * row_groups;
  const bf16* const scales = p.scale + f0 * row_groups;
  const uint8_t* const zeros = ZERO ? p.zero + f0 * row_groups : nullptr;
  const bool whole = D % 128 == 0;               // a chunk's groups of a row are one aligned load
  Pack<2 * GP> scale[RS][2];
  uint8_t zero[ZERO ? RS : 1][2][GP];
  auto load_scales = [&](int c) {
#pragma unroll
    for (int i = 0; i < RS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (whole) {
          scale[i][h] = *reinterpret_cast<const typename Pack<2 * GP>::type*>(scales + (scale_at[i][h] + c * GP));
        } else {
          scale[i][h] = Pack<2 * GP>{};
#pragma unroll
          for (int q = 0; q < GP; ++q)
            scale[i][h].set(q, reinterpret_cast<const uint16_t*>(scales)[scale_at[i][h] + min(c * GP + q, row_groups - 1)]);
        }
        if (ZERO)
#pragma unroll
          for (int q = 0; q < GP; ++q) zero[i][h][q] = zeros[scale_at[i][h] + min(c * GP + q, row_groups - 1)];
      }
  };
  // Lane l brings part l % 4 of rows l / 4, l / 4 + 8, ..
  const uint32_t ring = smem_u32(shared) + warp * (kStages * RS * 16 * kPitch);
  uint32_t row_at[2 * RS];
#pragma unroll
  for (int i = 0; i < 2 * RS; ++i) row_at[i] = min(i * 8 + g, last) * (D / 2);
  const uint8_t* const data = p.data + f0 * (D / 2);
  auto issue = [&](int c, int stage) {
    if (c < chunks) {
      const uint32_t col = min(c * 128 + t * 32, D - 32) / 2, to = ring + stage * (RS * 16 * kPitch) + g * kPitch + 16 * t;
#pragma unroll
      for (int i = 0; i < 2 * RS; ++i) cp_async_16(to + i * 8 * kPitch, data + (row_at[i] + col), true);
    }
    cp_async_commit();                           // one group a chunk, so that the wait below counts chunks
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) issue(warp + s * kFwdWarps, s);
  load_scales(warp < chunks ? warp : 0);

  float acc[RS][NT][4];
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][n][j] = 0.f;
  int stage = 0;
  for (int c = warp; c < chunks; c += kFwdWarps) {
    uint32_t b[NT][16];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int m = m0 + n * 8 + g;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int col = c * 128 + w / WG * G + t * (8 * WG) + w % WG * 8;
        const uint4 x = col < D && m < M ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m) * D + col)) : make_uint4(0, 0, 0, 0);
        b[n][4 * w] = __byte_perm(x.x, x.z, 0x5410);       // columns 0 and 4, as the halves of a word have them
        b[n][4 * w + 1] = __byte_perm(x.x, x.z, 0x7632);   // 1 and 5
        b[n][4 * w + 2] = __byte_perm(x.y, x.w, 0x5410);   // 2 and 6
        b[n][4 * w + 3] = __byte_perm(x.y, x.w, 0x7632);   // 3 and 7
      }
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t mine = ring + stage * (RS * 16 * kPitch) + g * kPitch + 4 * WG * t;
#pragma unroll
    for (int i = 0; i < RS; ++i) {
#pragma unroll
      for (int q = 0; q < GP; ++q) {
        uint32_t w0[WG], w1[WG];
        read_words<WG>(mine + i * 16 * kPitch + q * (G / 2), w0);
        read_words<WG>(mine + (i * 16 + 8) * kPitch + q * (G / 2), w1);
        const __nv_bfloat162 z0 = zero_pair(ZERO ? zero[i][0][q] : 8), z1 = zero_pair(ZERO ? zero[i][1][q] : 8);
        float s[NT][4];
#pragma unroll
        for (int k = 0; k < 2 * WG; ++k) {
          const int w = k / 2, e = 2 * (k % 2);   // values e and e + 4, e + 1 and e + 5 of the word
          const uint32_t p0 = w0[w] >> (4 * e), p1 = w1[w] >> (4 * e);
          const uint32_t frag[4] = {unpack_pair<false>(p0, z0), unpack_pair<false>(p1, z1), unpack_pair<true>(p0, z0), unpack_pair<true>(p1, z1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t b0 = b[n][4 * (q * WG + w) + e], b1 = b[n][4 * (q * WG + w) + e + 1];
            if (k) mma_bf16_16816(s[n], frag, b0, b1);
            else mma_first(s[n], frag, b0, b1);
          }
        }
        // sums j = 0, 1: row g; 2, 3: row g + 8; of vectors 2 t, 2 t + 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][n][j] += __uint_as_float(scale[i][j / 2].get(q) << 16) * s[n][j];
      }
    }
    if (c + kFwdWarps < chunks) load_scales(c + kFwdWarps);
    __syncwarp();
    issue(c + kStages * kFwdWarps, stage);       // into the stage that this chunk has left
    stage = stage + 1 < kStages ? stage + 1 : 0;
  }
  cp_async_wait<0>();
  __syncthreads();
  float(*const red)[RS * 16][8 * NT + 1] = reinterpret_cast<float(*)[RS * 16][8 * NT + 1]>(shared);
#pragma unroll
  for (int i = 0; i < RS; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[warp][i * 16 + g + 8 * (j / 2)][n * 8 + 2 * t + j % 2] = acc[i][n][j];
  __syncthreads();
  for (int i = threadIdx.x; i < RS * 16 * 8 * NT; i += 32 * kFwdWarps) {
    const int r = i % (RS * 16), v = i / (RS * 16);
    if (r > last || m0 + v >= M) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w) s += red[w][r][v];
    s *= kUnit;
    if (p.bias) s += __bfloat162float(p.bias[f0 + r]);
    p.y[(m0 + v) * p.F + f0 + r] = __float2bfloat16(s);
  }
}

// ---------------------------------------------------------------- backward
// dx[m, c] = sum_f (dy[m, f] scale[f, c / G]) (q[f, c] - zero): the contraction runs over the rows.  A CTA takes 128 columns
// and a run of rows in chunks of 256: two warps side by side, four below each other with 64 rows of a chunk each, the
// next chunks on their way into shared memory.  In a step of 16 rows a lane (g, t) holds eight columns of rows t, t + 4, t + 8
// and t + 12, pairs the rows, and product j of four is of two of its columns; the columns of a product are all of one group.
//   The other operand, dy times the scale, is held as bf16 numbers that add up to it: its first eight bits and the next, 16 bits
// between them, which is all that a product of bf16 numbers has, in neighbouring columns of the tile, so that a lane's two sums
// of a row add up to one result.  For dy in fp32 a third number holds the last eight bits of 24: it takes a second product,
// onto the sums of the column of the rests (98,304 x 2048, four vectors: 39 us instead of 34 with some 17 bits, which left 18 of
// 8192 outputs on the wrong side of their rounding; none is now).  The operand is the same for all columns of a group, so the CTA makes it once a chunk in
// shared memory, in the order in which the lanes take it.
//   The CTAs of one column block share the rows of W in `splits` runs, whose partial results w4_join_kernel adds in order.
constexpr int kBwdColWarps = 2, kBwdRowWarps = 4, kBwdWarps = kBwdColWarps * kBwdRowWarps;
constexpr int kBwdCols = 64 * kBwdColWarps, kBwdSteps = 4, kBwdRows = 16 * kBwdSteps * kBwdRowWarps, kQuads = kBwdRows / 4;
// A row of a chunk is 64 bytes; the halves of every third and fourth of four rows are exchanged, so that the four rows t and
// the 32 bytes of a warp's columns are in different banks.
constexpr int kBwdStage = kBwdRows * kBwdCols / 2, kBwdStages = 3;
struct W4BwdPlan {
  int64_t col_blocks, splits, rows;     // rows of W to a CTA, a multiple of kBwdRows
};
// CTAs of an SM at a time.  Two tiles of vectors, two groups a warp and a third number each take registers (and shared memory, which
// L1 then lacks): any two of them leave room for two (98,304 x 2048, dy in fp32: eight vectors, groups of 64, 66 us with three CTAs and
// 55 with two, four vectors, groups of 32, 60 and 52; dy in bf16, groups of 64, the other way round: 48 and 55).
constexpr int bwd_ctas(int group, int tiles, bool f32) { return (tiles == 2) + (group < 64) + f32 > 1 ? 2 : 3; }
// Runs so that all SMs have their CTAs at a time; passes over more than eight vectors follow one another (as many runs fewer left
// SMs idle: 32 vectors 306 us instead of 279).
W4BwdPlan w4_bwd_plan(int64_t M, int64_t D, int64_t F, int group, bool f32) {
  W4BwdPlan q;
  q.col_blocks = (D + kBwdCols - 1) / kBwdCols;
  q.splits = bwd_ctas(group, M > 4 ? 2 : 1, f32) * 152 / q.col_blocks;
  const int64_t most = (F + kBwdRows - 1) / kBwdRows;
  if (q.splits > most) q.splits = most;
  if (q.splits < 1) q.splits = 1;
  q.rows = ((F + q.splits - 1) / q.splits + kBwdRows - 1) / kBwdRows * kBwdRows;
  q.splits = (F + q.rows - 1) / q.rows;
  return q;
}
template <int G, int NT, bool ZERO, bool F32>
constexpr int bwd_smem() {
  constexpr int use = kBwdStages * kBwdStage + kBwdCols / G * kQuads * (NT * (F32 ? 96 : 64) + (ZERO ? 8 : 0));
  constexpr int red = kBwdRowWarps * 4 * NT * kBwdCols * 4;
  return use > red ? use : red;
}

// Four rows' numbers as N bf16 numbers each, every one the upper half of what those before it leave (cut, not rounded: a
// finite number stays finite however large it is, and N times eight bits are as many): part k in 2 k and 2 k + 1.  An infinite
// one leaves NaN, for which the maximum takes -2^120, which is below every rest that there is: next to the infinity it is nothing.
template <int N>
DSV_DEVICE void split4(const float (&v)[4], uint32_t (&parts)[2 * N]) {
  const __nv_bfloat162 least = __float2bfloat162_rn(-0x1p120f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a = v[2 * h], b = v[2 * h + 1];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t cut = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
      a -= bf16_lo(cut);
      b -= bf16_hi(cut);
      const __nv_bfloat162 r = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&cut), least);
      parts[2 * k + h] = k ? *reinterpret_cast<const uint32_t*>(&r) : cut;
    }
  }
}

template <int G, int NT, bool ZERO, bool F32>
__global__ void __launch_bounds__(32 * kBwdWarps, bwd_ctas(G, NT, F32))
w4_bwd_kernel(W4Params p, W4BwdPlan plan) {
  constexpr int CG = kBwdCols / G;               // groups of the CTA's columns
  extern __shared__ __align__(16) unsigned char shared[];   // the stages, the other operand and its third numbers, the zero points; then the warps' sums
  uint2(*const other)[NT][kQuads][8] = reinterpret_cast<uint2(*)[NT][kQuads][8]>(shared + kBwdStages * kBwdStage);   // [CG]
  uint2(*const third)[NT][kQuads][4] = reinterpret_cast<uint2(*)[NT][kQuads][4]>(other + CG);                        // [CG] for dy in fp32
  uint2(*const zeros)[kQuads] = reinterpret_cast<uint2(*)[kQuads]>(third + (F32 ? CG : 0));
  // the join kernel may be scheduled once every CTA has started; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int cw = warp % kBwdColWarps, rw = warp / kBwdColWarps;
  const int D = static_cast<int>(p.D), M = static_cast<int>(p.M), row_groups = D / G;
  const int cta0 = blockIdx.x * kBwdCols, m0 = blockIdx.z * (4 * NT);
  const int64_t f_lo = blockIdx.y * plan.rows, f_hi = min(f_lo + plan.rows, p.F);
  const int64_t stride = D / 2;

  // The weights on their way, a chunk to a stage.  Rows past the last read the last, whose scales count as 0 in the other operand;
  // columns past the last read the last sixteen bytes, and are not stored.
  constexpr int kParts = kBwdCols / 32, kRowsAtOnce = 32 * kBwdWarps / kParts;
  const uint32_t ring = smem_u32(shared);
  const int own_part = threadIdx.x % kParts, part_row = threadIdx.x / kParts;
  const uint32_t part_to = ring + part_row * (kBwdCols / 2) + 16 * (own_part ^ (part_row & 2));
  const uint8_t* part_from = p.data + (f_lo + part_row) * stride + min(cta0 + 32 * own_part, D - 32) / 2;   // of the next chunk
  auto issue = [&](int64_t f, int stage) {
    if (f < f_hi && f + kBwdRows <= p.F) {
#pragma unroll
      for (int k = 0; k < kBwdRows / kRowsAtOnce; ++k)
        cp_async_16(part_to + stage * kBwdStage + k * kRowsAtOnce * (kBwdCols / 2), part_from + k * kRowsAtOnce * stride, true);
    } else if (f < f_hi) {
#pragma unroll
      for (int k = 0; k < kBwdRows / kRowsAtOnce; ++k)
        cp_async_16(part_to + stage * kBwdStage + k * kRowsAtOnce * (kBwdCols / 2),
                    part_from + (min(f + part_row + k * kRowsAtOnce, p.F - 1) - f - part_row) * stride, true);
    }
    part_from += kBwdRows * stride;
    cp_async_commit();                           // one group a chunk, so that the wait below counts chunks
  };

  // This thread's part of the other operand: four rows of every fourth vector, for all of the CTA's groups.
  const int own_v = threadIdx.x % 4, own_quad = threadIdx.x / 4;
  const int own_row = own_quad / 4 * 16 + own_quad % 4;   // and the fourth, eighth and twelfth after it
  const bool whole = D % kBwdCols == 0;          // the CTA's groups of a row are one aligned load
  const int groups = min(CG, row_groups - cta0 / G);   // of the CTA's, those that there are
  // scales are two chunks ahead of their use, zero points and dy one
  using Scales = Pack<2 * CG>;
  const uint32_t scale_step = 4 * row_groups;    // elements between the four rows
  const bf16* scale_from = p.scale + (f_lo + own_row) * row_groups + cta0 / G;
  auto load_scales = [&](int64_t f, Scales (&to)[4]) {
    if (whole && f < f_hi && f + kBwdRows <= p.F) {
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = __ldcs(reinterpret_cast<const typename Scales::type*>(scale_from + i * scale_step));
    } else {
      const int64_t left = f < f_hi ? p.F - f - own_row : 0;   // rows to the end
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        to[i] = Scales{};
        if (4 * i < left)
#pragma unroll
          for (int q = 0; q < CG; ++q)
            if (q < groups) to[i].set(q, reinterpret_cast<const uint16_t*>(scale_from + i * scale_step)[q]);
      }
    }
    scale_from += kBwdRows * static_cast<int64_t>(row_groups);
  };
  const uint8_t* zero_from = ZERO ? p.zero + (f_lo + own_row) * row_groups + cta0 / G + min(own_v, groups - 1) : nullptr;
  uint32_t zero = 0;                             // of four rows, a byte each: group own_v
  float dys[NT][4];
  const int64_t dy_at = (m0 + own_v) * p.F + own_row;
  const int vectors = (M - m0 - own_v + 3) / 4;  // of this thread's, those that there are
  auto load_dy = [&](int64_t f) {
    const int64_t rest = p.F - f - own_row;
    const int left = rest < 16 ? static_cast<int>(rest) : 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int64_t at = dy_at + f + 4 * n * p.F;
      const float* const d32 = static_cast<const float*>(p.dy) + at;
      const bf16* const d16 = static_cast<const bf16*>(p.dy) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) dys[n][i] = 0.f;
      if (n >= vectors) continue;
      if constexpr (F32) {
        if (left == 16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) dys[n][i] = __ldg(d32 + 4 * i);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * i < left) dys[n][i] = __ldg(d32 + 4 * i);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * i < left) dys[n][i] = __bfloat162float(d16[4 * i]);
      }
    }
    if (ZERO) {
      zero = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * i < left) zero |= (zero_from[i * scale_step] & 15u) << (8 * i);
      zero_from += kBwdRows * static_cast<int64_t>(row_groups);
    }
  };

  float acc[NT][4][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][j][i] = 0.f;

#pragma unroll
  for (int s = 0; s < kBwdStages - 1; ++s) issue(f_lo + s * kBwdRows, s);
  Scales scales[4], scales1[4];
  load_scales(f_lo, scales);
  load_scales(f_lo + kBwdRows, scales1);
  load_dy(f_lo);
  int stage = 0;
  for (int64_t f = f_lo; f < f_hi; f += kBwdRows) {
    cp_async_wait<kBwdStages - 2>();
    if (f > f_lo) __syncthreads();               // every warp is done with the last chunk and its operand
#pragma unroll
    for (int q = 0; q < CG; ++q)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = dys[n][i] * __uint_as_float(scales[i].get(q) << 16);
        uint32_t parts[F32 ? 6 : 4];
        split4<F32 ? 3 : 2>(b, parts);
        *reinterpret_cast<uint4*>(&other[q][n][own_quad][2 * own_v]) = make_uint4(parts[0], parts[1], parts[2], parts[3]);
        if constexpr (F32) third[q][n][own_quad][own_v] = make_uint2(parts[4], parts[5]);
      }
    if (ZERO && own_v < CG)
      zeros[own_v][own_quad] = make_uint2(zero_of2(zero), zero_of2(zero >> 16));
    __syncthreads();
    issue(f + (kBwdStages - 1) * kBwdRows, stage ? stage - 1 : kBwdStages - 1);   // where the last chunk was
#pragma unroll
    for (int i = 0; i < 4; ++i) scales[i] = scales1[i];
    load_scales(f + 2 * kBwdRows, scales1);
    if (f + kBwdRows < f_hi) load_dy(f + kBwdRows);
    // groups of 64 and 128: the lane's word is columns 8 g ..; of 32: two bytes each of columns 4 g .. and 32 + 4 g ..
    const uint32_t mine = ring + stage * kBwdStage + (rw * (16 * kBwdSteps) + t) * (kBwdCols / 2) + (cw * 32 ^ (t & 2) * 16) + (G < 64 ? 2 : 4) * g;
    stage = stage + 1 < kBwdStages ? stage + 1 : 0;
#pragma unroll 2                                   // unrolled whole, the registers leave two CTAs on an SM instead of three
    for (int s = 0; s < kBwdSteps; ++s) {
      const int quad = (rw * kBwdSteps + s) * 4 + t;
      uint32_t now[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = mine + (16 * s + 4 * i) * (kBwdCols / 2);
        if constexpr (G < 64) now[i] = read_bytes2(at) | read_bytes2(at + 16) << 16;
        else read_words<1>(at, &now[i]);
      }
#pragma unroll
      for (int q = 0; q < (G < 64 ? 2 : 1); ++q) {
        const int group = G < 64 ? cw * 2 + q : cw * 64 / G;
        __nv_bfloat162 z01 = zero_pair(8), z23 = z01;
        if constexpr (ZERO) {
          const uint2 z = zeros[group][quad];
          z01 = *reinterpret_cast<const __nv_bfloat162*>(&z.x);
          z23 = *reinterpret_cast<const __nv_bfloat162*>(&z.y);
        }
        uint2 b[NT], b3[F32 ? NT : 1];           // the third numbers are in the columns of the rests, the odd ones
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n] = other[group][n][quad][g];
          if constexpr (F32) b3[n] = g & 1 ? third[group][n][quad][g / 2] : make_uint2(0, 0);
        }
#pragma unroll
        for (int j = G < 64 ? 2 * q : 0; j < (G < 64 ? 2 * q + 2 : 4); ++j) {
          const uint32_t pick = j * 0x0011u + (4 + j) * 0x1100u;   // byte j of either row
          const uint32_t p01 = __byte_perm(now[0], now[1], pick), p23 = __byte_perm(now[2], now[3], pick);
          const uint32_t frag[4] = {unpack_pair<false>(p01, z01), unpack_pair<true>(p01, z01), unpack_pair<false>(p23, z23), unpack_pair<true>(p23, z23)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16_16816(acc[n][j], frag, b[n].x, b[n].y);
            if constexpr (F32) mma_bf16_16816(acc[n][j], frag, b3[n].x, b3[n].y);
          }
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // sums i = 0, 1 are product j's first column, 2, 3 its second; tile columns 2 t, 2 t + 1: value and rests of vector t
  float(*const red)[4 * NT][kBwdCols] = reinterpret_cast<float(*)[4 * NT][kBwdCols]>(shared);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = cw * 64 + (G < 64 ? j / 2 * 32 + 4 * g + j % 2 * 2 : 8 * g + 2 * j);
      *reinterpret_cast<float2*>(&red[rw][n * 4 + t][col]) = make_float2(acc[n][j][0] + acc[n][j][1], acc[n][j][2] + acc[n][j][3]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * NT * kBwdCols; i += 32 * kBwdWarps) {
    const int v = i / kBwdCols, col = cta0 + i % kBwdCols;
    if (m0 + v >= M || col >= D) continue;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kBwdRowWarps; ++r) s += red[r][v][i % kBwdCols];
    s *= kUnit;
    const int64_t at = static_cast<int64_t>(m0 + v) * D + col;
    if (plan.splits == 1) p.dx[at] = __float2bfloat16(s);
    else p.partial[blockIdx.y * (p.M * p.D) + at] = s;
  }
}
// A CTA takes 32 numbers, a warp every eighth run; the eight sums are added in order.
__global__ void __launch_bounds__(256)
w4_join_kernel(W4Params p, int64_t splits) {
  __shared__ float red[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane, n = p.M * p.D;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float s = 0.f;
  if (i < n)
#pragma unroll 4
    for (int64_t k = warp; k < splits; k += 8) s += p.partial[k * n + i];
  red[warp][lane] = s;
  __syncthreads();
  if (warp || i >= n) return;
  for (int w = 1; w < 8; ++w) s += red[w][lane];
  p.dx[i] = __float2bfloat16(s);
}

// ---------------------------------------------------------------- from bf16
// G / 8 lanes hold a group, eight weights each.  Without zero points the scale is max |w| / 7, else the range of the
// group and 0 in 15 steps, both rounded to bf16; values are rounded to the nearest step (ties to even).  Once per model: 294,912 x 2048
// in 568 to 635 us (2.7 to 2.4 TB/s), 12,288 x 2048 in 27 to 29, not tuned further.
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
  // halves, which are exact, so that the range of finite weights is finite
  const bf16 scale = __float2bfloat16(p.zero ? (0.5f * hi - 0.5f * lo) / 7.5f : fmaxf(-lo, hi) / 7.f);
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

template <int G, int NT, int RS, bool ZERO>
cudaError_t fwd_zero(const W4Params& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.F + 16 * RS - 1) / (16 * RS)), static_cast<unsigned>((p.M + 8 * NT - 1) / (8 * NT)));
  constexpr int smem = fwd_smem<G, NT, RS>();
  constexpr auto kernel = w4_fwd_kernel<G, NT, RS, ZERO>;
  const cudaError_t e = allow_shared<kernel>(smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * kFwdWarps, smem, stream>>>(p);
  return cudaGetLastError();
}
template <int G, int NT, int RS>
cudaError_t fwd_rows(const W4Params& p, cudaStream_t stream) {
  return p.zero ? fwd_zero<G, NT, RS, true>(p, stream) : fwd_zero<G, NT, RS, false>(p, stream);
}
// Rows of a CTA: 32 share their loads of the vectors (12,288 x 2048: 5.4 us against 5.8 with 16, eight vectors 5.6 against 6.8),
// and 16 where that would leave SMs without two CTAs.
template <int G, int NT>
cudaError_t fwd(const W4Params& p, cudaStream_t stream) {
  return p.F < 32 * 2 * 152 ? fwd_rows<G, NT, 1>(p, stream) : fwd_rows<G, NT, 2>(p, stream);
}
template <int G>
cudaError_t fwd_group(const W4Params& p, cudaStream_t stream) {
  return p.M <= 8 ? fwd<G, 1>(p, stream) : p.M <= 16 ? fwd<G, 2>(p, stream) : fwd<G, 4>(p, stream);
}
template <int G, int NT, bool ZERO, bool F32>
cudaError_t bwd_type(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  constexpr int smem = bwd_smem<G, NT, ZERO, F32>();
  const dim3 grid(static_cast<unsigned>(plan.col_blocks), static_cast<unsigned>(plan.splits), static_cast<unsigned>((p.M + 4 * NT - 1) / (4 * NT)));
  constexpr auto kernel = w4_bwd_kernel<G, NT, ZERO, F32>;
  const cudaError_t e = allow_shared<kernel>(smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, 32 * kBwdWarps, smem, stream>>>(p, plan);
  return cudaGetLastError();
}
template <int G, int NT, bool ZERO>
cudaError_t bwd_zero(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  return p.dy_f32 ? bwd_type<G, NT, ZERO, true>(p, plan, stream) : bwd_type<G, NT, ZERO, false>(p, plan, stream);
}
template <int G, int NT>
cudaError_t bwd(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  return p.zero ? bwd_zero<G, NT, true>(p, plan, stream) : bwd_zero<G, NT, false>(p, plan, stream);
}
template <int G>
cudaError_t bwd_group(const W4Params& p, const W4BwdPlan& plan, cudaStream_t stream) {
  return p.M <= 4 ? bwd<G, 1>(p, plan, stream) : bwd<G, 2>(p, plan, stream);   // more than eight vectors: eight at a time
}

}  // namespace

size_t w4_bwd_workspace(int64_t M, int64_t D, int64_t F, int group, bool dy_f32) {
  return static_cast<size_t>(w4_bwd_plan(M, D, F, group, dy_f32).splits * M * D) * sizeof(float);
}

cudaError_t launch_w4_fwd(const W4Params& p, cudaStream_t stream) {
  ProfScope prof("w4_linear_fwd", stream);
  return p.group == 32 ? fwd_group<32>(p, stream) : p.group == 64 ? fwd_group<64>(p, stream) : fwd_group<128>(p, stream);
}

cudaError_t launch_w4_bwd(const W4Params& p, cudaStream_t stream) {
  const W4BwdPlan plan = w4_bwd_plan(p.M, p.D, p.F, p.group, p.dy_f32);
  {
    ProfScope prof("w4_linear_bwd", stream);
    const cudaError_t e = p.group == 32 ? bwd_group<32>(p, plan, stream) : p.group == 64 ? bwd_group<64>(p, plan, stream)
                                                                                         : bwd_group<128>(p, plan, stream);
    if (e != cudaSuccess) return e;
  }
  if (plan.splits == 1) return cudaSuccess;
  ProfScope prof("w4_join", stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.M * p.D + 31) / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4_join_kernel, p, plan.splits);
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
