// A branch's way back into the residual stream of a DiT block, and the norm in front of the next branch:
//   r = x + alpha gate[b] post(z),   y = pre(r) (1 + scale[b]) + shift[b],   and the gradients (include/dsv.h).
//
// HBM sees each tensor once: 8 bytes a feature forward and 12 backward with a bf16 stream, 12 and 18 with an fp32 one,
// against some 16 and 40 operations, so HBM bounds both directions, and what counts is bytes in flight: a row's sums have
// to be known before it can be stored, so a row that is loaded, summed and stored in turn leaves the memory idle meanwhile.
// Therefore CTAs stay: each walks the rows of one slab of a sample, keeps the sample's vectors in registers, and has the next rows
// on their way into shared memory (cp.async; a thread reads back only what it copied itself, so a row needs no barrier
// but those of its sums).  A row belongs to W warps, eight features (16 bytes of bf16) to a lane and vector; G rows at a time
// belong to a CTA.  Everything is fp32 from the loads on, with one rounding at each output.  The norm behind r
// reads r before its rounding to the stream's type.
#include "dsv_block.h"
#include "dsv_common.cuh"

namespace dsv {
namespace {

// ---------------------------------------------------------------- eight features of a row
struct Vec8 {
  float v[8];
};
DSV_DEVICE Vec8 unpack8(const uint4& a) {
  Vec8 o;
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o.v[2 * j] = bf16_lo(w[j]);
    o.v[2 * j + 1] = bf16_hi(w[j]);
  }
  return o;
}
DSV_DEVICE uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// Eight entries of a bf16 vector, or of one that is not there.
DSV_DEVICE Vec8 vector8(const bf16* p, int vec, float absent) {
  if (p) return unpack8(__ldg(reinterpret_cast<const uint4*>(p) + vec));
  Vec8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = absent;
  return o;
}

// Eight features of the residual stream, bf16 or fp32, in 16-byte parts.
template <bool F32>
struct Stream {
  static constexpr int kParts = F32 ? 2 : 1;
  static DSV_DEVICE Vec8 get(const uint4 (&a)[kParts]) {
    if constexpr (F32) {
      return Vec8{{__uint_as_float(a[0].x), __uint_as_float(a[0].y), __uint_as_float(a[0].z), __uint_as_float(a[0].w),
                   __uint_as_float(a[1].x), __uint_as_float(a[1].y), __uint_as_float(a[1].z), __uint_as_float(a[1].w)}};
    } else {
      return unpack8(a[0]);
    }
  }
  static DSV_DEVICE void store(void* p, int64_t vec, const float (&v)[8]) {
    if constexpr (F32) {
      static_cast<float4*>(p)[2 * vec] = make_float4(v[0], v[1], v[2], v[3]);
      static_cast<float4*>(p)[2 * vec + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      static_cast<uint4*>(p)[vec] = pack8(v);
    }
  }
};

// ---------------------------------------------------------------- how the work is laid out
constexpr int kMaxWarps = 16;           // of a row and of a CTA
struct RowPlan {
  int nvec, V, W, G;                    // vectors of eight features, V to a lane, W warps to a row, G rows at a time
  int64_t slabs, rows;                  // slabs of a sample (one CTA each), rows of a slab
};
// One vector a lane where 512 threads hold the row, else two (D <= 8192).  About `ctas` slabs over all samples, but no more
// than give each group of a CTA a row.
RowPlan row_plan(int64_t B, int64_t N, int64_t D, int64_t ctas) {
  RowPlan q;
  q.nvec = static_cast<int>(D / 8);
  q.V = q.nvec > 32 * kMaxWarps ? 2 : 1;
  q.W = (q.nvec + 32 * q.V - 1) / (32 * q.V);
  q.G = kMaxWarps / q.W;
  if (q.G > 15) q.G = 15;               // named barriers 1 .. 15
  q.slabs = (ctas + B - 1) / B;
  const int64_t most = (N + q.G - 1) / q.G;
  if (q.slabs > most) q.slabs = most;
  q.rows = (N + q.slabs - 1) / q.slabs;
  q.slabs = (N + q.rows - 1) / q.rows;
  return q;
}

// This thread's place: its row group, its warp and lane in it, its vectors, its CTA's rows.
template <int V>
struct Place {
  int group, warp, lane, vec[V];
  bool valid[V];
  int64_t b, n0, n1;
  DSV_DEVICE Place(const RowPlan& plan, int64_t N) {
    const int w = threadIdx.x >> 5;
    group = w / plan.W;
    warp = w % plan.W;
    lane = threadIdx.x & 31;
    b = blockIdx.x / plan.slabs;
    n0 = blockIdx.x % plan.slabs * plan.rows;
    n1 = n0 + plan.rows < N ? n0 + plan.rows : N;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      vec[i] = (warp * V + i) * 32 + lane;
      valid[i] = vec[i] < plan.nvec;
    }
  }
};

// Sums over a row.  The W warps of a row meet at a barrier of their own (1 + group).
constexpr int kSums = 3;
constexpr int kRedFloats = 2 * kSums * kMaxWarps;   // of a row group
struct RowSums {
  int W, group, warp, lane, turn;
  float* red;                           // [2][kSums][kMaxWarps] of the group, zero from W on
  // K sums over the row, the same bits in every thread.  Two buffers in turn: a thread writes one only after the
  // barrier of the sum in between, which every reader of its last use has passed.
  template <int K>
  DSV_DEVICE void operator()(float (&s)[K]) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < K; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if (W == 1) return;
    float* buf = red + turn * (kSums * kMaxWarps);
    turn ^= 1;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) buf[i * kMaxWarps + warp] = s[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory");
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float4* p = reinterpret_cast<const float4*>(buf + i * kMaxWarps);
      float4 t = p[0];
      s[i] = (t.x + t.y) + (t.z + t.w);
      for (int w = 4; w < W; w += 4) {
        t = p[w / 4];
        s[i] += (t.x + t.y) + (t.z + t.w);
      }
    }
  }
};
DSV_DEVICE RowSums row_sums(const RowPlan& plan, float* red, int group, int warp, int lane) {
  for (int i = threadIdx.x; i < 15 * kRedFloats; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
  return RowSums{plan.W, group, warp, lane, 0, red + group * kRedFloats};
}

// A thread's rows on their way: `S` stages of P 16-byte parts for each of its vectors in shared memory.
template <int P, int V, int S>
struct Ring {
  uint32_t base, stride;                // this thread's part 0 of stage 0; bytes between parts
  DSV_DEVICE Ring(void* smem) : base(smem_u32(smem) + 16 * threadIdx.x), stride(16 * blockDim.x) {}
  DSV_DEVICE uint32_t at(int stage, int i, int part) const { return base + ((stage * V + i) * P + part) * stride; }
  DSV_DEVICE void copy(int stage, int i, int part, const void* p, int64_t part16) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(at(stage, i, part)),
                 "l"(static_cast<const uint4*>(p) + part16)
                 : "memory");
  }
  DSV_DEVICE uint4 read(int stage, int i, int part) const {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at(stage, i, part)) : "memory");
    return v;
  }
  static size_t bytes(int threads) { return static_cast<size_t>(S) * V * P * 16 * threads; }
};

// ---------------------------------------------------------------- forward
constexpr int kFwdStages = 4;
constexpr int64_t kFwdCtas = 2 * 152;

template <bool F32, int V, bool POST, int PRE>
__global__ void __launch_bounds__(32 * kMaxWarps, V == 1 ? 2 : 1)
residual_norm_fwd_kernel(ResidualParams p, RowPlan plan) {
  extern __shared__ __align__(16) uint4 ring_mem[];
  __shared__ __align__(16) float red[15 * kRedFloats];
  using St = Stream<F32>;
  constexpr int P = St::kParts + 1, S = kFwdStages;
  const Place<V> at(plan, p.N);
  RowSums sum = row_sums(plan, red, at.group, at.warp, at.lane);
  const Ring<P, V, S> ring(ring_mem);
  const float D = static_cast<float>(p.D), inv_d = 1.f / D;

  auto issue = [&](int64_t n, int stage) {
    if (n < at.n1) {
      const int64_t base = (at.b * p.N + n) * plan.nvec;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.valid[i]) {
#pragma unroll
          for (int k = 0; k < St::kParts; ++k) ring.copy(stage, i, k, p.x, (base + at.vec[i]) * St::kParts + k);
          ring.copy(stage, i, St::kParts, p.z, base + at.vec[i]);
        }
    }
    cp_async_commit();                  // one group a row, so that the wait below counts rows
  };
  const int64_t first = at.n0 + at.group;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(first + s * plan.G, s);

  Vec8 c[V], f[V], sh[V];               // alpha gate w_post, w_pre (1 + scale), shift
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = at.valid[i] ? at.vec[i] : 0;
    const Vec8 g = vector8(p.gate ? p.gate + at.b * p.gate_stride : nullptr, vec, 1.f);
    const Vec8 wz = vector8(POST ? p.w_post : nullptr, vec, 1.f), wr = vector8(p.w_pre, vec, 1.f);
    const Vec8 sc = vector8(p.scale ? p.scale + at.b * p.scale_stride : nullptr, vec, 0.f);
    sh[i] = vector8(p.shift ? p.shift + at.b * p.shift_stride : nullptr, vec, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[i].v[j] = p.alpha * g.v[j] * wz.v[j];
      f[i].v[j] = wr.v[j] * (1.f + sc.v[j]);
    }
  }

  int stage = 0;
  for (int64_t n = first; n < at.n1; n += plan.G) {
    cp_async_wait<S - 2>();
    Vec8 r[V], z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (at.valid[i]) {
        uint4 x[St::kParts];
#pragma unroll
        for (int k = 0; k < St::kParts; ++k) x[k] = ring.read(stage, i, k);
        r[i] = St::get(x);
        z[i] = unpack8(ring.read(stage, i, St::kParts));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i].v[j] = z[i].v[j] = 0.f;
      }
    }
    issue(n + (S - 1) * plan.G, stage ? stage - 1 : S - 1);   // the stage that the last row was read from
    stage = stage + 1 < S ? stage + 1 : 0;
    const int64_t base = (at.b * p.N + n) * plan.nvec;

    float rz = 1.f;
    if constexpr (POST) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] += z[i].v[j] * z[i].v[j];
      sum(s);
      rz = __frsqrt_rn(s[0] * inv_d + p.eps);
    }
    float s[1] = {0.f};                 // of r (layer) or r^2 (rms)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!at.valid[i]) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i].v[j] += c[i].v[j] * (POST ? z[i].v[j] * rz : z[i].v[j]);
        s[0] += PRE == kNormLayer ? r[i].v[j] : r[i].v[j] * r[i].v[j];
      }
      St::store(p.r, base + at.vec[i], r[i].v);
    }
    if constexpr (PRE != kNormNone) {
      sum(s);
      if constexpr (PRE == kNormLayer) {
        const float mean = s[0] / D;    // divided, so that a constant row's deviations are 0
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (at.valid[i])
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              r[i].v[j] -= mean;
              s[0] += r[i].v[j] * r[i].v[j];
            }
        sum(s);
      }
      const float rstd = __frsqrt_rn(s[0] * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!at.valid[i]) continue;
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = r[i].v[j] * rstd * f[i].v[j] + sh[i].v[j];
        reinterpret_cast<uint4*>(p.y)[base + at.vec[i]] = pack8(y);
      }
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- backward
// With h = dy f, f = w_pre (1 + scale):  g = dr + rstd (h - mean h - xhat mean(h xhat)) is dx (rms: no mean h), and
// with u = alpha gate w_post g:  dz = rz (u - zhat mean(u zhat)) (no norm: dz = u).  A thread keeps the column sums
// S = sum g zhat,  T = sum dy xhat,  U = sum dy  of its features, from which every vector's gradient follows.  The CTA's
// sums, its row groups added in order, are one partial row.
constexpr int64_t kBwdCtas = 152;
int sums_of(int pre) { return pre == kNormNone ? 1 : 3; }
// Stages that fit beside each other: parts of 16 bytes a thread and vector, 512 threads.
template <int P, int V>
constexpr int bwd_stages() {
  return P * V <= 4 ? 4 : P * V <= 8 ? 3 : 2;
}

template <bool F32, int V, bool POST, int PRE>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
residual_norm_bwd_kernel(ResidualParams p, RowPlan plan) {
  extern __shared__ __align__(16) uint4 ring_mem[];
  __shared__ __align__(16) float red[15 * kRedFloats];
  using St = Stream<F32>;
  constexpr int SP = St::kParts, P = PRE == kNormNone ? SP + 1 : 2 * SP + 2, S = bwd_stages<P, V>();
  constexpr int K = PRE == kNormNone ? 1 : 3;
  constexpr int kDr = 0, kZ = SP, kDy = SP + 1, kR = SP + 2;    // parts of a vector
  const Place<V> at(plan, p.N);
  RowSums sum = row_sums(plan, red, at.group, at.warp, at.lane);
  const Ring<P, V, S> ring(ring_mem);
  const float D = static_cast<float>(p.D), inv_d = 1.f / D;

  auto issue = [&](int64_t n, int stage) {
    if (n < at.n1) {
      const int64_t base = (at.b * p.N + n) * plan.nvec;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.valid[i]) {
          const int64_t v = base + at.vec[i];
          if constexpr (PRE != kNormNone) {
#pragma unroll
            for (int k = 0; k < SP; ++k) ring.copy(stage, i, kR + k, p.r, v * SP + k);
            ring.copy(stage, i, kDy, p.dy, v);
          }
          ring.copy(stage, i, kZ, p.z, v);
          if (p.dr)
#pragma unroll
            for (int k = 0; k < SP; ++k) ring.copy(stage, i, kDr + k, p.dr, v * SP + k);
        }
    }
    cp_async_commit();
  };
  const int64_t first = at.n0 + at.group;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(first + s * plan.G, s);

  Vec8 c[V], f[V];                      // alpha gate w_post, w_pre (1 + scale)
  float acc[K][V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int vec = at.valid[i] ? at.vec[i] : 0;
    const Vec8 g = vector8(p.gate ? p.gate + at.b * p.gate_stride : nullptr, vec, 1.f);
    const Vec8 wz = vector8(POST ? p.w_post : nullptr, vec, 1.f), wr = vector8(p.w_pre, vec, 1.f);
    const Vec8 sc = vector8(p.scale ? p.scale + at.b * p.scale_stride : nullptr, vec, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[i].v[j] = p.alpha * g.v[j] * wz.v[j];
      f[i].v[j] = wr.v[j] * (1.f + sc.v[j]);
#pragma unroll
      for (int k = 0; k < K; ++k) acc[k][i][j] = 0.f;
    }
  }

  int stage = 0;
  for (int64_t n = first; n < at.n1; n += plan.G) {
    cp_async_wait<S - 2>();
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 rr[V][SP], gr[V][SP], zr[V], yr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = at.valid[i];
      zr[i] = in ? ring.read(stage, i, kZ) : none;
      yr[i] = PRE != kNormNone && in ? ring.read(stage, i, kDy) : none;
#pragma unroll
      for (int k = 0; k < SP; ++k) {
        rr[i][k] = PRE != kNormNone && in ? ring.read(stage, i, kR + k) : none;
        gr[i][k] = p.dr && in ? ring.read(stage, i, kDr + k) : none;
      }
    }
    issue(n + (S - 1) * plan.G, stage ? stage - 1 : S - 1);
    stage = stage + 1 < S ? stage + 1 : 0;
    const int64_t base = (at.b * p.N + n) * plan.nvec;

    float rz = 1.f, mean = 0.f, mh = 0.f, rstd = 0.f, mhx = 0.f;
    {
      float s[3] = {0.f, 0.f, 0.f};     // sum z^2; layer: sum r, sum h; rms: sum r^2, sum h r
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const Vec8 z = unpack8(zr[i]), r = St::get(rr[i]), dy = unpack8(yr[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (POST) s[0] += z.v[j] * z.v[j];
          const float h = dy.v[j] * f[i].v[j];
          s[1] += PRE == kNormLayer ? r.v[j] : r.v[j] * r.v[j];
          s[2] += PRE == kNormLayer ? h : h * r.v[j];
        }
      }
      if constexpr (POST && PRE == kNormNone) {
        float s1[1] = {s[0]};
        sum(s1);
        s[0] = s1[0];
      } else if constexpr (PRE != kNormNone && !POST) {
        float s2[2] = {s[1], s[2]};
        sum(s2);
        s[1] = s2[0];
        s[2] = s2[1];
      } else if constexpr (PRE != kNormNone) {
        sum(s);
      }
      if (POST) rz = __frsqrt_rn(s[0] * inv_d + p.eps);
      if (PRE == kNormLayer) {
        mean = s[1] / D;                // divided, so that a constant row's deviations are 0
        mh = s[2] * inv_d;
      }
      if (PRE == kNormRms) {
        rstd = __frsqrt_rn(s[1] * inv_d + p.eps);
        mhx = rstd * s[2] * inv_d;
      }
    }
    if constexpr (PRE == kNormLayer) {
      float s[2] = {0.f, 0.f};          // sum (r - mean)^2, sum h (r - mean)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!at.valid[i]) continue;
        const Vec8 r = St::get(rr[i]), dy = unpack8(yr[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = r.v[j] - mean;
          s[0] += d * d;
          s[1] += dy.v[j] * f[i].v[j] * d;
        }
      }
      sum(s);
      rstd = __frsqrt_rn(s[0] * inv_d + p.eps);
      mhx = rstd * s[1] * inv_d;
    }
    float s[1] = {0.f};                 // sum u z
    Vec8 u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!at.valid[i]) continue;
      const Vec8 r = St::get(rr[i]), dy = unpack8(yr[i]), z = unpack8(zr[i]);
      Vec8 g = St::get(gr[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (PRE != kNormNone) {
          const float xh = (r.v[j] - mean) * rstd;
          g.v[j] += rstd * (dy.v[j] * f[i].v[j] - mh - xh * mhx);
          acc[K - 2][i][j] += dy.v[j] * xh;
          acc[K - 1][i][j] += dy.v[j];
        }
        acc[0][i][j] += g.v[j] * (z.v[j] * rz);
        u[i].v[j] = c[i].v[j] * g.v[j];
        if (POST) s[0] += u[i].v[j] * z.v[j];
      }
      St::store(p.dx, base + at.vec[i], g.v);
    }
    float mu = 0.f;
    if constexpr (POST) {
      sum(s);
      mu = rz * s[0] * inv_d;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!at.valid[i]) continue;
      if (POST) {
        const Vec8 z = unpack8(zr[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i].v[j] = rz * (u[i].v[j] - z.v[j] * rz * mu);
      }
      reinterpret_cast<uint4*>(p.dz)[base + at.vec[i]] = pack8(u[i].v);
    }
  }

  // the row groups' sums, added in the groups' order, where the rows were
  cp_async_wait<0>();
  float* cols = reinterpret_cast<float*>(ring_mem);   // [K][D]
  for (int g = 0; g < plan.G; ++g) {
    __syncthreads();
    if (at.group == g)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (at.valid[i])
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float4* to = reinterpret_cast<float4*>(cols + k * p.D + 8 * at.vec[i]) + h;
              const float* a = &acc[k][i][4 * h];
              const float4 t = g ? *to : make_float4(0, 0, 0, 0);
              *to = make_float4(t.x + a[0], t.y + a[1], t.z + a[2], t.w + a[3]);
            }
  }
  __syncthreads();
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * K * p.D;
  for (int i = threadIdx.x; i < K * p.D; i += blockDim.x) out[i] = cols[i];
}

// The gradients of the vectors from the slabs' partial rows: a CTA takes 32 features of one sample, a warp every eighth
// slab; the eight sums are added in order.  With several samples the sums S and T stay behind the partial rows for the
// weights' gradients, which a last kernel adds over the samples.
__global__ void __launch_bounds__(256)
residual_vectors_kernel(ResidualParams p, int64_t slabs, int K, float* per_sample) {
  __shared__ float red[8][3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane, b = blockIdx.y;
  float s[3] = {0.f, 0.f, 0.f};
  if (d < p.D)
    for (int64_t t = warp; t < slabs; t += 8)
      for (int k = 0; k < K; ++k) s[k] += p.partial[((b * slabs + t) * K + k) * p.D + d];
  for (int k = 0; k < K; ++k) red[warp][k][lane] = s[k];
  __syncthreads();
  if (warp || d >= p.D) return;
  for (int k = 0; k < K; ++k) {
    s[k] = red[0][k][lane];
    for (int w = 1; w < 8; ++w) s[k] += red[w][k][lane];
  }
  const float wz = p.post == kNormRms && p.w_post ? __bfloat162float(p.w_post[d]) : 1.f;
  const float wr = p.w_pre ? __bfloat162float(p.w_pre[d]) : 1.f;
  if (p.d_gate) p.d_gate[b * p.d_stride + d] = p.alpha * wz * s[0];
  if (p.d_scale) p.d_scale[b * p.d_stride + d] = wr * s[1];
  if (p.d_shift) p.d_shift[b * p.d_stride + d] = s[2];
  const float gate = p.gate ? __bfloat162float(p.gate[b * p.gate_stride + d]) : 1.f;
  const float scale = p.scale ? __bfloat162float(p.scale[b * p.scale_stride + d]) : 0.f;
  const float post = p.alpha * gate * s[0], pre = (1.f + scale) * s[1];
  if (per_sample) {
    per_sample[(2 * b) * p.D + d] = post;
    per_sample[(2 * b + 1) * p.D + d] = pre;
  } else {
    if (p.dw_post) p.dw_post[d] = post;
    if (p.dw_pre) p.dw_pre[d] = pre;
  }
}
__global__ void __launch_bounds__(128)
residual_weights_kernel(ResidualParams p, const float* per_sample) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (d >= p.D) return;
  float post = 0.f, pre = 0.f;
  for (int64_t b = 0; b < p.B; ++b) {
    post += per_sample[(2 * b) * p.D + d];
    pre += per_sample[(2 * b + 1) * p.D + d];
  }
  if (p.dw_post) p.dw_post[d] = post;
  if (p.dw_pre) p.dw_pre[d] = pre;
}

template <bool F32, int V, bool POST, int PRE>
cudaError_t fwd(const ResidualParams& p, const RowPlan& plan, cudaStream_t stream) {
  auto kernel = residual_norm_fwd_kernel<F32, V, POST, PRE>;
  const int threads = 32 * plan.W * plan.G;
  const size_t smem = Ring<Stream<F32>::kParts + 1, V, kFwdStages>::bytes(threads);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  ProfScope prof("residual_norm_fwd", stream);
  kernel<<<static_cast<unsigned>(p.B * plan.slabs), threads, smem, stream>>>(p, plan);
  return cudaGetLastError();
}
template <bool F32, int V, bool POST, int PRE>
cudaError_t bwd(const ResidualParams& p, const RowPlan& plan, cudaStream_t stream) {
  const int K = sums_of(PRE), threads = 32 * plan.W * plan.G;
  constexpr int SP = Stream<F32>::kParts, P = PRE == kNormNone ? SP + 1 : 2 * SP + 2;
  const size_t cols = static_cast<size_t>(K) * p.D * sizeof(float), ring = Ring<P, V, bwd_stages<P, V>()>::bytes(threads);
  const size_t smem = cols > ring ? cols : ring;
  auto kernel = residual_norm_bwd_kernel<F32, V, POST, PRE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  {
    ProfScope prof("residual_norm_bwd", stream);
    kernel<<<static_cast<unsigned>(p.B * plan.slabs), threads, smem, stream>>>(p, plan);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const bool weights = p.dw_post || p.dw_pre;
  if (!p.d_gate && !p.d_scale && !p.d_shift && !weights) return cudaSuccess;
  float* per_sample = weights && p.B > 1 ? p.partial + p.B * plan.slabs * K * p.D : nullptr;
  {
    ProfScope prof("residual_vectors", stream);
    const dim3 grid(static_cast<unsigned>((p.D + 31) / 32), static_cast<unsigned>(p.B));
    residual_vectors_kernel<<<grid, 256, 0, stream>>>(p, plan.slabs, K, per_sample);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (!per_sample) return cudaSuccess;
  ProfScope prof("residual_weights", stream);
  residual_weights_kernel<<<static_cast<unsigned>((p.D + 127) / 128), 128, 0, stream>>>(p, per_sample);
  return cudaGetLastError();
}

// f<F32, V, POST, PRE>(args) for the call's stream type, row length and norms
#define DSV_RESIDUAL_PICK4(fn, F, V, P, ...)                                   \
  (p.pre == kNormNone ? fn<F, V, P, kNormNone>(__VA_ARGS__)                    \
                      : p.pre == kNormRms ? fn<F, V, P, kNormRms>(__VA_ARGS__) \
                                          : fn<F, V, P, kNormLayer>(__VA_ARGS__))
#define DSV_RESIDUAL_PICK3(fn, F, V, ...) \
  (p.post == kNormRms ? DSV_RESIDUAL_PICK4(fn, F, V, true, __VA_ARGS__) : DSV_RESIDUAL_PICK4(fn, F, V, false, __VA_ARGS__))
#define DSV_RESIDUAL_PICK2(fn, F, v, ...) \
  (v == 1 ? DSV_RESIDUAL_PICK3(fn, F, 1, __VA_ARGS__) : DSV_RESIDUAL_PICK3(fn, F, 2, __VA_ARGS__))
#define DSV_RESIDUAL_PICK(fn, v, ...) \
  (p.f32 ? DSV_RESIDUAL_PICK2(fn, true, v, __VA_ARGS__) : DSV_RESIDUAL_PICK2(fn, false, v, __VA_ARGS__))

}  // namespace

size_t residual_bwd_workspace(int64_t B, int64_t N, int64_t D, int pre) {
  const RowPlan q = row_plan(B, N, D, kBwdCtas);
  return static_cast<size_t>(B * q.slabs * sums_of(pre) + 2 * B) * D * sizeof(float);
}

cudaError_t launch_residual_norm_fwd(const ResidualParams& p, cudaStream_t stream) {
  const RowPlan plan = row_plan(p.B, p.N, p.D, kFwdCtas);
  return DSV_RESIDUAL_PICK(fwd, plan.V, p, plan, stream);
}
cudaError_t launch_residual_norm_bwd(const ResidualParams& p, cudaStream_t stream) {
  const RowPlan plan = row_plan(p.B, p.N, p.D, kBwdCtas);
  return DSV_RESIDUAL_PICK(bwd, plan.V, p, plan, stream);
}

}  // namespace dsv
