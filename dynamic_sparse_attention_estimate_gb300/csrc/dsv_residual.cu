// A branch's way back into the residual stream of a DiT block, and the norm in front of the next branch:
//   r = x + alpha gate[b] post(z),   y = pre(r) (1 + scale[b]) + shift[b],   and the gradients (include/dsv.h).
//
// A row of D features belongs to W warps, eight features (16 bytes of bf16) to a lane and vector; the row stays in
// registers from its loads to its stores, so HBM sees each tensor once: 8 bytes a feature forward and 12 backward
// with a bf16 stream, 12 and 18 with an fp32 one, against some 16 and 40 operations: HBM bounds both directions.
// The sums of a row are shuffles and, for several warps, a barrier of the row's warps alone.
// Everything is fp32 from the loads on, with one rounding at each output.  The norm behind r reads r before its
// rounding to the stream's type.
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

// The residual stream's eight features as they are loaded, bf16 or fp32.
template <bool F32>
struct Raw;
template <>
struct Raw<false> {
  uint4 a;
  DSV_DEVICE void zero() { a = make_uint4(0, 0, 0, 0); }
  DSV_DEVICE void load(const void* p, int64_t vec) { a = static_cast<const uint4*>(p)[vec]; }
  DSV_DEVICE Vec8 get() const { return unpack8(a); }
  static DSV_DEVICE void store(void* p, int64_t vec, const float (&v)[8]) { static_cast<uint4*>(p)[vec] = pack8(v); }
};
template <>
struct Raw<true> {
  float4 a, b;
  DSV_DEVICE void zero() { a = b = make_float4(0, 0, 0, 0); }
  DSV_DEVICE void load(const void* p, int64_t vec) {
    a = static_cast<const float4*>(p)[2 * vec];
    b = static_cast<const float4*>(p)[2 * vec + 1];
  }
  DSV_DEVICE Vec8 get() const { return Vec8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
  static DSV_DEVICE void store(void* p, int64_t vec, const float (&v)[8]) {
    static_cast<float4*>(p)[2 * vec] = make_float4(v[0], v[1], v[2], v[3]);
    static_cast<float4*>(p)[2 * vec + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// Eight entries of a bf16 vector, or of one that is not there.
DSV_DEVICE Vec8 vector8(const bf16* p, int vec, float absent) {
  if (p) return unpack8(__ldg(reinterpret_cast<const uint4*>(p) + vec));
  Vec8 o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = absent;
  return o;
}

// ---------------------------------------------------------------- sums over a row
// The W warps of a row; the rows of a CTA meet only their own warps (barrier 1 + group).
struct RowGroup {
  int W, group, warp, lane;   // warps to a row; this thread's row group, warp in it, lane
  float* red;                 // [2][kSums][W] of the group
  int turn;
  DSV_DEVICE void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory"); }
  // K sums over the row, the same bits in every thread.  Two buffers in turn: a thread writes one only after the
  // barrier of the sum in between, which every reader of its last use has passed.
  template <int K>
  DSV_DEVICE void sum(float (&s)[K]) {
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
    sync();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      float t = buf[i * kMaxWarps];
      for (int w = 1; w < W; ++w) t += buf[i * kMaxWarps + w];
      s[i] = t;
    }
  }
  static constexpr int kSums = 3, kMaxWarps = 16;
};
constexpr int kRedFloats = 2 * RowGroup::kSums * RowGroup::kMaxWarps;   // of a row group

// How D is laid over lanes: vectors of eight features, V to a lane, W warps to a row, G rows at a time in a CTA.
struct RowPlan {
  int nvec, V, W, G;
};
// One vector a lane where 512 threads hold the row, else two (D <= 8192); rows of few warps share a CTA of up to
// `warps` warps.
RowPlan row_plan(int64_t D, int warps) {
  RowPlan r;
  r.nvec = static_cast<int>(D / 8);
  r.V = r.nvec > 512 ? 2 : 1;
  r.W = (r.nvec + 32 * r.V - 1) / (32 * r.V);
  r.G = r.W >= warps ? 1 : warps / r.W;
  if (r.G > 15) r.G = 15;   // barriers 1 .. 15
  return r;
}

// ---------------------------------------------------------------- forward
template <bool F32, int V, bool POST, int PRE>
__global__ void __launch_bounds__(512)
residual_norm_fwd_kernel(ResidualParams p, RowPlan plan) {
  __shared__ float red[15 * kRedFloats];
  const int warp = threadIdx.x >> 5;
  RowGroup rg{plan.W, warp / plan.W, warp % plan.W, static_cast<int>(threadIdx.x & 31), nullptr, 0};
  rg.red = red + rg.group * kRedFloats;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * plan.G + rg.group;
  if (row >= p.B * p.N) return;   // the row's warps leave together
  const int64_t b = row / p.N, base = row * plan.nvec;
  const float inv_d = 1.f / static_cast<float>(p.D);

  int vec[V];
  bool valid[V];
  Raw<F32> xr[V];
  uint4 zr[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    vec[i] = (rg.warp * V + i) * 32 + rg.lane;
    valid[i] = vec[i] < plan.nvec;
    xr[i].zero();
    zr[i] = make_uint4(0, 0, 0, 0);
    if (valid[i]) {
      xr[i].load(p.x, base + vec[i]);
      zr[i] = reinterpret_cast<const uint4*>(p.z)[base + vec[i]];
    }
  }
  float rz = 1.f;
  if (POST) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Vec8 z = unpack8(zr[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += z.v[j] * z.v[j];
    }
    rg.sum(s);
    rz = __frsqrt_rn(s[0] * inv_d + p.eps);
  }
  Vec8 r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r[i] = xr[i].get();
    if (!valid[i]) continue;
    const Vec8 z = unpack8(zr[i]), g = vector8(p.gate ? p.gate + b * p.gate_stride : nullptr, vec[i], 1.f);
    const Vec8 w = vector8(POST ? p.w_post : nullptr, vec[i], 1.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t = z.v[j];
      if (POST) t = t * rz * w.v[j];
      r[i].v[j] += p.alpha * g.v[j] * t;
    }
    Raw<F32>::store(p.r, base + vec[i], r[i].v);
  }
  if (PRE == kNormNone) return;
  float mean = 0.f;
  if (PRE == kNormLayer) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += r[i].v[j];
    rg.sum(s);
    mean = s[0] / static_cast<float>(p.D);   // divided, so that a constant row's deviations are 0
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (valid[i])
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i].v[j] -= mean;
        s[0] += r[i].v[j] * r[i].v[j];
      }
  rg.sum(s);
  const float rstd = __frsqrt_rn(s[0] * inv_d + p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!valid[i]) continue;
    const Vec8 sc = vector8(p.scale ? p.scale + b * p.scale_stride : nullptr, vec[i], 0.f);
    const Vec8 sh = vector8(p.shift ? p.shift + b * p.shift_stride : nullptr, vec[i], 0.f);
    const Vec8 w = vector8(p.w_pre, vec[i], 1.f);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = r[i].v[j] * rstd * (w.v[j] * (1.f + sc.v[j])) + sh.v[j];
    reinterpret_cast<uint4*>(p.y)[base + vec[i]] = pack8(y);
  }
}

// ---------------------------------------------------------------- backward
// With h = dy f, f = w_pre (1 + scale):  g = dr + rstd (h - mean h - xhat mean(h xhat)) is dx (rms: no mean h), and
// with u = alpha gate w_post g:  dz = rz (u - zhat mean(u zhat)) (no norm: dz = u).  A CTA walks the rows of one slab of a
// sample; a thread keeps the column sums  S = sum g zhat,  T = sum dy xhat,  U = sum dy  of its features, from which
// every vector's gradient follows.  The CTA's sums, its row groups added in order, are one partial row.
constexpr int kBwdWarps = 16;           // of a CTA
constexpr int64_t kBwdCtas = 152;       // slabs of rows over all samples
struct BwdPlan {
  RowPlan row;
  int64_t slabs, rows;                  // slabs of a sample, rows of a slab
};
BwdPlan bwd_plan(int64_t B, int64_t N, int64_t D) {
  BwdPlan q;
  q.row = row_plan(D, kBwdWarps);
  q.slabs = (kBwdCtas + B - 1) / B;
  const int64_t most = (N + q.row.G - 1) / q.row.G;   // a row for each group of a CTA
  if (q.slabs > most) q.slabs = most;
  q.rows = (N + q.slabs - 1) / q.slabs;
  q.slabs = (N + q.rows - 1) / q.rows;
  return q;
}
int sums_of(int pre) { return pre == kNormNone ? 1 : 3; }

template <bool F32, int V, bool POST, int PRE>
__global__ void __launch_bounds__(512)
residual_norm_bwd_kernel(ResidualParams p, BwdPlan plan) {
  extern __shared__ float cols[];       // [K][D]
  __shared__ float red[15 * kRedFloats];
  constexpr int K = PRE == kNormNone ? 1 : 3;
  const int warp = threadIdx.x >> 5, nvec = plan.row.nvec;
  RowGroup rg{plan.row.W, warp / plan.row.W, warp % plan.row.W, static_cast<int>(threadIdx.x & 31), nullptr, 0};
  rg.red = red + rg.group * kRedFloats;
  const int64_t b = blockIdx.x / plan.slabs, slab = blockIdx.x % plan.slabs;
  const int64_t n0 = slab * plan.rows, n1 = n0 + plan.rows < p.N ? n0 + plan.rows : p.N;
  const float inv_d = 1.f / static_cast<float>(p.D);

  int vec[V];
  bool valid[V];
  Vec8 c[V], f[V];                      // alpha gate w_post, w_pre (1 + scale)
  float acc[K][V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    vec[i] = (rg.warp * V + i) * 32 + rg.lane;
    valid[i] = vec[i] < nvec;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[i].v[j] = f[i].v[j] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) acc[k][i][j] = 0.f;
    }
    if (!valid[i]) continue;
    const Vec8 g = vector8(p.gate ? p.gate + b * p.gate_stride : nullptr, vec[i], 1.f);
    const Vec8 wz = vector8(POST ? p.w_post : nullptr, vec[i], 1.f), wr = vector8(p.w_pre, vec[i], 1.f);
    const Vec8 sc = vector8(p.scale ? p.scale + b * p.scale_stride : nullptr, vec[i], 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[i].v[j] = p.alpha * g.v[j] * wz.v[j];
      f[i].v[j] = wr.v[j] * (1.f + sc.v[j]);
    }
  }

  for (int64_t n = n0 + rg.group; n < n1; n += plan.row.G) {
    const int64_t base = (b * p.N + n) * nvec;
    Raw<F32> rr[V], gr[V];
    uint4 zr[V], yr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      rr[i].zero();
      gr[i].zero();
      zr[i] = yr[i] = make_uint4(0, 0, 0, 0);
      if (!valid[i]) continue;
      if (PRE != kNormNone) {
        rr[i].load(p.r, base + vec[i]);
        yr[i] = reinterpret_cast<const uint4*>(p.dy)[base + vec[i]];
      }
      zr[i] = reinterpret_cast<const uint4*>(p.z)[base + vec[i]];
      if (p.dr) gr[i].load(p.dr, base + vec[i]);
    }
    float s1[3] = {0.f, 0.f, 0.f};      // sum z^2, sum r, sum h
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const Vec8 z = unpack8(zr[i]), r = rr[i].get(), dy = unpack8(yr[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (POST) s1[0] += z.v[j] * z.v[j];
        s1[1] += r.v[j];
        s1[2] += dy.v[j] * f[i].v[j];
      }
    }
    if (POST || PRE == kNormLayer) rg.sum(s1);
    const float rz = POST ? __frsqrt_rn(s1[0] * inv_d + p.eps) : 1.f;
    const float mean = PRE == kNormLayer ? s1[1] / static_cast<float>(p.D) : 0.f, mh = PRE == kNormLayer ? s1[2] * inv_d : 0.f;
    float rstd = 0.f, mhx = 0.f;
    if (PRE != kNormNone) {
      float s2[2] = {0.f, 0.f};         // sum (r - mean)^2, sum h (r - mean)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!valid[i]) continue;
        const Vec8 r = rr[i].get(), dy = unpack8(yr[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = r.v[j] - mean;
          s2[0] += d * d;
          s2[1] += dy.v[j] * f[i].v[j] * d;
        }
      }
      rg.sum(s2);
      rstd = __frsqrt_rn(s2[0] * inv_d + p.eps);
      mhx = rstd * s2[1] * inv_d;
    }
    float s3[1] = {0.f};                // sum u z
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!valid[i]) continue;
      const Vec8 r = rr[i].get(), dy = unpack8(yr[i]), z = unpack8(zr[i]);
      Vec8 g = gr[i].get();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (PRE != kNormNone) {
          const float xh = (r.v[j] - mean) * rstd;
          g.v[j] += rstd * (dy.v[j] * f[i].v[j] - mh - xh * mhx);
          acc[K - 2][i][j] += dy.v[j] * xh;
          acc[K - 1][i][j] += dy.v[j];
        }
        acc[0][i][j] += g.v[j] * (z.v[j] * rz);
        if (POST) s3[0] += c[i].v[j] * g.v[j] * z.v[j];
      }
      Raw<F32>::store(p.dx, base + vec[i], g.v);
      if (!POST) {
        float dz[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) dz[j] = c[i].v[j] * g.v[j];
        reinterpret_cast<uint4*>(p.dz)[base + vec[i]] = pack8(dz);
      } else {                          // u, in fp32 until its row's sum is known
        // kept through a second walk below
      }
    }
    if (POST) {
      rg.sum(s3);
      const float mu = rz * s3[0] * inv_d;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!valid[i]) continue;
        const Vec8 r = rr[i].get(), dy = unpack8(yr[i]), z = unpack8(zr[i]);
        Vec8 g = gr[i].get();
        float dz[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (PRE != kNormNone) {
            const float xh = (r.v[j] - mean) * rstd;
            g.v[j] += rstd * (dy.v[j] * f[i].v[j] - mh - xh * mhx);
          }
          dz[j] = rz * (c[i].v[j] * g.v[j] - z.v[j] * rz * mu);
        }
        reinterpret_cast<uint4*>(p.dz)[base + vec[i]] = pack8(dz);
      }
    }
  }

  // the row groups' sums, added in the groups' order
  for (int g = 0; g < plan.row.G; ++g) {
    if (rg.group == g)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (valid[i])
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float* at = cols + k * p.D + 8 * vec[i] + j;
              *at = g ? *at + acc[k][i][j] : acc[k][i][j];
            }
    __syncthreads();
  }
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
  const int64_t ctas = (p.B * p.N + plan.G - 1) / plan.G;
  ProfScope prof("residual_norm_fwd", stream);
  residual_norm_fwd_kernel<F32, V, POST, PRE><<<static_cast<unsigned>(ctas), 32 * plan.W * plan.G, 0, stream>>>(p, plan);
  return cudaGetLastError();
}
template <bool F32, int V, bool POST, int PRE>
cudaError_t bwd(const ResidualParams& p, const BwdPlan& plan, cudaStream_t stream) {
  const int K = sums_of(PRE);
  const size_t smem = static_cast<size_t>(K) * p.D * sizeof(float);
  auto kernel = residual_norm_bwd_kernel<F32, V, POST, PRE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  {
    ProfScope prof("residual_norm_bwd", stream);
    kernel<<<static_cast<unsigned>(p.B * plan.slabs), 32 * plan.row.W * plan.row.G, smem, stream>>>(p, plan);
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
  const BwdPlan q = bwd_plan(B, N, D);
  return static_cast<size_t>(B * q.slabs * sums_of(pre) + 2 * B) * D * sizeof(float);
}

cudaError_t launch_residual_norm_fwd(const ResidualParams& p, cudaStream_t stream) {
  const RowPlan plan = row_plan(p.D, 4);
  return DSV_RESIDUAL_PICK(fwd, plan.V, p, plan, stream);
}
cudaError_t launch_residual_norm_bwd(const ResidualParams& p, cudaStream_t stream) {
  const BwdPlan plan = bwd_plan(p.B, p.N, p.D);
  return DSV_RESIDUAL_PICK(bwd, plan.row.V, p, plan, stream);
}

}  // namespace dsv
