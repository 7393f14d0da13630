// A branch's way back into the residual stream of a DiT block, and the norm in front of the next branch:
//   r = x + alpha gate[b] post(z),   y = pre(r) (1 + scale[b]) + shift[b],   and the gradients (include/dsv.h).
//
// HBM sees each tensor once: 8 bytes a feature forward and 12 backward with a bf16 stream, 12 and 18 with an fp32 one,
// against some 16 and 40 operations, so HBM bounds both directions, and what counts is bytes in flight: a row's sums have
// to be known before it can be stored, so a row that is loaded, summed and stored in turn leaves the memory idle meanwhile.
// Therefore CTAs stay: each takes rows of one sample in turn, keeps the sample's vectors, and has the next rows on their way into
// shared memory (cp.async, into places that the reading warp alone uses, so that a row needs no barrier but those of its
// sums).  A row belongs to W warps, eight features to a lane and vector; G rows at a time belong to a CTA.
// Everything is fp32 from the loads on, with one rounding at each output.  The norm behind r reads r before its rounding to
// the stream's type.
//   Measured with the calls in a row: forward 520,192 x 2048, RMS norms, 1,325 us (6.4 TB/s, 0.97 of the copy rate), backward
// 65,536 x 2048, RMS and layer norm, 269 us (6.0 TB/s, 0.90); simple kernels, a row loaded, summed and stored in turn, 2,681 and 670.
#include "dsv_block.h"
#include "dsv_common.cuh"

namespace dsv {
namespace {

// ---------------------------------------------------------------- eight features of a row
// Elementwise work runs on pairs (fma.rn.f32x2 and its like: two IEEE operations to an instruction).
DSV_DEVICE uint64_t as_u64(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
DSV_DEVICE float2 as_f2(uint64_t v) { return *reinterpret_cast<float2*>(&v); }
DSV_DEVICE float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(d);
}
DSV_DEVICE float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
DSV_DEVICE float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(d);
}
DSV_DEVICE float2 both(float v) { return make_float2(v, v); }

struct Vec8 {
  float2 v[4];
};
DSV_DEVICE Vec8 all8(float v) { return Vec8{{both(v), both(v), both(v), both(v)}}; }
DSV_DEVICE Vec8 unpack8(const uint4& a) {
  return Vec8{{make_float2(bf16_lo(a.x), bf16_hi(a.x)), make_float2(bf16_lo(a.y), bf16_hi(a.y)),
               make_float2(bf16_lo(a.z), bf16_hi(a.z)), make_float2(bf16_lo(a.w), bf16_hi(a.w))}};
}
DSV_DEVICE uint4 pack8(const Vec8& a) {
  return make_uint4(pack_bf16x2(a.v[0].x, a.v[0].y), pack_bf16x2(a.v[1].x, a.v[1].y), pack_bf16x2(a.v[2].x, a.v[2].y),
                    pack_bf16x2(a.v[3].x, a.v[3].y));
}
// Eight features of the residual stream, bf16 or fp32, in 16-byte parts.
template <bool F32>
struct Stream {
  static constexpr int kParts = F32 ? 2 : 1;
  static DSV_DEVICE Vec8 get(const uint4 (&a)[kParts]) {
    if constexpr (F32) {
      return Vec8{{make_float2(__uint_as_float(a[0].x), __uint_as_float(a[0].y)), make_float2(__uint_as_float(a[0].z), __uint_as_float(a[0].w)),
                   make_float2(__uint_as_float(a[1].x), __uint_as_float(a[1].y)), make_float2(__uint_as_float(a[1].z), __uint_as_float(a[1].w))}};
    } else {
      return unpack8(a[0]);
    }
  }
};

// ---------------------------------------------------------------- how the work is laid out
constexpr int kMaxWarps = 16;           // of a row and of a CTA
constexpr int kMaxShared = 221 * 1024;  // dynamic shared memory of a CTA: what the sums over a row leave of 227 KB
struct RowPlan {
  int nvec, V, W, G;                    // vectors of eight features, V to a lane, W warps to a row, G rows at a time
  int warps;                            // that a CTA may have: its kernel's registers allow no more
  int64_t ctas;                         // of a sample: CTA c takes rows c G, .., c G + G - 1 of every ctas G
};
// Two vectors a lane where a row has more than 32: a row's sums, its scalars and its addresses cost a lane about as much as
// eight features do, so one vector a lane was half the rate (32,768 x 2048 backward, both norms: 268 us).  A sample has as many
// CTAs as fill `ctas` SMs once, or some times over where the samples do not divide them (80 samples would leave 72 of 152 idle): a
// round costs its turns and those that a CTA's start and end are worth, and a further round has to save a twentieth (80 samples of
// 1024 x 1152: forward 163 us in one round, 125 in three, backward 386 and 259, 200 samples 343 and 293, 770 and 564).
constexpr int64_t kTurnsOfStart = 4;
RowPlan row_plan(int64_t B, int64_t N, int64_t D, int64_t ctas, int warps) {
  RowPlan q;
  q.nvec = static_cast<int>(D / 8);
  q.V = q.nvec > 32 ? 2 : 1;
  q.W = (q.nvec + 32 * q.V - 1) / (32 * q.V);
  q.warps = q.W > warps ? kMaxWarps : warps;
  q.G = q.warps / q.W;
  if (q.G > 15) q.G = 15;               // named barriers 1 .. 15
  const int64_t most = (N + q.G - 1) / q.G, rounds = (B + ctas - 1) / ctas;
  int64_t least = -1;
  for (int64_t r = rounds; r < rounds + 4; ++r) {
    const int64_t c = r * ctas / B < most ? r * ctas / B : most;
    const int64_t cost = (B * c + ctas - 1) / ctas * ((N + c * q.G - 1) / (c * q.G) + kTurnsOfStart);
    if (least < 0 || 20 * cost < 19 * least) least = cost, q.ctas = c;
  }
  return q;
}

// This thread's place: its row group, its warp and lane in it, its CTA's rows, and its features.  A vector of a warp is 256 features.
// Of a bf16 stream a lane has eight neighbours of them (16 bytes); of an fp32 one four and, 128 further, four (16 bytes each), so
// that a warp copies and stores 512 bytes in a row there too (with eight neighbours to a lane, whose halves two instructions
// bring, 80,000 x 1536 without norms took 241 us forward instead of 191).
template <bool F32, int V>
struct Place {
  int group, warp, lane;
  int own, span;                        // this lane's first feature, that of the warp's features that it copies of a bf16 tensor
  bool copies[V], valid[V][2];          // whether these are in the row: vector i's copy, and half h of what the lane works on
  int64_t b, first, step, end;          // sample; rows: first, first + step, .. below end
  DSV_DEVICE Place(const RowPlan& plan, int64_t N) {
    const int w = threadIdx.x >> 5;
    group = w / plan.W;
    warp = w % plan.W;
    lane = threadIdx.x & 31;
    own = warp * V * 256 + (F32 ? 4 : 8) * lane;
    span = F32 ? 4 * lane : 0;
    b = blockIdx.x / plan.ctas;
    first = blockIdx.x % plan.ctas * plan.G + group;
    step = plan.ctas * plan.G;
    end = N;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      copies[i] = own + span + 256 * i < 8 * plan.nvec;
#pragma unroll
      for (int h = 0; h < 2; ++h) valid[i][h] = F32 ? col(i, h) < 8 * plan.nvec : copies[i];
    }
  }
  static constexpr int kHalf = F32 ? 128 : 4;   // features from its first half to its second
  DSV_DEVICE int col(int i, int h) const { return own + 256 * i + kHalf * h; }
  DSV_DEVICE int slot(int i) const { return (warp * V + i) * 32 + lane; }
  // those entries of a bf16 vector (zeros past its end), or of one that is not there
  DSV_DEVICE Vec8 vector(const bf16* p, int i, float absent) const {
    Vec8 o = all8(0.f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!valid[i][h]) continue;
      o.v[2 * h] = o.v[2 * h + 1] = both(absent);
      if (p) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p + col(i, h)));
        o.v[2 * h] = make_float2(bf16_lo(a.x), bf16_hi(a.x));
        o.v[2 * h + 1] = make_float2(bf16_lo(a.y), bf16_hi(a.y));
      }
    }
    return o;
  }
  // stores them to a bf16 tensor, or to the stream; `at`: the element of this lane's first feature in the row
  DSV_DEVICE void store(bf16* p, int64_t at, int i, const Vec8& a) const {
    const uint4 v = pack8(a);
    bf16* const to = p + at + 256 * i;
    if constexpr (!F32) {
      if (copies[i]) *reinterpret_cast<uint4*>(to) = v;
    } else {
      if (valid[i][0]) *reinterpret_cast<uint2*>(to) = make_uint2(v.x, v.y);
      if (valid[i][1]) *reinterpret_cast<uint2*>(to + kHalf) = make_uint2(v.z, v.w);
    }
  }
  DSV_DEVICE void store_stream(void* p, int64_t at, int i, const Vec8& a) const {
    if constexpr (!F32) {
      store(static_cast<bf16*>(p), at, i, a);
    } else {
      float* const to = static_cast<float*>(p) + at + 256 * i;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (valid[i][h]) *reinterpret_cast<float4*>(to + kHalf * h) = make_float4(a.v[2 * h].x, a.v[2 * h].y, a.v[2 * h + 1].x, a.v[2 * h + 1].y);
    }
  }
};

// Sums over a row.  The W warps of a row meet at a barrier of their own (1 + group).  HALVES: of two sums over more than four warps
// each half of the lanes adds up one (forward, both norms, 16,384 x 8192 168 us against 185, 32,768 x 4096 164 against 170; in the
// backward 65,536 x 2048 took 259 instead of 270 and 131,072 x 768 194 instead of 187, which have four and two warps a row: how the
// compiler places the rest; it stays as it was).
constexpr int kSums = 3;
constexpr int kRedFloats = 2 * kSums * kMaxWarps;   // of a row group
template <bool HALVES>
struct RowSums {
  int W, group, warp, lane, turn;
  float* red;                           // [2][kSums][kMaxWarps] of the group, zero from W on
  // K sums over the row, the same bits in every thread.  Two and three sums share their shuffles: the lanes' halves
  // (quarters) each go on with one of them.  Two buffers in turn: a thread writes one only after the barrier of the sum in
  // between, which every reader of its last use has passed.
  template <int K>
  DSV_DEVICE void operator()(float (&s)[K]) {
    constexpr unsigned kAll = 0xffffffffu;
    float v = s[0];
    if constexpr (K > 1) {
      const bool high = lane & 16;
      const float give = high ? s[0] : s[1];
      v = (high ? s[1] : s[0]) + __shfl_xor_sync(kAll, give, 16);
    }
    if constexpr (K > 2) {
      const bool third = lane & 8;
      const float w = s[2] + __shfl_xor_sync(kAll, s[2], 16), give = third ? v : w;
      v = (third ? w : v) + __shfl_xor_sync(kAll, give, 8);
    }
#pragma unroll
    for (int o = K == 1 ? 16 : K == 2 ? 8 : 4; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    // sum k is in lane 0, 16, 8
    if (W == 1) {
      s[0] = K == 1 ? v : __shfl_sync(kAll, v, 0);
      if constexpr (K > 1) s[1] = __shfl_sync(kAll, v, 16);
      if constexpr (K > 2) s[2] = __shfl_sync(kAll, v, 8);
      return;
    }
    float* buf = red + turn * (kSums * kMaxWarps);
    turn ^= 1;
    if (lane == 0 || (K > 1 && lane == 16) || (K > 2 && lane == 8)) buf[(lane == 16 ? 1 : lane == 8 ? 2 : 0) * kMaxWarps + warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(32 * W) : "memory");
    auto warps = [&](int k) {             // the warps' parts of sum k
      const float4* p = reinterpret_cast<const float4*>(buf + k * kMaxWarps);
      float4 t = p[0];
      float2 a = add2(make_float2(t.x, t.y), make_float2(t.z, t.w));
      for (int w = 4; w < W; w += 4) {
        t = p[w / 4];
        a = add2(a, add2(make_float2(t.x, t.y), make_float2(t.z, t.w)));
      }
      return a.x + a.y;
    };
    if constexpr (HALVES && K == 2) {
      if (W > 4) {
        const float mine = warps(lane >> 4), other = __shfl_xor_sync(kAll, mine, 16);
        s[0] = lane & 16 ? other : mine;
        s[1] = lane & 16 ? mine : other;
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < K; ++i) s[i] = warps(i);
  }
};
// s / D to the last bit wherever that is a number of fp32, without a division.
DSV_DEVICE float mean_of(float s, float D, float inv_d) {
  const float m = s * inv_d;
  return fmaf(fmaf(-m, D, s), inv_d, m);
}
// A layer norm's mean is only as exact as the sum over the row: rounded, it can be some last bits of the features off, which in a
// row far from 0 with little spread is much of the spread (of a constant row of 1000.1, 768 features, it made xhat 0.06
// instead of 0).  So the deviations d from that mean are summed too, beside their squares: their own mean is what it is off by, and
// (sum d^2) / D - off^2 is the variance, in which nothing large cancels: off is a few roundings of the mean.
struct Spread {
  float off, rstd;
};
DSV_DEVICE Spread spread_of(float d, float dd, float D, float inv_d, float eps) {
  const float off = mean_of(d, D, inv_d), var = fmaf(-off, off, dd * inv_d);
  return Spread{off, rsqrtf((var < 0.f ? 0.f : var) + eps)};   // a variance that is NaN stays so
}
template <bool HALVES>
DSV_DEVICE RowSums<HALVES> row_sums(const RowPlan& plan, float* red, int group, int warp, int lane) {
  for (int i = threadIdx.x; i < 15 * kRedFloats; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
  return RowSums<HALVES>{plan.W, group, warp, lane, 0, red + group * kRedFloats};
}

// A row's features on their way: S stages of P 16-byte parts for each vector of a thread in shared memory.  Parts of the stream
// and, with a bf16 stream, all parts are read by the thread that copied them.  With an fp32 stream a bf16 tensor's are read by the
// lanes that work on them, behind a __syncwarp.
template <bool F32, int P, int V, int S>
struct Ring {
  uint32_t base, stride;                // this thread's part 0 of stage 0; bytes between parts
  DSV_DEVICE Ring(void* smem) : base(smem_u32(smem) + 16 * threadIdx.x), stride(16 * blockDim.x) {
    // lanes past the row's end, and a tensor that is not there, are zeros throughout: they add nothing to a sum
#pragma unroll
    for (int k = 0; k < S * V * P; ++k) asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};\n" ::"r"(base + k * stride), "r"(0) : "memory");
    __syncwarp();
  }
  DSV_DEVICE uint32_t at(int stage, int i, int part) const { return base + ((stage * V + i) * P + part) * stride; }
  static DSV_DEVICE void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(from) : "memory");
  }
  // of a bf16 tensor, of the stream; `at`: the element of this lane's first feature in the row
  DSV_DEVICE void copy(const Place<F32, V>& me, int stage, int i, int part, const bf16* p, int64_t from) const {
    if (me.copies[i]) copy16(at(stage, i, part), p + from + me.span + 256 * i);
  }
  DSV_DEVICE void copy_stream(const Place<F32, V>& me, int stage, int i, int part, const void* p, int64_t from) const {
    if constexpr (!F32) {
      copy(me, stage, i, part, static_cast<const bf16*>(p), from);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (me.valid[i][h]) copy16(at(stage, i, part + h), static_cast<const float*>(p) + from + 256 * i + me.kHalf * h);
    }
  }
  static DSV_DEVICE uint4 read(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
  }
  DSV_DEVICE Vec8 bf8(const Place<F32, V>& me, int stage, int i, int part) const { return unpack8(bf16x8(me, stage, i, part)); }
  DSV_DEVICE uint4 bf16x8(const Place<F32, V>& me, int stage, int i, int part) const {
    if constexpr (!F32) {
      return read(at(stage, i, part));
    } else {
      uint4 v;
      const uint32_t a = at(stage, i, part) - 8 * me.lane;   // the warp's 512 bytes: from 8 l and 256 + 8 l on
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
      asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(v.z), "=r"(v.w) : "r"(a + 256) : "memory");
      return v;
    }
  }
  DSV_DEVICE Vec8 stream8(int stage, int i, int part) const {
    uint4 v[Stream<F32>::kParts];
#pragma unroll
    for (int k = 0; k < Stream<F32>::kParts; ++k) v[k] = read(at(stage, i, part + k));
    return Stream<F32>::get(v);
  }
  static __host__ __device__ size_t bytes(int threads) { return static_cast<size_t>(S) * V * P * 16 * threads; }
};

// ---------------------------------------------------------------- forward
constexpr int kFwdStages = 4;
constexpr int64_t kFwdCtas = 152;

template <bool F32, int V, bool POST, int PRE>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
residual_norm_fwd_kernel(ResidualParams p, RowPlan plan) {
  extern __shared__ __align__(16) uint4 ring_mem[];
  __shared__ __align__(16) float red[15 * kRedFloats];
  constexpr int SP = Stream<F32>::kParts, P = SP + 1, S = kFwdStages;
  const Place<F32, V> me(plan, p.N);
  RowSums<true> sum = row_sums<true>(plan, red, me.group, me.warp, me.lane);
  const Ring<F32, P, V, S> ring(ring_mem);
  const float D = static_cast<float>(p.D), inv_d = 1.f / D;

  const int64_t step = me.step * p.D;   // elements between this thread's rows
  int64_t row = (me.b * p.N + me.first) * p.D + me.own;
  auto issue = [&](int64_t n, int64_t at, int stage) {
    if (n < me.end) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ring.copy_stream(me, stage, i, 0, p.x, at);
        ring.copy(me, stage, i, SP, p.z, at);
      }
    }
    cp_async_commit();                  // one group a row, so that the wait below counts rows
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(me.first + s * me.step, row + s * step, s);

  Vec8 c[V], f[V], sh[V];               // alpha gate w_post, w_pre (1 + scale), shift
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const Vec8 g = me.vector(p.gate ? p.gate + me.b * p.gate_stride : nullptr, i, 1.f);
    const Vec8 wz = me.vector(POST ? p.w_post : nullptr, i, 1.f), wr = me.vector(p.w_pre, i, 1.f);
    const Vec8 sc = me.vector(p.scale ? p.scale + me.b * p.scale_stride : nullptr, i, 0.f);
    sh[i] = me.vector(p.shift ? p.shift + me.b * p.shift_stride : nullptr, i, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[i].v[j] = mul2(mul2(both(p.alpha), g.v[j]), wz.v[j]);
      f[i].v[j] = mul2(wr.v[j], add2(both(1.f), sc.v[j]));
    }
  }

  // The branch's norm of a row is known before the row's turn: its sum shares the reduction of the row before it (520,192 x 2048,
  // RMS norms, 1,325 us instead of 1,382, 16,384 x 8192 166 instead of 178).
  uint4 ahead[V];                       // z of the next row
  auto look_ahead = [&](int at) {
    float2 a = both(0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ahead[i] = ring.bf16x8(me, at, i, SP);
      const Vec8 z = unpack8(ahead[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) a = fma2(z.v[j], z.v[j], a);
    }
    return a.x + a.y;
  };
  float rz = 1.f;
  if constexpr (POST) {
    cp_async_wait<S - 2>();
    if (F32) __syncwarp();
    float s[1] = {look_ahead(0)};
    sum(s);
    rz = rsqrtf(s[0] * inv_d + p.eps);
  }
  int stage = 0;
  for (int64_t n = me.first; n < me.end; n += me.step, row += step) {
    cp_async_wait<POST ? S - 3 : S - 2>();
    if (F32) __syncwarp();
    Vec8 r[V], z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      r[i] = ring.stream8(stage, i, 0);
      z[i] = POST ? unpack8(ahead[i]) : ring.bf8(me, stage, i, SP);
    }
    const int last = stage ? stage - 1 : S - 1;   // where the last row was read from
    stage = stage + 1 < S ? stage + 1 : 0;
    const float sz = POST ? look_ahead(stage) : 0.f;
    if (F32) __syncwarp();
    issue(n + (S - 1) * me.step, row + (S - 1) * step, last);
    float2 a = both(0.f);               // sum of r (layer) or r^2 (rms)
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[i].v[j] = fma2(c[i].v[j], POST ? mul2(z[i].v[j], both(rz)) : z[i].v[j], r[i].v[j]);
        a = PRE == kNormLayer ? add2(a, r[i].v[j]) : fma2(r[i].v[j], r[i].v[j], a);
      }
      me.store_stream(p.r, row, i, r[i]);
    }
    if constexpr (POST && PRE == kNormNone) {
      float s[1] = {sz};
      sum(s);
      rz = rsqrtf(s[0] * inv_d + p.eps);
    }
    if constexpr (PRE != kNormNone) {
      float s[1];
      if constexpr (POST) {
        float s2[2] = {a.x + a.y, sz};
        sum(s2);
        s[0] = s2[0];
        rz = rsqrtf(s2[1] * inv_d + p.eps);
      } else {
        s[0] = a.x + a.y;
        sum(s);
      }
      float2 rstd, shifted = both(0.f);
      if constexpr (PRE == kNormLayer) {
        const float mean = mean_of(s[0], D, inv_d);
        float2 e = both(0.f);
        a = both(0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            r[i].v[j] = add2(r[i].v[j], both(me.valid[i][j / 2] ? -mean : 0.f));
            e = add2(e, r[i].v[j]);
            a = fma2(r[i].v[j], r[i].v[j], a);
          }
        }
        float s2[2] = {e.x + e.y, a.x + a.y};
        sum(s2);
        const Spread t = spread_of(s2[0], s2[1], D, inv_d, p.eps);
        rstd = both(t.rstd);
        shifted = both(-t.off * t.rstd);
      } else {
        rstd = both(rsqrtf(s[0] * inv_d + p.eps));
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 xh = PRE == kNormLayer ? fma2(r[i].v[j], rstd, shifted) : mul2(r[i].v[j], rstd);
          r[i].v[j] = fma2(xh, f[i].v[j], sh[i].v[j]);
        }
        me.store(p.y, row, i, r[i]);
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
//   A row's passes read it from shared memory again, in bf16 as it came: held in registers in fp32 it would leave room for 12
// warps instead of 16, and for eight where a row takes all of them (16,384 x 8192: 766 us
// against 440 so, 370 with rows in turn then, and 379 now with the next paragraph's sums).
//   A layer norm's deviations need the mean, which is a reduction away.  The first pass takes them from the mean p of a lane's own
// eight features: with d = r - p and a = p - mean, sum (r - mean)^2 = sum d^2 + a (2 sum d + 8 a) and sum h (r - mean) =
// sum h d + a sum h, with nothing large to cancel however far the row lies from 0, and no pass over the row
// between the two reductions (65,536 x 2048, both norms, 277 to 269 us; 131,072 x 768, no branch norm, 197 to 186; 16,384 x 8192 370 to 379).
//   Of an fp32 stream the second reduction also sums r - mean, whose own mean is taken off (spread_of; 80,000 x 1536, both norms, 351 us
// instead of 366, 3 x 3,645 x 1160 60 instead of 57).  A bf16 stream needs that in the forward alone, whose rows are new in fp32:
// its features have eight bits, so that up to 8192 of them within a factor of eight add up exactly, and of others the sum's roundings are
// 2^-11 of the spread at most (with that sum all the same 65,536 x 2048 took 293 us).
constexpr int64_t kBwdCtas = 152;
constexpr int sums_of(int pre) { return pre == kNormNone ? 1 : 3; }
// Warps of a CTA: with an fp32 stream 12, whose two stages and factors fill shared memory, and 16 for rows that need more.
template <bool F32>
constexpr int bwd_warps() {
  return F32 ? 12 : kMaxWarps;
}
// The factors alpha gate w_post and w_pre (1 + scale) stay in shared memory, 64 bytes a vector of a row; where rows of fp32 take 16
// warps they are made again from the bf16 vectors.
template <bool F32, int WARPS>
constexpr bool kept_factors() {
  return WARPS <= bwd_warps<F32>();
}
template <int P>
constexpr int bwd_stages() {
  return P <= 3 ? 3 : 2;
}

template <bool F32, int V, bool POST, int PRE, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1)
residual_norm_bwd_kernel(ResidualParams p, RowPlan plan) {
  extern __shared__ __align__(16) uint4 ring_mem[];
  __shared__ __align__(16) float red[15 * kRedFloats];
  constexpr int SP = Stream<F32>::kParts, P = PRE == kNormNone ? SP + 1 : 2 * SP + 2, S = bwd_stages<P>();
  constexpr int K = PRE == kNormNone ? 1 : 3;
  constexpr bool kCentred = F32 && PRE == kNormLayer;           // the deviations' own mean is taken off them
  constexpr int kDr = 0, kZ = SP, kDy = SP + 1, kR = SP + 2;    // parts of a vector
  // the kernel of the sums may be scheduled once every CTA has started; it waits for this grid before it reads
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const Place<F32, V> me(plan, p.N);
  RowSums<false> sum = row_sums<false>(plan, red, me.group, me.warp, me.lane);
  const Ring<F32, P, V, S> ring(ring_mem);
  const float D = static_cast<float>(p.D), inv_d = 1.f / D;

  const int64_t step = me.step * p.D;   // elements between this thread's rows
  int64_t row = (me.b * p.N + me.first) * p.D + me.own;
  auto issue = [&](int64_t n, int64_t at, int stage) {
    if (n < me.end) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if constexpr (PRE != kNormNone) {
          ring.copy_stream(me, stage, i, kR, p.r, at);
          ring.copy(me, stage, i, kDy, p.dy, at);
        }
        ring.copy(me, stage, i, kZ, p.z, at);
        if (p.dr) ring.copy_stream(me, stage, i, kDr, p.dr, at);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(me.first + s * me.step, row + s * step, s);

  // the two factors of vector i
  auto make_c = [&](int i) {
    Vec8 c = me.vector(p.gate ? p.gate + me.b * p.gate_stride : nullptr, i, 1.f);
    const Vec8 w = me.vector(POST ? p.w_post : nullptr, i, 1.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) c.v[j] = mul2(mul2(both(p.alpha), c.v[j]), w.v[j]);
    return c;
  };
  auto make_f = [&](int i) {
    Vec8 f = me.vector(p.w_pre, i, 1.f);
    const Vec8 sc = me.vector(p.scale ? p.scale + me.b * p.scale_stride : nullptr, i, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = mul2(f.v[j], add2(both(1.f), sc.v[j]));
    return f;
  };
  constexpr bool kKept = kept_factors<F32, WARPS>();
  const int row_vecs = 32 * V * plan.W;          // with those past the end
  float4* const kept = reinterpret_cast<float4*>(reinterpret_cast<char*>(ring_mem) + Ring<F32, P, V, S>::bytes(blockDim.x));   // [4][row_vecs]
  auto keep = [&](int slot, int vec, const Vec8& a) {
    kept[slot * row_vecs + vec] = make_float4(a.v[0].x, a.v[0].y, a.v[1].x, a.v[1].y);
    kept[(slot + 1) * row_vecs + vec] = make_float4(a.v[2].x, a.v[2].y, a.v[3].x, a.v[3].y);
  };
  auto kept8 = [&](int slot, int vec) {
    const float4 lo = kept[slot * row_vecs + vec], hi = kept[(slot + 1) * row_vecs + vec];
    return Vec8{{make_float2(lo.x, lo.y), make_float2(lo.z, lo.w), make_float2(hi.x, hi.y), make_float2(hi.z, hi.w)}};
  };
  Vec8 acc[K][V];                       // S, T, U
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (kKept && me.group == 0) {
      keep(0, me.slot(i), make_c(i));
      if (PRE != kNormNone) keep(2, me.slot(i), make_f(i));
    }
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k][i] = all8(0.f);
  }
  if (kKept) __syncthreads();

  int stage = 0;
  for (int64_t n = me.first; n < me.end; n += me.step, row += step) {
    cp_async_wait<S - 2>();
    if (F32) __syncwarp();
    issue(n + (S - 1) * me.step, row + (S - 1) * step, stage ? stage - 1 : S - 1);   // where the last row was
    // the row's features of vector i, and h = dy f
    auto stream8 = [&](int i, int part) { return ring.stream8(stage, i, part); };
    auto bf8 = [&](int i, int part) { return ring.bf8(me, stage, i, part); };
    auto h8 = [&](int i, const Vec8& dy) {
      Vec8 f = kKept ? kept8(2, me.slot(i)) : make_f(i);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = mul2(dy.v[j], f.v[j]);
      return f;
    };

    float rz = 1.f, mean = 0.f;
    float2 k0 = both(0.f), k1 = both(0.f), k2 = both(0.f), k3 = both(0.f);   // of  g = dr + k2 h + k1 xhat + k0,  xhat = k2 (r - mean) + k3
    if constexpr (POST || PRE != kNormNone) {
      float2 a0 = both(0.f), a1 = both(0.f), a2 = both(0.f);   // sum z^2; layer: sum d^2, sum h d; rms: sum r^2, sum h r
      float s1 = 0.f, s2 = 0.f;         // layer: sum r, sum h
      float pivot[V], off[V], hs[V];    // layer, of each vector: the mean of its features, sum d, sum h
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (POST) {
          const Vec8 z = bf8(i, kZ);
#pragma unroll
          for (int j = 0; j < 4; ++j) a0 = fma2(z.v[j], z.v[j], a0);
        }
        if constexpr (PRE != kNormNone) {
          const Vec8 r = stream8(i, kR), h = h8(i, bf8(i, kDy));
          if constexpr (PRE == kNormLayer) {
            const float2 tr = add2(add2(r.v[0], r.v[1]), add2(r.v[2], r.v[3])), th = add2(add2(h.v[0], h.v[1]), add2(h.v[2], h.v[3]));
            const float sr = tr.x + tr.y;
            hs[i] = th.x + th.y;
            s1 += sr;
            s2 += hs[i];
            pivot[i] = sr * (me.valid[i][1] ? 0.125f : 0.25f);
            float2 e = both(0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 d = add2(r.v[j], both(me.valid[i][j / 2] ? -pivot[i] : 0.f));
              e = add2(e, d);
              a1 = fma2(d, d, a1);
              a2 = fma2(h.v[j], d, a2);
            }
            off[i] = e.x + e.y;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              a1 = fma2(r.v[j], r.v[j], a1);
              a2 = fma2(h.v[j], r.v[j], a2);
            }
          }
        }
      }
      float s0 = a0.x + a0.y;
      if constexpr (PRE == kNormRms) {
        s1 = a1.x + a1.y;
        s2 = a2.x + a2.y;
      }
      if constexpr (PRE == kNormNone) {
        float s[1] = {s0};
        sum(s);
        s0 = s[0];
      } else if constexpr (!POST) {
        float s[2] = {s1, s2};
        sum(s);
        s1 = s[0];
        s2 = s[1];
      } else {
        float s[3] = {s0, s1, s2};
        sum(s);
        s0 = s[0];
        s1 = s[1];
        s2 = s[2];
      }
      if (POST) rz = rsqrtf(s0 * inv_d + p.eps);
      if constexpr (PRE != kNormNone) {
        float mh = 0.f, rstd;           // mean h
        if constexpr (PRE == kNormLayer) {
          mean = mean_of(s1, D, inv_d);
          mh = s2 * inv_d;
          float s[kCentred ? 3 : 2] = {a1.x + a1.y, a2.x + a2.y};   // sums of (r - mean)^2, h (r - mean) and r - mean
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float a = pivot[i] - mean, n = me.valid[i][1] ? 8.f : me.valid[i][0] ? 4.f : 0.f;
            s[0] = fmaf(a, fmaf(n, a, 2.f * off[i]), s[0]);
            s[1] = fmaf(a, hs[i], s[1]);
            if constexpr (kCentred) s[2] += fmaf(n, a, off[i]);
          }
          sum(s);
          s1 = s[0];
          if constexpr (kCentred) {
            const Spread t = spread_of(s[2], s1, D, inv_d, p.eps);
            rstd = t.rstd;
            k3 = both(-t.off * rstd);
            s2 = fmaf(-t.off, s2, s[1]);
          } else {
            s2 = s[1];
          }
        }
        if constexpr (!kCentred) rstd = rsqrtf(s1 * inv_d + p.eps);
        const float mhx = rstd * s2 * inv_d;   // mean(h xhat)
        k0 = both(-rstd * mh);
        k1 = both(-rstd * mhx);
        k2 = both(rstd);
      }
    }
    float2 a = both(0.f);               // sum u zhat
    Vec8 u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      Vec8 g = stream8(i, kDr);
      if constexpr (PRE != kNormNone) {
        const Vec8 dy = bf8(i, kDy), h = h8(i, dy), r = stream8(i, kR);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 d = PRE == kNormLayer ? add2(r.v[j], both(-mean)) : r.v[j], xh = kCentred ? fma2(d, k2, k3) : mul2(d, k2);
          g.v[j] = add2(g.v[j], fma2(k2, h.v[j], fma2(k1, xh, k0)));
          acc[K - 2][i].v[j] = fma2(dy.v[j], xh, acc[K - 2][i].v[j]);
          acc[K - 1][i].v[j] = add2(acc[K - 1][i].v[j], dy.v[j]);
        }
      }
      me.store_stream(p.dx, row, i, g);
      const Vec8 c = kKept ? kept8(0, me.slot(i)) : make_c(i), z = bf8(i, kZ);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 zh = POST ? mul2(z.v[j], both(rz)) : z.v[j];
        acc[0][i].v[j] = fma2(g.v[j], zh, acc[0][i].v[j]);
        u[i].v[j] = mul2(c.v[j], g.v[j]);
        if (POST) a = fma2(u[i].v[j], zh, a);
      }
    }
    float2 mu = both(0.f);              // -mean(u zhat)
    if constexpr (POST) {
      float s[1] = {a.x + a.y};
      sum(s);
      mu = both(-s[0] * inv_d);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (POST) {
        const Vec8 z = bf8(i, kZ);
#pragma unroll
        for (int j = 0; j < 4; ++j) u[i].v[j] = mul2(both(rz), fma2(mul2(z.v[j], both(rz)), mu, u[i].v[j]));
      }
      me.store(p.dz, row, i, u[i]);
    }
    if (F32) __syncwarp();              // the next row's copies go where other lanes have read this one's
    stage = stage + 1 < S ? stage + 1 : 0;
  }

  // the row groups' sums, where the rows were, added in the groups' order
  cp_async_wait<0>();
  __syncthreads();
  float* const cols = reinterpret_cast<float*>(ring_mem);   // [G][K][D]
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (me.valid[i][h])
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float2 lo = acc[k][i].v[2 * h], hi = acc[k][i].v[2 * h + 1];
          *reinterpret_cast<float4*>(cols + (me.group * K + k) * p.D + me.col(i, h)) = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
  __syncthreads();
  float4* const out = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * K * p.D);
  const int quads = K * static_cast<int>(p.D) / 4;
  for (int i = threadIdx.x; i < quads; i += blockDim.x) {
    float4 t = reinterpret_cast<const float4*>(cols)[i];
    for (int g = 1; g < plan.G; ++g) {
      const float4 a = reinterpret_cast<const float4*>(cols)[g * quads + i];
      t = make_float4(t.x + a.x, t.y + a.y, t.z + a.z, t.w + a.w);
    }
    out[i] = t;
  }
}

// The gradients of the vectors from the CTAs' partial rows: a CTA takes 32 features of one of the sums S, T, U, a sample's `each`
// warps every each-th partial row, ten loads leaving together; their sums are added in order.  `each` is what the sample's partial
// rows keep busy, and the CTA's other warps take the next samples (sixteen warps to each of them: 200 samples of 64 x 1152 122 us for
// the call instead of 63, 24 of 1024 x 1152 77 instead of 70).  The weights' gradients are sums over the samples too: a few samples are the same CTA's in turn, more leave
// their parts behind the partial rows, for a last kernel.
constexpr int kSumWarps = 16, kLoads = 10;
constexpr int64_t kSamplesInTurn = 4;
__global__ void __launch_bounds__(32 * kSumWarps)
residual_vectors_kernel(ResidualParams p, int64_t parts, int each, int64_t samples, float* per_sample) {
  __shared__ float red[2][kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.y, K = gridDim.y;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t first = blockIdx.z * samples, last = min(first + samples, p.B);   // the CTA's samples
  const int at_once = kSumWarps / each;
  const bool inside = d < p.D;
  float weight = 0.f;                   // the gradient of w_post (S) or w_pre (T)
  int turn = 0;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the partial rows
  for (int64_t b0 = first; b0 < last; b0 += at_once, turn ^= 1) {
    const int64_t b = b0 + warp / each;
    const bool here = inside && b < last;
    const float* const rows = p.partial + (b * parts * K + k) * p.D + d;
    float s = 0.f;
    for (int64_t t0 = warp % each; t0 < parts; t0 += kLoads * each) {
      float v[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) v[u] = here && t0 + u * each < parts ? rows[(t0 + u * each) * K * p.D] : 0.f;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) s += v[u];
    }
    red[turn][warp][lane] = s;          // the last turn's are read meanwhile
    __syncthreads();
    if (warp % each || !here) continue;
    for (int w = 1; w < each; ++w) s += red[turn][warp + w][lane];
    float part = 0.f;                   // of the weight's gradient
    if (k == 0) {
      if (p.d_gate) p.d_gate[b * p.d_stride + d] = p.alpha * s * (p.w_post ? __bfloat162float(p.w_post[d]) : 1.f);
      part = p.alpha * s * (p.gate ? __bfloat162float(p.gate[b * p.gate_stride + d]) : 1.f);
    } else if (k == 1) {
      if (p.d_scale) p.d_scale[b * p.d_stride + d] = s * (p.w_pre ? __bfloat162float(p.w_pre[d]) : 1.f);
      part = s * (1.f + (p.scale ? __bfloat162float(p.scale[b * p.scale_stride + d]) : 0.f));
    } else if (p.d_shift) {
      p.d_shift[b * p.d_stride + d] = s;
    }
    if (per_sample && k < 2) per_sample[(2 * b + k) * p.D + d] = part;
    weight += part;
  }
  // with no kernel after this one a CTA has all samples, one at a time
  if (warp || !inside || per_sample) return;
  if (k == 0 && p.dw_post) p.dw_post[d] = weight;
  if (k == 1 && p.dw_pre) p.dw_pre[d] = weight;
}
// The weights' gradients from the samples' parts: 32 features of one of them to a CTA, every sixteenth sample to a warp.
__global__ void __launch_bounds__(32 * kSumWarps)
residual_weights_kernel(ResidualParams p, const float* per_sample) {
  __shared__ float red[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.y;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float* const out = k ? p.dw_pre : p.dw_post;
  float s = 0.f;
  if (d < p.D && out) {
#pragma unroll 8
    for (int64_t b = warp; b < p.B; b += kSumWarps) s += per_sample[(2 * b + k) * p.D + d];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp || d >= p.D || !out) return;
  for (int w = 1; w < kSumWarps; ++w) s += red[w][lane];
  out[d] = s;
}

template <bool F32, int V, bool POST, int PRE>
cudaError_t fwd(const ResidualParams& p, const RowPlan& plan, cudaStream_t stream) {
  constexpr auto kernel = residual_norm_fwd_kernel<F32, V, POST, PRE>;
  const int threads = 32 * plan.W * plan.G;
  const size_t smem = Ring<F32, Stream<F32>::kParts + 1, V, kFwdStages>::bytes(threads);
  const cudaError_t e = allow_shared<kernel>(kMaxShared);
  if (e != cudaSuccess) return e;
  ProfScope prof("residual_norm_fwd", stream);
  kernel<<<static_cast<unsigned>(p.B * plan.ctas), threads, smem, stream>>>(p, plan);
  return cudaGetLastError();
}
template <bool F32, int V, bool POST, int PRE, int WARPS>
cudaError_t bwd_rows(const ResidualParams& p, const RowPlan& plan, cudaStream_t stream) {
  const int K = sums_of(PRE), threads = 32 * plan.W * plan.G;
  constexpr int SP = Stream<F32>::kParts, P = PRE == kNormNone ? SP + 1 : 2 * SP + 2;
  const size_t cols = static_cast<size_t>(K) * plan.G * p.D * sizeof(float), ring = Ring<F32, P, V, bwd_stages<P>()>::bytes(threads);
  const size_t factors = kept_factors<F32, WARPS>() ? static_cast<size_t>(V) * 64 * 32 * plan.W : 0;
  const size_t smem = cols > ring + factors ? cols : ring + factors;
  constexpr auto kernel = residual_norm_bwd_kernel<F32, V, POST, PRE, WARPS>;
  const cudaError_t e = allow_shared<kernel>(kMaxShared);
  if (e != cudaSuccess) return e;
  ProfScope prof("residual_norm_bwd", stream);
  kernel<<<static_cast<unsigned>(p.B * plan.ctas), threads, smem, stream>>>(p, plan);
  return cudaGetLastError();
}
template <bool F32, int V, bool POST, int PRE>
cudaError_t bwd(const ResidualParams& p, const RowPlan& plan, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  constexpr int kWarps = bwd_warps<F32>();
  if (V == 1 || plan.warps == kWarps) e = bwd_rows<F32, V, POST, PRE, kWarps>(p, plan, stream);
  else if constexpr (V == 2) e = bwd_rows<F32, V, POST, PRE, kMaxWarps>(p, plan, stream);
  if (e != cudaSuccess) return e;
  const bool weights = p.dw_post || p.dw_pre;
  if (!p.d_gate && !p.d_scale && !p.d_shift && !weights) return cudaSuccess;
  const bool turns = weights && p.B <= kSamplesInTurn;   // a sample costs a turn about 1 us, another kernel 3
  float* per_sample = weights && !turns ? p.partial + p.B * plan.ctas * sums_of(PRE) * p.D : nullptr;
  {
    ProfScope prof("residual_vectors", stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    int each = kSumWarps;
    while (!turns && each > 1 && plan.ctas <= kLoads * each / 2) each /= 2;
    const int64_t samples = turns ? p.B : kSumWarps / each;
    cfg.gridDim = dim3(static_cast<unsigned>((p.D + 31) / 32), sums_of(PRE), static_cast<unsigned>((p.B + samples - 1) / samples));
    cfg.blockDim = dim3(32 * kSumWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, residual_vectors_kernel, p, plan.ctas, each, samples, per_sample)) != cudaSuccess) return e;
  }
  if (!per_sample) return cudaSuccess;
  ProfScope prof("residual_weights", stream);
  residual_weights_kernel<<<dim3(static_cast<unsigned>((p.D + 31) / 32), 2), 32 * kSumWarps, 0, stream>>>(p, per_sample);
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

size_t residual_bwd_workspace(int64_t B, int64_t N, int64_t D, int pre, bool f32) {
  const RowPlan q = row_plan(B, N, D, kBwdCtas, f32 ? bwd_warps<true>() : bwd_warps<false>());
  return static_cast<size_t>(B * q.ctas * sums_of(pre) + 2 * B) * D * sizeof(float);
}

cudaError_t launch_residual_norm_fwd(const ResidualParams& p, cudaStream_t stream) {
  const RowPlan plan = row_plan(p.B, p.N, p.D, kFwdCtas, kMaxWarps);
  return DSV_RESIDUAL_PICK(fwd, plan.V, p, plan, stream);
}
cudaError_t launch_residual_norm_bwd(const ResidualParams& p, cudaStream_t stream) {
  const RowPlan plan = row_plan(p.B, p.N, p.D, kBwdCtas, p.f32 ? bwd_warps<true>() : bwd_warps<false>());
  return DSV_RESIDUAL_PICK(bwd, plan.V, p, plan, stream);
}

}  // namespace dsv
