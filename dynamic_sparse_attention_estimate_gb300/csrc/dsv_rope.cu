// Rotary positions with several axes (time, height, width), alone and behind the per-head RMS norm
// of queries and keys, both directions.
//
// A head row of d features is d / 8 16-byte vectors, one per lane (LPR = 8 or 16 lanes a row).  Its
// pairs (x0, x1) turn by the angle of their axis: y0 = x0 c - x1 s, y1 = x0 s + x1 c; the backward
// turns by the negative angle.  The angles separate over the axes, so (cos, sin) come from one
// small table per axis (rows = positions, a few KB in all, L1-resident) instead of a [N][d/2]
// array of the clip (266 MB at 520,192 tokens and d = 128): a token costs its 12 bytes of
// coordinates.  With the norm, n = x rstd w with rstd = 1 / sqrt(mean(x^2) + eps) before the
// rotation; the backward recomputes rstd from x:
//   g = rotation^T(dy),  dw = sum_rows g x rstd,  dx = rstd (g w - x rstd^2 mean(g w x)).
//
// Bound: HBM.  A group of LPR lanes owns one token and walks its heads, so a token's (cos, sin) and
// the weights are read once for all its heads and both tensors; a packed token-major projection
// is read front to back, and the head-major outputs get rows of consecutive tokens from
// neighbouring groups.  Queries, keys and values go in one launch: the loads of several
// rows are issued before the first is used, which is what keeps HBM busy (no staging is needed:
// nothing is read twice).  Measured (GB300, 16 heads of 128, 65,536 tokens; a plain copy runs at 6.67 TB/s): rope3d
// 6.3 TB/s, norm and rotation forward 241 us = 6.7 TB/s (520,192 tokens 1.82 ms = 7.0), backward 341 us = 6.3 TB/s,
// halves 2 to 4 % below.  One head of 524,288 tokens: forward 216 us, backward 311 us, about half of that rate: each
// token has its positions, its table entries and, worked out for it anew though they are the lane's, the axis, row
// length and offset of each pair, shared by its heads; two heads are at 0.82 and 0.74 of the copy, eight at the rates above.
#include <type_traits>

#include "dsv_block.h"
#include "dsv_common.cuh"
#include "dsv_internal.h"

namespace dsv {
namespace {

constexpr int kThreads = 128;
constexpr double kBackSetup = 1.5;
constexpr int kBackCtas = 4;   // of the backward, on an SM (128 registers; 5 spill: mid clip 529 us where 4 take 341)

DSV_DEVICE uint32_t word(const uint4& u, int j) { return j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w; }

DSV_DEVICE void unpack(const uint4& u, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(word(u, j));
    f[2 * j + 1] = bf16_hi(word(u, j));
  }
}
DSV_DEVICE uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
DSV_DEVICE uint4 shfl(const uint4& u, int src) {
  return make_uint4(__shfl_sync(0xffffffffu, u.x, src), __shfl_sync(0xffffffffu, u.y, src),
                    __shfl_sync(0xffffffffu, u.z, src), __shfl_sync(0xffffffffu, u.w, src));
}

// Sum over the LPR lanes of a row (every lane gets it; the order is fixed).
template <int LPR>
DSV_DEVICE float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The rotation of one lane's vector at one token: (cos, +-sin) of its pairs.
//   interleaved: pair i of the vector is its elements (2i, 2i + 1); 4 pairs, those from `turned` on pass
//   halves:      element e pairs with element e of the vector `partner` lanes hold; 8 pairs, all or none
template <bool HALF>
struct Turn {
  static constexpr int P = HALF ? 8 : 4;
  float c[P], s[P];
  int turned;   // pairs of this vector that are rotated
};

struct Pos {
  int v[3];
};
DSV_DEVICE Pos load_pos(const RopeGeom& g, const int32_t* __restrict__ pos, int64_t row, bool active) {
  Pos p{{0, 0, 0}};
  if (active && g.pairs) {
#pragma unroll
    for (int a = 0; a < 3; ++a) p.v[a] = __ldg(pos + row * 3 + a);
  }
  return p;
}

// sign: +1 forward, -1 backward.  An axis whose position is outside its table turns its pairs by the
// angle 0 and sets the status bit.  All lanes of the warp call it.
// A lane reads four pairs.  In halves two vectors turn by the same eight: each lane gets the other four from its partner
// (pairs are read 64 bytes apart there, many L1 accesses to a load: with all eight read by both, 524,288 tokens of one
// head took 330 us forward and 396 backward where they take 285 and 336; 131,072 of 16 heads 483 and 710, now 477 and 690).
template <bool HALF>
DSV_DEVICE void make_turn(Turn<HALF>& t, const RopeGeom& g, const float2* __restrict__ table, const Pos& pos,
                          bool active, int vec, int partner, float sign, unsigned int* status) {
  const int half_vecs = g.pairs / 8;   // HALF: vectors of a half (pairs is a multiple of 8)
  const bool second = HALF && vec >= half_vecs;
  int j0;
  if (HALF) {
    j0 = second ? (vec - half_vecs) * 8 + 4 : vec * 8;
    t.turned = vec < 2 * half_vecs ? 8 : 0;
    if (!second) sign = -sign;   // y0 = x0 c - x1 s; y1 = x1 c + x0 s
  } else {
    j0 = vec * 4;
    const int left = g.pairs - j0;
    t.turned = left < 0 ? 0 : left > 4 ? 4 : left;
  }
#pragma unroll
  for (int i = 0; i < Turn<HALF>::P; ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
  }
  if (active && t.turned != 0) {
    int p[3];
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      p[a] = pos.v[a];
      if (g.axis_pairs[a] > 0 && static_cast<uint32_t>(p[a]) >= static_cast<uint32_t>(g.len[a])) {
        flag_status(status, kStatusBadPosition);
        p[a] = -1;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = j0 + i;
      if (i >= t.turned) continue;
      int a = 0, first = 0;
      if (j >= g.axis_pairs[0]) { a = 1; first = g.axis_pairs[0]; }
      if (j >= g.axis_pairs[0] + g.axis_pairs[1]) { a = 2; first = g.axis_pairs[0] + g.axis_pairs[1]; }
      const int pa = a == 0 ? p[0] : a == 1 ? p[1] : p[2];
      const int np = a == 0 ? g.axis_pairs[0] : a == 1 ? g.axis_pairs[1] : g.axis_pairs[2];
      const int64_t off = a == 0 ? 0 : a == 1 ? g.table_off[1] : g.table_off[2];
      if (pa < 0) continue;
      const float2 cs = __ldg(table + off + static_cast<int64_t>(pa) * np + (j - first));
      t.c[i] = cs.x;
      t.s[i] = HALF ? cs.y : sign * cs.y;
    }
  }
  if constexpr (HALF) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = t.c[i], s = t.s[i];
      const float oc = __shfl_sync(0xffffffffu, c, partner), os = __shfl_sync(0xffffffffu, s, partner);
      t.c[i] = second ? oc : c;
      t.s[i] = sign * (second ? os : s);
      t.c[i + 4] = second ? c : oc;
      t.s[i + 4] = sign * (second ? s : os);
    }
  }
}

// f (this lane's 8 values) turned; fp: the partner vector's values (HALF only).
template <bool HALF>
DSV_DEVICE void turn(const Turn<HALF>& t, float (&f)[8], const float (&fp)[8]) {
  if constexpr (HALF) {
    if (t.turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], t.c[e], fp[e] * t.s[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= t.turned) continue;   // features past the rotated ones pass, infinities too
      const float a = f[2 * i], b = f[2 * i + 1];
      f[2 * i] = fmaf(a, t.c[i], -(b * t.s[i]));
      f[2 * i + 1] = fmaf(a, t.s[i], b * t.c[i]);
    }
  }
}

// HALF: the lane of this row that holds the partner vector (itself where nothing turns).
template <int LPR>
DSV_DEVICE int partner_lane(const RopeGeom& g, int lane, int vec) {
  const int hv = g.pairs / 8;
  const int p = vec < hv ? vec + hv : vec < 2 * hv ? vec - hv : vec;
  return (lane & ~(LPR - 1)) | p;
}

// What a group of LPR lanes works on: a token and a chunk of its heads.  (Samples, heads and tokens fit 32 bits.)
struct Lane {
  int b, n, h0, h1;
  bool active;
};

template <int LPR>
DSV_DEVICE Lane lane_of(const RopeGeom& g, int64_t unit) {
  constexpr int kTok = kThreads / LPR;
  const int tile = static_cast<int>(unit / g.chunks), chunk = static_cast<int>(unit - tile * g.chunks);
  const int tiles = static_cast<int>(g.tiles_per_b), per = static_cast<int>(g.heads_per_chunk);
  Lane l;
  l.b = tile / tiles;
  l.n = (tile - l.b * tiles) * kTok + threadIdx.x / LPR;
  l.active = l.n < g.N;
  l.h0 = chunk * per;
  l.h1 = l.h0 + per < g.H ? l.h0 + per : static_cast<int>(g.H);
  return l;
}
DSV_DEVICE int64_t pos_row(const RopeGeom& g, const Lane& l) { return l.b * g.pos_batch + l.n; }

DSV_DEVICE uint4 load_row(const bf16* p) { return *reinterpret_cast<const uint4*>(p); }
// U rows of a view, heads h .. h + U - 1 of this group's token (zeros past its heads).
template <int U>
DSV_DEVICE void load_rows(uint4 (&v)[U], const bf16* p, int64_t stride, int h, const Lane& l) {
#pragma unroll
  for (int u = 0; u < U; ++u)
    v[u] = l.active && h + u < l.h1 ? load_row(p + (h + u) * stride) : make_uint4(0, 0, 0, 0);
}
DSV_DEVICE void store_row(bf16* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }

// ---------------------------------------------------------------- rotation alone
template <int D, bool HALF, int U>
__global__ void __launch_bounds__(kThreads)
rope3d_kernel(RopeGeom g, RopeView x, RopeView y, const int32_t* __restrict__ pos, const float2* __restrict__ table,
              float sign, unsigned int* status) {
  constexpr int LPR = D / 8;
  const Lane l = lane_of<LPR>(g, blockIdx.x);
  const int vec = threadIdx.x & (LPR - 1);
  const bf16* xp = x.p + l.b * x.sb + l.n * x.sn + vec * 8;
  bf16* yp = y.p + l.b * y.sb + l.n * y.sn + vec * 8;
  uint4 next[U];
  load_rows<U>(next, xp, x.sh, l.h0, l);   // on their way while the table is read
  const int partner = HALF ? partner_lane<LPR>(g, threadIdx.x & 31, vec) : 0;
  Turn<HALF> t;
  make_turn<HALF>(t, g, table, load_pos(g, pos, pos_row(g, l), l.active), l.active, vec, partner, sign, status);
  for (int h = l.h0; h < l.h1; h += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = next[u];
    load_rows<U>(next, xp, x.sh, h + U, l);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float f[8], fp[8];
      unpack(v[u], f);
      if constexpr (HALF) unpack(shfl(v[u], partner), fp);
      turn<HALF>(t, f, fp);
      if (l.active && h + u < l.h1) store_row(yp + (h + u) * y.sh, pack(f));
    }
  }
}

// ---------------------------------------------------------------- norm + rotation, forward
template <int D, bool HALF>
DSV_DEVICE uint4 norm_turn(const uint4& v, const uint4& w, const uint4& wp, const Turn<HALF>& t, int partner,
                           float eps) {
  constexpr int LPR = D / 8;
  float f[8], fw[8], fp[8];
  unpack(v, f);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
  const float rstd = rsqrtf(fmaf(row_sum<LPR>(ss), 1.f / D, eps));
  unpack(w, fw);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * fw[e];
  if constexpr (HALF) {
    unpack(shfl(v, partner), fp);
    unpack(wp, fw);
#pragma unroll
    for (int e = 0; e < 8; ++e) fp[e] = fp[e] * rstd * fw[e];
  }
  turn<HALF>(t, f, fp);
  return pack(f);
}

DSV_DEVICE uint4 load_weight(const bf16* w, int vec) {
  // without a weight: ones (bf16 1.0 = 0x3f80)
  return w ? __ldg(reinterpret_cast<const uint4*>(w) + vec)
           : make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
}

// Pairs in halves need 143 registers: held to 128 a fourth CTA fits on the SM (mid clip 285 -> 252 us; the
// interleaved form has 96, and any bound there costs it: 247 -> 268 us).
template <int D, bool HALF, int U>
__global__ void __launch_bounds__(kThreads, HALF ? 4 : 0)
qk_norm_rope_fwd_kernel(RopeGeom g, RopeView q, RopeView k, RopeView v, RopeView qo, RopeView ko, RopeView vo,
                        const bf16* __restrict__ wq, const bf16* __restrict__ wk, const int32_t* __restrict__ pos,
                        const float2* __restrict__ table, float eps, unsigned int* status) {
  constexpr int LPR = D / 8;
  const Lane l = lane_of<LPR>(g, blockIdx.x);
  const int vec = threadIdx.x & (LPR - 1);
  const bool has_v = v.p != nullptr;
  const bf16* qp = q.p + l.b * q.sb + l.n * q.sn + vec * 8;
  const bf16* kp = k.p + l.b * k.sb + l.n * k.sn + vec * 8;
  const bf16* vp = has_v ? v.p + l.b * v.sb + l.n * v.sn + vec * 8 : nullptr;
  bf16* qop = qo.p + l.b * qo.sb + l.n * qo.sn + vec * 8;
  bf16* kop = ko.p + l.b * ko.sb + l.n * ko.sn + vec * 8;
  bf16* vop = has_v ? vo.p + l.b * vo.sb + l.n * vo.sn + vec * 8 : nullptr;
  uint4 na[U], nb[U], nc[U];
  auto fetch = [&](int h) {
    load_rows<U>(na, qp, q.sh, h, l);
    load_rows<U>(nb, kp, k.sh, h, l);
    if (has_v) load_rows<U>(nc, vp, v.sh, h, l);
  };
  fetch(l.h0);   // on their way while the table and the weights are read
  const int partner = HALF ? partner_lane<LPR>(g, threadIdx.x & 31, vec) : 0;
  Turn<HALF> t;
  make_turn<HALF>(t, g, table, load_pos(g, pos, pos_row(g, l), l.active), l.active, vec, partner, 1.f, status);
  const uint4 fq = load_weight(wq, vec), fk = load_weight(wk, vec);
  uint4 fqp = fq, fkp = fk;
  if constexpr (HALF) {
    fqp = shfl(fq, partner);
    fkp = shfl(fk, partner);
  }
  for (int h = l.h0; h < l.h1; h += U) {
    uint4 a[U], b[U], c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      a[u] = na[u];
      b[u] = nb[u];
      c[u] = nc[u];
    }
    fetch(h + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = l.active && h + u < l.h1;
      const uint4 ra = norm_turn<D, HALF>(a[u], fq, fqp, t, partner, eps);
      const uint4 rb = norm_turn<D, HALF>(b[u], fk, fkp, t, partner, eps);
      if (on) {
        store_row(qop + (h + u) * qo.sh, ra);
        store_row(kop + (h + u) * ko.sh, rb);
        if (has_v) store_row(vop + (h + u) * vo.sh, c[u]);
      }
    }
  }
}

// ---------------------------------------------------------------- norm + rotation, backward
// dx of one vector; its part of the weight's gradient is added to dw.
template <int D, bool HALF>
DSV_DEVICE uint4 norm_turn_back(const uint4& dy, const uint4& x, const uint4& w, const Turn<HALF>& t, int partner,
                                float eps, bool on, float (&dw)[8]) {
  constexpr int LPR = D / 8;
  float gr[8], f[8], fw[8], fp[8];
  unpack(dy, gr);
  if constexpr (HALF) unpack(shfl(dy, partner), fp);
  turn<HALF>(t, gr, fp);
  unpack(x, f);
  unpack(w, fw);
  float ss = 0.f, m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ss = fmaf(f[e], f[e], ss);
    m = fmaf(gr[e] * fw[e], f[e], m);
  }
  ss = row_sum<LPR>(ss);
  m = row_sum<LPR>(m);
  const float rstd = rsqrtf(fmaf(ss, 1.f / D, eps));
  m *= rstd * (1.f / D);                       // mean(g w xhat)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float xhat = f[e] * rstd;
    if (on) dw[e] = fmaf(gr[e], xhat, dw[e]);   // a row of zeros past the heads has no finite xhat at eps = 0
    f[e] = rstd * fmaf(-xhat, m, gr[e] * fw[e]);
  }
  return pack(f);
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, kBackCtas)
qk_norm_rope_bwd_kernel(RopeGeom g, RopeView dqo, RopeView dko, RopeView dvo, RopeView q, RopeView k, RopeView dq,
                        RopeView dk, RopeView dv, const bf16* __restrict__ wq, const bf16* __restrict__ wk,
                        const int32_t* __restrict__ pos, const float2* __restrict__ table, float eps,
                        float* __restrict__ partial, unsigned int* status) {
  constexpr int LPR = D / 8, kTok = kThreads / LPR;
  // the column sums may be scheduled once every CTA of this grid has started; they wait for its end
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __shared__ __align__(16) float red[kTok][2 * D];
  const int vec = threadIdx.x & (LPR - 1), grp = threadIdx.x / LPR;
  const uint4 fq = load_weight(wq, vec), fk = load_weight(wk, vec);
  const int partner = HALF ? partner_lane<LPR>(g, threadIdx.x & 31, vec) : 0;
  const bool has_v = dvo.p != nullptr;
  // the thread's own sums so far, in its own places (16 registers more would cost spills)
  float4 *sum_q = reinterpret_cast<float4*>(&red[grp][vec * 8]), *sum_k = reinterpret_cast<float4*>(&red[grp][D + vec * 8]);
  sum_q[0] = sum_q[1] = sum_k[0] = sum_k[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [](float4* to, const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 s = to[i];
      s.x += v[4 * i], s.y += v[4 * i + 1], s.z += v[4 * i + 2], s.w += v[4 * i + 3];
      to[i] = s;
    }
  };
  auto at = [&](const RopeView& r, const Lane& l) { return r.p + l.b * r.sb + l.n * r.sn + vec * 8; };
  // A step is a head of all three tensors, its loads one step ahead through everything the CTA does (n..: the rows on
  // their way).  Two heads of one tensor to a step keep as many rows in flight and took 349 us where this takes
  // 341 (mid clip, 16 heads), 766 where it takes 729 (long clip, 4 heads).
  uint4 nqy, nqx, nky, nkx, nv;
  auto fetch = [&](const Lane& l, int h) {
    const bool on = l.active;
    auto row = [&](const RopeView& r) { return on ? load_row(at(r, l) + h * r.sh) : make_uint4(0, 0, 0, 0); };
    nqy = row(dqo);
    nqx = row(q);
    nky = row(dko);
    nkx = row(k);
    if (has_v) nv = row(dvo);
  };
  Lane l = lane_of<LPR>(g, blockIdx.x);
  fetch(l, l.h0);
  Pos ahead = load_pos(g, pos, pos_row(g, l), l.active);
  for (int64_t unit = blockIdx.x; unit < g.units; unit += gridDim.x) {
    Turn<HALF> t;
    make_turn<HALF>(t, g, table, ahead, l.active, vec, partner, -1.f, status);
    Lane nl = l;
    nl.active = false;
    if (unit + gridDim.x < g.units) {
      nl = lane_of<LPR>(g, unit + gridDim.x);
      ahead = load_pos(g, pos, pos_row(g, nl), nl.active);
    }
    // a token's heads are summed first and its sum then added: two short chains of fp32 additions instead of one as
    // long as the clip
    float tq[8], tk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) tq[e] = tk[e] = 0.f;
    for (int h = l.h0; h < l.h1; ++h) {
      const uint4 qy = nqy, qx = nqx, ky = nky, kx = nkx, v = nv;
      if (h + 1 < l.h1) fetch(l, h + 1);
      else fetch(nl, nl.h0);
      const uint4 rq = norm_turn_back<D, HALF>(qy, qx, fq, t, partner, eps, l.active, tq);
      if (l.active) {
        store_row(at(dq, l) + h * dq.sh, rq);
        if (has_v) store_row(at(dv, l) + h * dv.sh, v);
      }
      const uint4 rk = norm_turn_back<D, HALF>(ky, kx, fk, t, partner, eps, l.active, tk);
      if (l.active) store_row(at(dk, l) + h * dk.sh, rk);
    }
    add(sum_q, tq);
    add(sum_k, tk);
    l = nl;
  }
  if (!partial) return;   // no weights: nothing to sum
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
    for (int r = 0; r < kTok; ++r) s += red[r][i];
    partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
  }
}

// dw[i] = sum over the CTAs of partial[c][i], in a fixed order: 32 columns a CTA, 32 warps take
// every 32nd row each, then the 32 sums in warp order.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
qk_norm_colsum_kernel(const float* partial, int rows, int D, float* __restrict__ dwq,
                      float* __restrict__ dwk) {
  __shared__ float red[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float s0 = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += kSumWarps) s0 += __ldcg(partial + static_cast<int64_t>(r) * 2 * D + col);
  red[warp][lane] = s0;
  __syncthreads();
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) s += red[w][lane];
    float* out = col < D ? dwq : dwk;
    if (out) out[col < D ? col : col - D] = s;
  }
}

// ---------------------------------------------------------------- the table
// (cos, sin) of angle p theta^(-2i / r) in double, rounded once: far positions keep their phase.
__global__ void __launch_bounds__(kThreads)
rope3d_table_kernel(RopeGeom g, double th0, double th1, double th2, int64_t total, float2* __restrict__ table) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (e >= total) return;
  const int a = e >= g.table_off[2] ? 2 : e >= g.table_off[1] ? 1 : 0;
  const double theta = a == 0 ? th0 : a == 1 ? th1 : th2;
  const int np = g.axis_pairs[a];
  const int64_t local = e - g.table_off[a];
  const int64_t p = local / np;
  const int i = static_cast<int>(local % np);
  const double ang = static_cast<double>(p) * pow(theta, -static_cast<double>(i) / np);
  double s, c;
  sincos(ang, &s, &c);
  table[e] = make_float2(static_cast<float>(c), static_cast<float>(s));
}

constexpr int64_t kBackAtOnce = 152 * kBackCtas;   // persistent CTAs of the backward

void cut_heads(RopeGeom& g, int64_t tiles, int64_t chunks) {
  g.heads_per_chunk = (g.H + chunks - 1) / chunks;
  g.chunks = (g.H + g.heads_per_chunk - 1) / g.heads_per_chunk;
  g.units = tiles * g.chunks;
}

}  // namespace

// How the work is cut into units of a CTA: a tile of tokens and a chunk of their heads.
// Forward: a CTA walks all heads of its tokens unless that leaves the card's 152 SMs short of CTAs.
// Backward: its CTAs take units in turns, so the cut with the least turns times the length of one (a step for each
// head, and kBackSetup steps' worth of positions and table) is taken.
RopeGeom rope_plan(const RopeGeom& in, int d, bool backward) {
  RopeGeom g = in;
  const int64_t tok = kThreads / (d / 8);
  g.tiles_per_b = (g.N + tok - 1) / tok;
  const int64_t tiles = g.B * g.tiles_per_b;
  if (!backward) {
    const int64_t chunks = (kRopeWantCtas + tiles - 1) / tiles;
    cut_heads(g, tiles, chunks < g.H ? chunks : g.H);
    return g;
  }
  int64_t best = 1;
  double least = 0;
  for (int64_t chunks = 1; chunks <= g.H && chunks <= 64; ++chunks) {
    cut_heads(g, tiles, chunks);
    const double turns = static_cast<double>((g.units + kBackAtOnce - 1) / kBackAtOnce);
    const double cost = turns * (static_cast<double>(g.heads_per_chunk) + kBackSetup);
    if (chunks == 1 || cost < least) {
      least = cost;
      best = chunks;
    }
  }
  cut_heads(g, tiles, best);
  return g;
}

// Persistent CTAs of the backward (rows of its partial sums).
int64_t rope_bwd_ctas(const RopeGeom& g) { return g.units < kBackAtOnce ? g.units : kBackAtOnce; }

cudaError_t launch_rope3d_table(const RopeGeom& g, const double (&theta)[3], float* table, cudaStream_t stream) {
  int64_t total = 0;
  for (int a = 0; a < 3; ++a) total += g.len[a] * g.axis_pairs[a];
  if (total == 0) return cudaSuccess;
  ProfScope prof("rope3d_table", stream);
  rope3d_table_kernel<<<static_cast<unsigned>((total + kThreads - 1) / kThreads), kThreads, 0, stream>>>(
      g, theta[0], theta[1], theta[2], total, reinterpret_cast<float2*>(table));
  return cudaGetLastError();
}

template <class F>
void pick(const RopeParams& p, F&& go) {
  auto dim = [&](auto half) {
    p.d == 128 ? go(std::integral_constant<int, 128>(), half) : go(std::integral_constant<int, 64>(), half);
  };
  p.half ? dim(std::true_type()) : dim(std::false_type());
}

// The forward and rope3d load U = 2 heads of each tensor ahead.  Where a group has only one or two heads to walk, half
// of that would be loads of nothing or registers that keep other CTAs out: U = 1.  Measured with U = 2 / U = 1
// (d = 64, 524,288 tokens): norm and rotation of 1 head 167 / 117 us, 2 heads (262,144 tokens) 99 / 82 us,
// 8 heads (65,536 tokens) 71 / 74 us; rope3d alone 66 / 60, 40 / 39, 29 / 33.  Persistent CTAs as in the backward cost the
// forward 8 to 10 % (mid clip 241 -> 266 us): it has registers for more CTAs than they take.
template <class F>
void pick_rows(const RopeParams& p, const RopeGeom& g, F&& go) {
  pick(p, [&](auto d, auto half) {
    g.heads_per_chunk <= 2 ? go(d, half, std::integral_constant<int, 1>()) : go(d, half, std::integral_constant<int, 2>());
  });
}

cudaError_t launch_rope3d(const RopeParams& p, cudaStream_t stream) {
  const RopeGeom g = rope_plan(p.g, p.d, false);
  const float2* table = reinterpret_cast<const float2*>(p.table);
  ProfScope prof(p.backward ? "rope3d_bwd" : "rope3d_fwd", stream);
  pick_rows(p, g, [&](auto d, auto half, auto u) {
    rope3d_kernel<decltype(d)::value, decltype(half)::value, decltype(u)::value>
        <<<static_cast<unsigned>(g.units), kThreads, 0, stream>>>(g, p.q, p.qo, p.pos, table, p.backward ? -1.f : 1.f,
                                                                  p.status);
  });
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope_fwd(const RopeParams& p, cudaStream_t stream) {
  const RopeGeom g = rope_plan(p.g, p.d, false);
  const float2* table = reinterpret_cast<const float2*>(p.table);
  ProfScope prof("qk_norm_rope_fwd", stream);
  pick_rows(p, g, [&](auto d, auto half, auto u) {
    qk_norm_rope_fwd_kernel<decltype(d)::value, decltype(half)::value, decltype(u)::value>
        <<<static_cast<unsigned>(g.units), kThreads, 0, stream>>>(g, p.q, p.k, p.v, p.qo, p.ko, p.vo, p.wq, p.wk,
                                                                  p.pos, table, p.eps, p.status);
  });
  return cudaGetLastError();
}

cudaError_t launch_qk_norm_rope_bwd(const RopeParams& p, cudaStream_t stream) {
  const RopeGeom g = rope_plan(p.g, p.d, true);
  const float2* table = reinterpret_cast<const float2*>(p.table);
  const int64_t ctas = rope_bwd_ctas(g);
  float* partial = p.dwq || p.dwk ? p.partial : nullptr;
  {
    ProfScope prof("qk_norm_rope_bwd", stream);
    pick(p, [&](auto d, auto half) {
      qk_norm_rope_bwd_kernel<decltype(d)::value, decltype(half)::value>
          <<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(g, p.qo, p.ko, p.vo, p.q, p.k, p.dq, p.dk, p.dv, p.wq,
                                                                 p.wk, p.pos, table, p.eps, partial, p.status);
    });
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!partial) return cudaSuccess;
  ProfScope prof("qk_norm_colsum", stream);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.d / 32));
  cfg.blockDim = dim3(32 * kSumWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_norm_colsum_kernel, static_cast<const float*>(partial), static_cast<int>(ctas),
                            p.d, p.dwq, p.dwk);
}

}  // namespace dsv
