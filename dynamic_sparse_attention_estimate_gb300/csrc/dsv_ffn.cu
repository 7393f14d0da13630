// Gated feed-forward of a DiT block: h = act(x Wg^T) * (x Wu^T), forward and backward, on the tcgen05
// tensor cores.
//
// One persistent GEMM kernel in five modes, all bf16 operands with fp32 accumulators in tensor memory:
//   kGate      g, u = x Wg^T, x Wu^T;  h = act(g) u                      (K = D, both K-major)
//   kGateGrad  the same products again; dg = dh u act'(g), du = dh act(g)   (nothing is kept of the forward)
//   kDx        dx = dg Wg + du Wu                                         (K = F twice; W is MN-major)
//   kDw        dWg = dg^T x, dWu = du^T x                                  (K = M; both MN-major)
//   kBack      kDx and kDw in one launch, where each alone leaves many pairs idle
// An accumulator tile is 256 rows by 256 columns, held by a pair of CTAs (cta_group::2: each holds 128 rows
// of A and of the result, and half of B); in the gated modes its columns are 128 of g and the 128 of u
// they meet in the epilogue, so g and u never leave the SM in kGate.  dg and du are rounded to bf16
// between the backward's kernels: the tensor cores take them as operands of that type (at most 2^-8 of
// each value, as every activation between layers; a few tokens keep them in fp32, below).
//
// Roles (384 threads a CTA): one thread of warp 0 issues the TMA loads of A and one of warp 2 those of B into a
// ring of 64-wide stages; one thread of warp 1 of the pair's first CTA issues the MMAs, into one of two
// accumulators (2 x 256 of the 512 TMEM columns); warps 4-11 empty the other one: two warpgroups, each on half
// of the columns, through swizzled staging tiles that TMA stores write (rows and columns past the matrices
// are clipped there, and zero-filled by the loads).  Every wait is bounded.
//
// What bounds it (GB300, M x D x F): the tensor cores.  65,536 x 2048 x 5632 forward 1.48 ms = 2.05 PFLOP/s from a cool start
// (a library's plain product of that size 1.51 ms), 520 to 540 of the ideal 512 cycles to a
// stage; run for a second the card's 1.4 kW limit holds both back (1.71 ms here, 1.69 ms there).
// 16,384-token backward 1.21 to 1.29 ms = 1.76 to 1.88 PFLOP/s, 1.39 at the limit: its three products pass 0.6 GB of dh, dg
// and du and end in partial rounds of tiles.  Few tiles: 5.5 us a launch and 0.28 us a stage.  Short D is bound by the epilogue and, where rows do not start on 128 bytes,
// by the loads: 34,070 x 360 x 3312 forward 155 us against 85.  A pair beats single CTAs of 128 x 256 tiles (1.74 ms)
// for its half B to a CTA and six stages instead of four; pairs of pairs that shared B by multicast ran at
// the same cycles to a stage on 144 of the 152 SMs (1.69 ms).
#include <cuda.h>

#include <type_traits>

#include "dsv_block.h"
#include "dsv_common.cuh"
#include "dsv_internal.h"
#include "dsv_tc.cuh"

namespace dsv {
namespace {

constexpr int kThreads = 384;
constexpr int kBK = 64;                    // K elements of a stage (128 bytes)
constexpr uint32_t kWaitLimit = 1u << 20;   // polls, each suspended in the hardware for up to kWaitNs
// Without the hint the waiting warps poll, and pay for it in watts: at 16,384 x 2048 x 5632 a second of
// forward calls at the card's power limit runs at 1.68 PFLOP/s without and 1.73 with it.
constexpr uint32_t kWaitNs = 2000;
constexpr int kTile = 128 * 128;           // bytes of a [128 rows][64] or two [64 rows][64] bf16 tiles
constexpr int kPart = 128 * 64;            // bytes of a [128 rows][32] bf16 tile: what one TMA store writes

enum Mode { kGate = 0, kGateGrad = 1, kDx = 2, kDw = 3, kBack = 4 };

struct Maps {
  CUtensorMap a0, a1;      // A: x; dg, du for dx
  CUtensorMap t0, t1;      // dg, du for the weights' gradients
  CUtensorMap b0, b1, b2;  // B: Wg, Wu; x for the weights' gradients
  CUtensorMap c0, c1, c2;  // results: h; dg, du; dx, dWg, dWu
};

// One product and how it is cut.
struct Product {
  bool dw;          // the weights' gradients
  int64_t m_tiles, n_tiles, tiles;
  int64_t units;    // tiles, or tiles times the parts of K they are split into (unit = part * tiles + tile)
  int kb_half;      // dx: k blocks of one of its two pairs of operands
  int kb;           // k blocks of a tile
  int kb_part;      // of a unit
  float* partial;   // split: [unit][256][256] sums
  int64_t rows, cols;   // of the result (the weights': of one of the two)
  int64_t half_tiles;   // the weights': m tiles of the first result
};
struct Shape {
  Product p[2];     // kBack: dx and the weights' gradients, the one with longer units first; else p[0]
  int64_t skip;     // see Walk
  const bf16* dh;   // kGateGrad
  int group;        // m tiles that share their n tiles' operands in L2
  int act;
};

// The units of one pair of CTAs of P: they go round the pairs.
template <bool TWO>
struct Walk {
  static constexpr int cls = 0;
  int64_t n, pairs, t;
  DSV_DEVICE Walk(const Shape& sh) {
    n = sh.p[0].units;
    pairs = gridDim.x / 2;
    t = blockIdx.x / 2;
  }
  DSV_DEVICE bool more() const { return t < n; }
  DSV_DEVICE void next() { t += pairs; }
};
// Of two products (cls: which): those of p[0] go round the pairs; after its last round, L pairs have had
// one less, and take `skip` units of p[1] each (unit i of these: pair P - L + i % L) before the rest of p[1] goes round all of
// them, the L first.
template <>
struct Walk<true> {
  int64_t n0, n1, pairs, pair, skip, t;
  int64_t short_from;   // P - L (0: every pair had the same number)
  int64_t extra;        // units of `skip` still to come
  int cls;
  DSV_DEVICE Walk(const Shape& sh) {
    n0 = sh.p[0].units;
    n1 = sh.p[1].units;
    pairs = gridDim.x / 2;
    t = pair = blockIdx.x / 2;
    skip = sh.skip;
    short_from = n0 % pairs;
    cls = 0;
    extra = 0;
    if (t >= n0) second();
  }
  DSV_DEVICE void second() {
    cls = 1;
    extra = short_from && pair >= short_from ? skip : 0;
    t = extra ? pair - short_from : rest();
  }
  DSV_DEVICE int64_t rest() const {
    const int64_t i = pair - short_from;
    return (short_from ? skip * (pairs - short_from) : 0) + (i < 0 ? i + pairs : i);
  }
  DSV_DEVICE bool more() const { return t < (cls ? n1 : n0); }
  DSV_DEVICE void next() {
    if (cls == 0) {
      t += pairs;
      if (t >= n0) second();
    } else if (extra) {
      t = --extra ? t + pairs - short_from : rest();
    } else {
      t += pairs;
    }
  }
};

template <int MODE>
struct Cfg {
  static constexpr int kStageA = kTile;
  static constexpr int kStageB = kTile;
  static constexpr int kStage = kStageA + kStageB;
  static constexpr int kResults = MODE == kGateGrad ? 2 : 1;
  static constexpr int kOut = 2 * 2 * kResults * kPart;   // staging: two warpgroups, two parts of each result
  static constexpr int kStages = (227 * 1024 - 2048 - kOut) / kStage;
  static constexpr int kSmem = kStages * kStage + kOut + 1024;
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int fail;
};

DSV_DEVICE bool wait_bar(uint32_t bar, uint32_t parity, volatile int* fail) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kWaitNs)
        : "memory");
    if (ok) return true;
    if ((i & 255) == 255 && *fail) return false;   // (a look at it in every round costs the MMAs' rate)
  }
  return false;
}

// A place in a ring of N stages and the parity of its round (kept as two small numbers: a division of a
// running count would sit between two stages' MMAs).
template <int N>
struct Ring {
  uint32_t s = 0, round = 0;
  DSV_DEVICE void next() {
    if (++s == N) {
      s = 0;
      round ^= 1;
    }
  }
};

DSV_DEVICE uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
DSV_DEVICE void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of a matrix into this CTA's shared memory, counted on a barrier of either CTA of the pair.
DSV_DEVICE void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}
DSV_DEVICE void tma_store(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(map), "r"(x),
               "r"(y), "r"(src)
               : "memory");
}
DSV_DEVICE void stores_commit() { asm volatile("cp.async.bulk.commit_group;\n" ::: "memory"); }
// Waits until all groups of stores but the last one have read their tiles.
DSV_DEVICE void stores_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;\n" ::: "memory"); }
DSV_DEVICE void store_done() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }
DSV_DEVICE void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory"); }
// A barrier whose threads agree: true where all of them came with true.
DSV_DEVICE bool bar_all(int id, int n, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %3, 0;\n bar.red.and.pred q, %1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------- pairs of CTAs (cta_group::2)
DSV_DEVICE uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
DSV_DEVICE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;\n" ::: "memory");
}
// (What this arrival orders are reads of tensor memory, which the tcgen05 fences around it cover.  A release at
// cluster scope would also wait for the thread's stores: 34,070 x 360 x 3312 forward 175 us with it, 155 without.)
DSV_DEVICE void arrive_cluster(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_bar) : "memory");
}
DSV_DEVICE void tmem_alloc_pair(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst), "r"(cols));
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::);
}
DSV_DEVICE void tmem_dealloc_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(addr), "r"(cols));
}
DSV_DEVICE void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// Arrive on this barrier of both CTAs once every MMA issued so far has completed.
DSV_DEVICE void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Activation and its derivative.  Both activations are g times a logistic function:
//   silu: s(g);  gelu (tanh form): s(2 c (g + 0.044715 g^3)), c = sqrt(2 / pi).
DSV_DEVICE float logistic(float z) { return __fdividef(1.f, 1.f + fast_exp2(-kLog2e * z)); }
constexpr float kGelu2C = 1.5957691216057308f;   // 2 sqrt(2 / pi)
DSV_DEVICE float act_value(float g, int act) {
  const float z = act == 0 ? g : kGelu2C * fmaf(0.044715f * g * g, g, g);
  return g * logistic(z);
}
DSV_DEVICE void act_both(float g, int act, float& a, float& slope) {
  const float z = act == 0 ? g : kGelu2C * fmaf(0.044715f * g * g, g, g);
  // (held finite: beyond |g| = 1.8e19 g^2 is not, and the factor it meets below is then 0, not small)
  const float dz = act == 0 ? 1.f : fminf(kGelu2C * fmaf(3.f * 0.044715f * g, g, 1.f), 1e30f);
  const float s = logistic(z);
  a = g * s;
  slope = fmaf(a * (1.f - s), dz, s);
}
// dg = dh act'(g) u, the slope (at most 1.13) first: dh u alone can pass fp32 where a slope of 0 makes dg 0.
DSV_DEVICE float grad_gate(float dh, float slope, float u) { return dh * slope * u; }

DSV_DEVICE void tile_of(const Product& pr, int64_t group, int64_t t, int64_t& m, int64_t& n) {
  const int64_t per = group * pr.n_tiles;
  const int64_t g = t / per, r = t % per;
  const int64_t left = pr.m_tiles - g * group;
  const int64_t gm = left < group ? left : group;
  m = g * group + r % gm;
  n = r / gm;
}

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
ffn_gemm_kernel(const __grid_constant__ Maps maps, Shape sh, unsigned int* status) {
  using C = Cfg<MODE>;
  constexpr bool kGated = MODE == kGate || MODE == kGateGrad, kTwo = MODE == kBack;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());              // of this CTA in its pair
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t ring = (raw + 1023u) & ~1023u;          // swizzled tiles need 1024-byte alignment
  const uint32_t out = ring + C::kStages * C::kStage;
  auto bar = [](uint64_t& b) { return smem_u32(&b); };

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::mbar_init(bar(bars.full[s]), 1);
      tc::mbar_init(bar(bars.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(bar(bars.acc_full[b]), 1);
      tc::mbar_init(bar(bars.acc_empty[b]), 16);
    }
    tc::mbar_init(bar(bars.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    bars.fail = 0;
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&bars.tmem), 512);
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTAs' barriers exist
  tc::tc_fence_after();
  // what follows in this call may start setting itself up; this kernel goes on when what came before is done
  asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;\n" ::: "memory");
  const uint32_t tmem = bars.tmem;
  volatile int* fail = &bars.fail;

  if (warp == 0 || warp == 2) {
    // ================================================================ TMA loads: one thread for A (warp 0), one for B
    if (lane == 0) {
      const bool for_a = warp == 0;
      const uint32_t empty0 = bar(bars.empty[0]), full0 = bar(bars.full[0]);
      const uint32_t lead0 = map_rank(full0, 0);   // the copies count on the first CTA's barriers, where the MMAs are issued
      Ring<C::kStages> at;
      int64_t issued = 0;   // stages
      bool ok = true;
      for (Walk<kTwo> w(sh); w.more() && ok; w.next()) {
        const Product& pr = sh.p[w.cls];
        const bool dw = MODE == kDw || (kTwo && pr.dw);
        int64_t m, n;
        tile_of(pr, sh.group, SPLIT ? w.t % pr.tiles : w.t, m, n);
        const bool second = dw && m >= pr.half_tiles;
        const int m0 = static_cast<int>((second ? m - pr.half_tiles : m) * 256) + rank * 128;
        // B: the pair's second CTA holds the tile's second 128 columns (in the gated modes those of u)
        const int n0 = static_cast<int>(n * (kGated ? 128 : 256)) + (kGated ? 0 : rank * 128);
        const int kb0 = SPLIT ? static_cast<int>(w.t / pr.tiles) * pr.kb_part : 0;
        const int kb1 = SPLIT && kb0 + pr.kb_part < pr.kb ? kb0 + pr.kb_part : pr.kb;
        const int kb_half = !kGated && !dw ? pr.kb_half : kb1;   // dx: from here on the second of its two products
        for (int kb = kb0; kb < kb1; ++kb, ++issued, at.next()) {
          // (a fresh barrier passes for the parity before its first round)
          if (!wait_bar(empty0 + 8 * at.s, at.round ^ 1, fail)) {
            ok = false;
            break;
          }
          const uint32_t full = lead0 + 8 * at.s;
          const uint32_t a = ring + at.s * C::kStage, b = a + C::kStageA;
          const bool late = kb >= kb_half;
          const int k0 = (late ? kb - kb_half : kb) * kBK;
          if (for_a) {
            if (rank == 0) expect_tx(full0 + 8 * at.s, 2 * C::kStage);
            if (dw) {
              const CUtensorMap* map = second ? &maps.t1 : &maps.t0;
              tma_load_pair(a, map, m0, k0, full);
              tma_load_pair(a + kTile / 2, map, m0 + 64, k0, full);
            } else {
              tma_load_pair(a, late ? &maps.a1 : &maps.a0, k0, m0, full);
            }
          } else {
            if constexpr (kGated) {
              tma_load_pair(b, rank == 1 ? &maps.b1 : &maps.b0, k0, n0, full);
            } else {
              const CUtensorMap* map = dw ? &maps.b2 : late ? &maps.b1 : &maps.b0;
              tma_load_pair(b, map, n0, k0, full);
              tma_load_pair(b + kTile / 2, map, n0 + 64, k0, full);
            }
          }
        }
      }
      // the stages still out come back before this CTA may leave: the MMAs arrive on them
      const int64_t out_first = issued > C::kStages ? issued - C::kStages : 0;
      Ring<C::kStages> last;
      last.s = static_cast<uint32_t>(out_first % C::kStages);
      last.round = static_cast<uint32_t>((out_first / C::kStages) & 1);
      Ring<C::kStages> load = last;
      for (int64_t c = out_first; c < issued && ok; ++c, last.next()) ok = wait_bar(empty0 + 8 * last.s, last.round, fail);
      if (!ok) {
        *fail = 1;
        // the copies in flight land before this CTA's shared memory can go away (again bounded)
        for (int64_t c = out_first; c < issued && rank == 0; ++c, load.next())
          tc::mbar_wait(full0 + 8 * load.s, load.round, kWaitLimit);
      }
    }
  } else if (warp == 1) {
    // ================================================================ MMA issue (one thread of the pair)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t id_k = tc::idesc_bf16(256, 256, 0, !kGated), id_mn = tc::idesc_bf16(256, 256, 1, 1);
      static_assert((id_k | id_mn) >> 29 == 0 && ((id_k >> 24) & 31) == 16 && ((id_mn >> 24) & 31) == 16 &&
                        ((id_k >> 17) & 63) == 32 && ((id_mn >> 17) & 63) == 32, "M and N in their fields");
      // descriptors of the first stage; a stage, and 16 elements of K in it, are so many 16-byte units on
      // (K-major: 16 elements are 32 bytes; MN-major: two 8-row groups of 1024 bytes, column blocks of 64
      // elements 8 KB apart)
      const uint64_t a_k = tc::smem_desc(ring, 16, 1024), a_mn = tc::smem_desc(ring, kTile / 2, 1024);
      const uint64_t b0 = kGated ? tc::smem_desc(ring + C::kStageA, 16, 1024) : tc::smem_desc(ring + C::kStageA, kTile / 2, 1024);
      constexpr uint32_t kStepK = 32 >> 4, kStepMn = 2048 >> 4, kStepB = kGated ? kStepK : kStepMn;
      Ring<C::kStages> at;
      int64_t tile = 0;
      bool ok = true;
      for (Walk<kTwo> w(sh); w.more() && ok; w.next(), ++tile) {
        const Product& pr = sh.p[w.cls];
        const bool dw = MODE == kDw || (kTwo && pr.dw);
        const uint32_t id = dw ? id_mn : id_k, step_a = dw ? kStepMn : kStepK;
        const uint64_t a0 = dw ? a_mn : a_k;
        const int buf = static_cast<int>(tile & 1);
        if (tile >= 2) ok = wait_bar(bar(bars.acc_empty[buf]), static_cast<uint32_t>(((tile >> 1) - 1) & 1), fail);
        tc::tc_fence_after();
        const uint32_t acc = tmem + buf * 256;
        const int kb0 = SPLIT ? static_cast<int>(w.t / pr.tiles) * pr.kb_part : 0;
        const int kb1 = SPLIT && kb0 + pr.kb_part < pr.kb ? kb0 + pr.kb_part : pr.kb;
        for (int kb = kb0; kb < kb1 && ok; ++kb, at.next()) {
          const uint32_t s = at.s;
          ok = wait_bar(bar(bars.full[s]), at.round, fail);
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t da = a0 + s * (C::kStage >> 4), db = b0 + s * (C::kStage >> 4);
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j) mma_pair(acc, da + j * step_a, db + j * kStepB, id, kb > kb0 || j > 0 ? 1u : 0u);
          commit_pair(bar(bars.empty[s]));
        }
        if (ok) commit_pair(bar(bars.acc_full[buf]));
      }
      if (!ok) {   // what was issued ends before the accumulators are given back (again bounded)
        *fail = 1;
        commit_pair(bar(bars.drain));
        tc::mbar_wait(bar(bars.drain), 0, kWaitLimit);
      }
    }
  } else if (warp >= 4) {
    // ================================================================ epilogue
    const int wg = (warp - 4) >> 2;                       // columns [64 wg, ..) of g and u, or [128 wg, ..)
    const int row = (warp & 3) * 32 + lane;               // of the tile (TMEM lane)
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool elect = (tid & 127) == 0;
    const uint32_t stage = out + wg * (C::kOut / 2);
    // 16 columns from c (0 or 16) of this row into a [128 rows][32] tile, 64-byte rows, swizzled: 16-byte chunk k of
    // row r sits at chunk k ^ (r / 2 % 4), so the 8 rows of a quarter warp fill all banks
    auto put = [&](uint32_t tile, int c, const uint32_t (&w)[8]) {
      const uint32_t base = tile + row * 64, turn = (row >> 1) & 3;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(base + (((c / 8 + q) ^ turn) << 4)), "r"(w[4 * q]),
                     "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3]));
    };
    auto release_acc = [&](int buf) {   // to the thread that issues the MMAs
      arrive_cluster(map_rank(bar(bars.acc_empty[buf]), 0));
    };
    int64_t tile = 0;
    bool ok = true;
    for (Walk<kTwo> w(sh); w.more() && ok; w.next(), ++tile) {
      const Product& pr = sh.p[w.cls];
      int64_t m, n;
      tile_of(pr, sh.group, SPLIT ? w.t % pr.tiles : w.t, m, n);
      const CUtensorMap* c_map = &maps.c0;
      if (MODE == kDw || (kTwo && pr.dw)) {
        c_map = m >= pr.half_tiles ? &maps.c2 : &maps.c1;
        if (m >= pr.half_tiles) m -= pr.half_tiles;
      }
      const int m0 = static_cast<int>(m * 256) + rank * 128;
      const int n0 = static_cast<int>(n * (kGated ? 128 : 256) + wg * (kGated ? 64 : 128));
      const int buf = static_cast<int>(tile & 1);
      // this row's 64 values of dh, on their way while the products end (through a TMA load into the staging tile, which
      // has to be free first, 16,384 x 2048 x 5632 took 462 us instead of 445)
      uint4 dh[MODE == kGateGrad && !SPLIT ? 8 : 1];
      if constexpr (MODE == kGateGrad && !SPLIT) {
        const bool in = m0 + row < pr.rows;
        const bf16* p = sh.dh + (m0 + row) * pr.cols + n0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dh[i] = in && n0 + 8 * i < pr.cols ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
      }
      ok = wait_bar(bar(bars.acc_full[buf]), static_cast<uint32_t>((tile >> 1) & 1), fail);
      ok = bar_all(1 + wg, 128, ok);                      // the warpgroup goes on together, or not at all
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + lane_base + buf * 256;
      if (SPLIT && (!kTwo || pr.partial)) {
        // a part of K: its sums as they are, joined with the others' by ffn_join_kernel (rows past the result's stay out)
        const bool in = m0 + row < pr.rows;
        float4* to = reinterpret_cast<float4*>(pr.partial + ((w.t * 256 + rank * 128 + row) * 256 + wg * 128));
#pragma unroll 1
        for (int c = 0; c < 128; c += 16) {
          uint32_t a[16];
          tc::tmem_ld16(acc + wg * 128 + c, a);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (in) to[c / 4 + i] = make_float4(__uint_as_float(a[4 * i]), __uint_as_float(a[4 * i + 1]),
                                        __uint_as_float(a[4 * i + 2]), __uint_as_float(a[4 * i + 3]));
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) release_acc(buf);
      } else if constexpr (!SPLIT || kTwo) {
        // 32 columns at a time through two staging tiles in turn: one is read by its store while the other fills (four
        // warpgroups with one tile each win where D is short, 16,384 x 128 x 1024 20 us instead of 23, and lose
        // elsewhere, 16,384 x 768 x 2048 67 instead of 64)
        constexpr int kParts = kGated ? 2 : 4;
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const uint32_t st0 = stage + (part & 1) * (C::kResults * kPart), st1 = st0 + kPart;
          if (elect) stores_read_but_one();               // (a group to a part, empty ones too)
          bar_sync(1 + wg, 128);
#pragma unroll
          for (int c = 0; c < 32; c += 16) {
            const int col = part * 32 + c;
            uint32_t w0[8];
            if constexpr (kGated) {
              uint32_t g[16], u[16], w1[8];
              tc::tmem_ld16(acc + wg * 64 + col, g);
              tc::tmem_ld16(acc + 128 + wg * 64 + col, u);
              tc::tmem_wait_ld();
              if constexpr (MODE == kGate) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  w0[i] = pack_bf16x2(act_value(__uint_as_float(g[2 * i]), sh.act) * __uint_as_float(u[2 * i]),
                                      act_value(__uint_as_float(g[2 * i + 1]), sh.act) * __uint_as_float(u[2 * i + 1]));
              } else {
                const uint4 d0 = dh[col / 8], d1 = dh[col / 8 + 1];
                const uint32_t d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  float dg[2], du[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    float a, slope;
                    act_both(__uint_as_float(g[2 * i + e]), sh.act, a, slope);
                    const float v = e ? bf16_hi(d[i]) : bf16_lo(d[i]);
                    dg[e] = grad_gate(v, slope, __uint_as_float(u[2 * i + e]));
                    du[e] = v * a;
                  }
                  w0[i] = pack_bf16x2(dg[0], dg[1]);
                  w1[i] = pack_bf16x2(du[0], du[1]);
                }
                put(st1, c, w1);
              }
            } else {
              uint32_t a[16];
              tc::tmem_ld16(acc + wg * 128 + col, a);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) w0[i] = pack_bf16x2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
            }
            put(st0, c, w0);
          }
          if (part == kParts - 1) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) release_acc(buf);
          }
          tc::fence_async_shared();
          bar_sync(1 + wg, 128);
          if (elect) {
            if (m0 < pr.rows && n0 + part * 32 < pr.cols) {
              tma_store(c_map, n0 + part * 32, m0, st0);
              if (MODE == kGateGrad) tma_store(&maps.c1, n0 + part * 32, m0, st1);
            }
            stores_commit();
          }
        }
      }
    }
    if (!ok) *fail = 1;
    if (elect) store_done();
  }
  tc::tc_fence_before();
  __syncthreads();
  cluster_sync();   // nothing of the cluster is in flight into this CTA any more
  if (tid == 0 && bars.fail) flag_status(status, kStatusTimeout);
  if (warp == 1) {
    tc::tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- parts of K joined
struct JoinOut {
  bf16 *c0, *c1, *c2;    // kGate h; kGateGrad dg, du; else dx, dWg, dWu
};

// 8 columns of a unit's row, summed over the parts in their order.
DSV_DEVICE void join8(const Product& pr, int64_t tile, int row, int col, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll 4
  for (int64_t u = tile; u < pr.units; u += pr.tiles) {
    const float4* p = reinterpret_cast<const float4*>(pr.partial + ((u * 256 + row) * 256 + col));
    const float4 a = __ldcg(p), b = __ldcg(p + 1);   // (of the kernel before: past L1)
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
    v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
  }
}
DSV_DEVICE void store8(bf16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// One thread: 8 columns of a row of a result (blockIdx.y: of dx, dWg, dWu those the launch is for).
template <int MODE>
__global__ void __launch_bounds__(256) ffn_join_kernel(Shape sh, JoinOut o) {
  constexpr bool kGated = MODE == kGate || MODE == kGateGrad;
  asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;\n" ::: "memory");
  const int result = blockIdx.y + (MODE == kDw);   // 0, or 1 and 2: the weights' gradients
  const Product& pr = sh.p[MODE == kBack && sh.p[0].dw != (result > 0)];
  if (!pr.partial) return;   // whole tiles: stored by the products' kernel
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t per_row = pr.cols / 8;
  if (i >= pr.rows * per_row) return;
  const int64_t r = i / per_row, col = i % per_row * 8;
  const int64_t m = r / 256 + (result > 1 ? pr.half_tiles : 0), n = col / (kGated ? 128 : 256);
  const int64_t g = m / sh.group, left = pr.m_tiles - g * sh.group, gm = left < sh.group ? left : sh.group;
  const int64_t tile = g * sh.group * pr.n_tiles + n * gm + (m - g * sh.group);   // tile_of's inverse
  const int row = static_cast<int>(r % 256), c = static_cast<int>(col % (kGated ? 128 : 256));
  const int64_t at = r * pr.cols + col;
  float v[8];
  join8(pr, tile, row, c, v);
  if constexpr (kGated) {
    float u[8];
    join8(pr, tile, row, 128 + c, u);
    if constexpr (MODE == kGate) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = act_value(v[e], sh.act) * u[e];
      store8(o.c0 + at, v);
    } else {
      const uint4 d4 = *reinterpret_cast<const uint4*>(sh.dh + at);
      const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float a, slope;
        act_both(v[e], sh.act, a, slope);
        const float dh = e & 1 ? bf16_hi(d[e >> 1]) : bf16_lo(d[e >> 1]);
        v[e] = grad_gate(dh, slope, u[e]);
        u[e] = dh * a;
      }
      store8(o.c0 + at, v);
      store8(o.c1 + at, u);
    }
  } else {
    store8((result == 0 ? o.c0 : result == 1 ? o.c1 : o.c2) + at, v);
  }
}

// ---------------------------------------------------------------- a few tokens
DSV_DEVICE uint64_t as_u64(float2 v) { return *reinterpret_cast<uint64_t*>(&v); }
DSV_DEVICE float2 fma2(float2 a, float2 b, float2 c) {   // two fp32 FMAs in one instruction
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return *reinterpret_cast<float2*>(&d);
}
DSV_DEVICE float2 pair_of(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

// For a few tokens the weights' bytes are the work: `warps` warps take a row of Wg and the same of Wu, read
// them once, 16 bytes a lane, and meet all tokens with them in registers.  One vector of each weight row is in flight to a
// lane: 4096 -> 8192 runs at 3.8 TB/s, 0.57 of the copy rate.
// GRAD: dg and du (fp32) from dh in place of h.
template <int R, bool GRAD>
__global__ void __launch_bounds__(256)
ffn_rows_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w_gate, const uint4* __restrict__ w_up,
                bf16* __restrict__ h, const bf16* __restrict__ dh, float* __restrict__ dg, float* __restrict__ du,
                int M, int64_t D, int64_t F, int warps, int act) {
  if (GRAD) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __shared__ float2 red[8][R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % warps;
  const int64_t f = static_cast<int64_t>(blockIdx.x) * (8 / warps) + warp / warps, nv = D / 8;
  float2 g[R], u[R];
#pragma unroll
  for (int r = 0; r < R; ++r) g[r] = u[r] = make_float2(0.f, 0.f);
  if (f < F) {
    // (one vector of each row at a time: batches of 2 and 4 cost more in resident warps than they put in flight)
    for (int64_t v = part * 32 + lane; v < nv; v += 32 * warps) {
      const uint4 a4 = __ldcs(w_gate + f * nv + v), b4 = __ldcs(w_up + f * nv + v);
      uint4 x4[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x4[r] = r < M ? __ldg(x + r * nv + v) : make_uint4(0, 0, 0, 0);
      const float2 a[4] = {pair_of(a4.x), pair_of(a4.y), pair_of(a4.z), pair_of(a4.w)};
      const float2 b[4] = {pair_of(b4.x), pair_of(b4.y), pair_of(b4.z), pair_of(b4.w)};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 xs[4] = {pair_of(x4[r].x), pair_of(x4[r].y), pair_of(x4[r].z), pair_of(x4[r].w)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[r] = fma2(a[j], xs[j], g[r]);
          u[r] = fma2(b[j], xs[j], u[r]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 s = make_float2(g[r].x + g[r].y, u[r].x + u[r].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    if (lane == 0) red[warp][r] = s;
  }
  __syncthreads();
  if (part == 0 && lane < R && lane < M && f < F) {   // the row's warps in their order
    float2 s = red[warp][lane];
    for (int w = 1; w < warps; ++w) {
      s.x += red[warp + w][lane].x;
      s.y += red[warp + w][lane].y;
    }
    if constexpr (GRAD) {
      float a, slope;
      act_both(s.x, act, a, slope);
      const float d = __bfloat162float(dh[lane * F + f]);
      dg[lane * F + f] = grad_gate(d, slope, s.y);
      du[lane * F + f] = d * a;
    } else {
      h[lane * F + f] = __float2bfloat16_rn(act_value(s.x, act) * s.y);
    }
  }
}

// The backward's two products for a few tokens, in one pass over the weights (the call's second: dg and du needed all of
// a row first) that also writes their gradients: a lane owns 8 columns of D, a warp takes every eighth row f of the CTA's
// chunk of F and adds dg Wg + du Wu to its part of dx while it writes dWg[f] = sum_r dg x and dWu[f].  dg and du stay
// fp32 here (of one or two tokens' rounding to bf16 little averages out).  partial: [chunk][token][D].
template <int R>
__global__ void __launch_bounds__(256, R == 4 ? 2 : 0)
ffn_rows_back_kernel(const uint4* __restrict__ x, const uint4* __restrict__ w_gate, const uint4* __restrict__ w_up,
                     const float* dg, const float* du, uint4* __restrict__ dw_gate,
                     uint4* __restrict__ dw_up, float* __restrict__ partial, int M, int64_t D, int64_t F,
                     int64_t chunk) {
  asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;\n" ::: "memory");
  __shared__ float2 red[8][R][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t nv = D / 8, v = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t f0 = blockIdx.y * chunk, f1 = f0 + chunk < F ? f0 + chunk : F;
  const bool on = v < nv;
  float2 xs[R][4], acc[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint4 t = on && r < M ? __ldg(x + r * nv + v) : make_uint4(0, 0, 0, 0);
    xs[r][0] = pair_of(t.x), xs[r][1] = pair_of(t.y), xs[r][2] = pair_of(t.z), xs[r][3] = pair_of(t.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[r][j] = make_float2(0.f, 0.f);
  }
#pragma unroll 2
  for (int64_t f = f0 + warp; f < f1; f += 8) {
    const uint4 a4 = on ? __ldcs(w_gate + f * nv + v) : make_uint4(0, 0, 0, 0);
    const uint4 b4 = on ? __ldcs(w_up + f * nv + v) : make_uint4(0, 0, 0, 0);
    const float2 a[4] = {pair_of(a4.x), pair_of(a4.y), pair_of(a4.z), pair_of(a4.w)};
    const float2 b[4] = {pair_of(b4.x), pair_of(b4.y), pair_of(b4.z), pair_of(b4.w)};
    float2 wa[4], wb[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) wa[j] = wb[j] = make_float2(0.f, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= M) continue;
      const float g = __ldcg(dg + r * F + f), u = __ldcg(du + r * F + f);   // (of the kernel before: past L1)
      const float2 g2 = make_float2(g, g), u2 = make_float2(u, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[r][j] = fma2(u2, b[j], fma2(g2, a[j], acc[r][j]));
        wa[j] = fma2(g2, xs[r][j], wa[j]);
        wb[j] = fma2(u2, xs[r][j], wb[j]);
      }
    }
    if (on) {
      dw_gate[f * nv + v] = make_uint4(pack_bf16x2(wa[0].x, wa[0].y), pack_bf16x2(wa[1].x, wa[1].y),
                                       pack_bf16x2(wa[2].x, wa[2].y), pack_bf16x2(wa[3].x, wa[3].y));
      dw_up[f * nv + v] = make_uint4(pack_bf16x2(wb[0].x, wb[0].y), pack_bf16x2(wb[1].x, wb[1].y),
                                     pack_bf16x2(wb[2].x, wb[2].y), pack_bf16x2(wb[3].x, wb[3].y));
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j) red[warp][r][j][lane] = acc[r][j];
  __syncthreads();
  // warp w: pair j = w % 4 of tokens w / 4, w / 4 + 2, .. summed over the warps in their order
  for (int r = warp >> 2; r < M; r += 2) {
    const int j = warp & 3;
    float2 s = red[0][r][j][lane];
    for (int w = 1; w < 8; ++w) {
      s.x += red[w][r][j][lane].x;
      s.y += red[w][r][j][lane].y;
    }
    if (on)
      *reinterpret_cast<float2*>(partial + (static_cast<int64_t>(blockIdx.y) * M + r) * D + v * 8 + 2 * j) = s;
  }
}

// dx = the chunks' sums: 32 pairs of columns to a CTA, each warp takes every eighth chunk, then the warps in order.
__global__ void __launch_bounds__(256)
ffn_rows_join_kernel(const float2* partial, uint32_t* __restrict__ dx, int64_t pairs, int chunks) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  __shared__ float2 red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float2 s = make_float2(0.f, 0.f);
  if (i < pairs) {
#pragma unroll 4
    for (int c = warp; c < chunks; c += 8) {
      const float2 p = __ldcg(partial + c * pairs + i);
      s.x += p.x;
      s.y += p.y;
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && i < pairs) {
    for (int w = 1; w < 8; ++w) {
      s.x += red[w][lane].x;
      s.y += red[w][lane].y;
    }
    dx[i] = pack_bf16x2(s.x, s.y);
  }
}

// ---------------------------------------------------------------- host
// A [rows][cols] row-major bf16 matrix seen through swizzled boxes of box_rows x box_cols (64: 128-byte rows,
// operands; 32: 64-byte rows, results).
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int box_rows, int box_cols = 64) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Where the rows kernels run instead of tiles of 256 rows: for one and two tokens, and up to four on weights of at
// most 2^22 entries (its unpacking of the tokens grows with them).  Measured rows / tiles, us, L2 cold:
//   forward   1 token 1024 -> 2816 9 / 16, 2048 -> 5632 15 / 23, 4096 -> 8192 35 / 43; 2 tokens 2048 -> 5632 16 / 23;
//             4 tokens 1024 -> 2816 12.5 / 15, 4096 -> 512 10.5 / 20.5, 2048 -> 5632 27 / 24, 4096 -> 8192 49 / 46
//   backward  1 token 17 / 32, 40 / 53, 95 / 105; 2 tokens 48 / 53; 4 tokens 34 / 30, 21.5 / 30, 75 / 53, 161 / 104
// (the same sizes in the same order; 4 tokens 1024 -> 2816 stay with the rows, which keep dg and du in fp32).
bool few_rows(int64_t M, int64_t D, int64_t F) { return M <= 2 || (M <= 4 && D * F <= (1 << 22)); }
// A part costs its sums' way to memory and back and a second launch, about 6 us or 24 k blocks: K is split where more
// than that is saved.
constexpr int kSplitSaves = 24;

constexpr int64_t kPairs = 76;      // of CTAs, on the card's 152 SMs
// m tiles that take the same n tiles in turn, so that their operands meet in L2: 19, so that the 76 pairs work on 19
// by 4 tiles at a time (a second of 2048 x 5632 calls at the power limit: 65,536-token forward 1713 us with 19, 1735 with 16,
// 1760 with 8 or 10; 16,384-token backward 1410, 1432, 1430).  One number for all products: the gated ones have 44 n tiles
// there, dx and dW 8, so a group of theirs takes two rounds, and its dg and du are read from memory twice (dx of 8,192
// tokens reads 569 MB, its operands are 231; it is not bound by HBM).
constexpr int kGroup = 19;

Product product(Mode mode, int64_t M, int64_t D, int64_t F) {
  const bool gated = mode == kGate || mode == kGateGrad, dw = mode == kDw;
  Product p{};
  p.dw = dw;
  p.half_tiles = dw ? ceil_div(F, 256) : 0;
  p.m_tiles = dw ? 2 * p.half_tiles : ceil_div(M, 256);
  p.n_tiles = gated ? ceil_div(F, 128) : ceil_div(D, 256);
  p.tiles = p.m_tiles * p.n_tiles;
  p.kb_half = gated || dw ? 0 : static_cast<int>(ceil_div(F, kBK));
  p.kb = gated ? static_cast<int>(ceil_div(D, kBK)) : dw ? static_cast<int>(ceil_div(M, kBK)) : 2 * p.kb_half;
  p.rows = dw ? F : M;
  p.cols = gated ? F : D;
  return p;
}
void cut(Product& p, int64_t parts) {
  p.kb_part = static_cast<int>(ceil_div(p.kb, parts));
  p.units = p.tiles * ceil_div(p.kb, p.kb_part);
}
// Parts of K that a product may be cut into: of 8 k blocks or more, and where at least half of the pairs would have
// no tile.
int64_t most_parts(const Product& p) {
  const int64_t parts = kPairs / p.tiles, long_enough = p.kb / 8;
  const int64_t most = parts < long_enough ? parts : long_enough;
  return most < 1 ? 1 : most;
}

// K blocks that the busiest pair works through, with the best `skip` for it (Walk's rounds, counted).
int64_t busiest(const Shape& sh, int64_t* skip) {
  const Product &a = sh.p[0], &b = sh.p[1];
  const int64_t pairs = a.units + b.units < kPairs ? a.units + b.units : kPairs;
  const int64_t rounds = a.units / pairs, h = a.units % pairs, l = h ? pairs - h : 0;
  int64_t best = 0;
  for (int64_t s = 0; s <= 8 && s * l <= b.units; ++s) {
    const int64_t left = b.units - s * l, full = left / pairs, rest = left % pairs;
    const int64_t few = rounds * a.kb_part + (s + full + (rest > 0)) * b.kb_part;
    const int64_t many = h ? (rounds + 1) * a.kb_part + (full + (rest > l)) * b.kb_part : 0;
    const int64_t most = few > many ? few : many;
    if (s == 0 || most < best) {
      best = most;
      *skip = s;
    }
    if (!l) break;
  }
  return best;
}

// One product: whole tiles, or parts of K where that saves more than a part costs.
Shape one_shape(Mode mode, int64_t M, int64_t D, int64_t F, int act) {
  Shape sh{};
  sh.p[0] = product(mode, M, D, F);
  sh.group = kGroup;
  sh.act = act;
  int64_t parts = most_parts(sh.p[0]);
  if (sh.p[0].kb - sh.p[0].kb / parts < kSplitSaves) parts = 1;
  cut(sh.p[0], parts);
  return sh;
}

// The backward's last two products in one launch: the longer units first, and either cut into parts of K where the
// busiest pair is saved more than the parts cost.
int64_t split_cost(const Product& p) { return p.units > p.tiles ? kSplitSaves : 0; }
Shape back_shape(int64_t M, int64_t D, int64_t F, int64_t* cost) {
  Product dx = product(kDx, M, D, F), dw = product(kDw, M, D, F);
  const int64_t most_dx = most_parts(dx), most_dw = most_parts(dw);
  Shape best{};
  *cost = -1;
  for (int64_t i = 1; i <= most_dx; i += 1 + i / 2)      // (1, 2, 4, 7, 11, ..)
    for (int64_t j = 1; j <= most_dw; j += 1 + j / 2) {
      cut(dx, i);
      cut(dw, j);
      Shape sh{};
      sh.p[0] = dx.kb_part > dw.kb_part ? dx : dw;
      sh.p[1] = dx.kb_part > dw.kb_part ? dw : dx;
      const int64_t c = busiest(sh, &sh.skip) + (split_cost(dx) > split_cost(dw) ? split_cost(dx) : split_cost(dw));
      if (*cost < 0 || c < *cost) {
        *cost = c;
        best = sh;
      }
    }
  best.group = kGroup;
  return best;
}
struct BackPlan {
  bool merged;
  Shape both, dx, dw;
};
// Whether they share a launch.  It saves the rounds in which one product leaves pairs idle, and a launch (kLaunch k
// blocks); but its pairs fall out of step, and tiles that were read together no longer meet in L2, which costs a
// long run about 6 % (16,384 x 2048 x 5632: 810 us merged, 792 in two launches, for 2432 against 2512 k blocks; 2048 x
// 1024 x 2816 backward 54 us merged, 73 in two, for 152 against 216).
constexpr int64_t kLaunch = 16;
BackPlan back_plan(int64_t M, int64_t D, int64_t F) {
  BackPlan b{};
  int64_t merged = 0, skip = 0;
  b.both = back_shape(M, D, F, &merged);
  b.dx = one_shape(kDx, M, D, F, 0);
  b.dw = one_shape(kDw, M, D, F, 0);
  const int64_t apart = busiest(b.dx, &skip) + split_cost(b.dx.p[0]) + busiest(b.dw, &skip) + split_cost(b.dw.p[0]);
  b.merged = merged + merged / 16 < apart + kLaunch;
  return b;
}
size_t partial_bytes(const Product& p) {
  return p.units > p.tiles ? static_cast<size_t>(p.units) * 256 * 256 * sizeof(float) : 0;
}
size_t partial_bytes(const Shape& sh) { return partial_bytes(sh.p[0]) + partial_bytes(sh.p[1]); }
size_t partial_bytes(const BackPlan& b) {
  const size_t dx = partial_bytes(b.dx), dw = partial_bytes(b.dw);
  return b.merged ? partial_bytes(b.both) : dx > dw ? dx : dw;
}

// A kernel that may set itself up while the one before it on the stream ends.
template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <int MODE, bool SPLIT>
cudaError_t launch_part(const char* name, const Maps& maps, const Shape& sh, bool first, unsigned int* status,
                        cudaStream_t stream) {
  using C = Cfg<MODE>;
  auto kernel = ffn_gemm_kernel<MODE, SPLIT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const int64_t units = sh.p[0].units + sh.p[1].units;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < kPairs ? units : kPairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 2;   // a call's first kernel waits for the stream, the others for the one before them
  ProfScope prof(name, stream);
  return cudaLaunchKernelEx(&cfg, kernel, maps, sh, status);
}

template <int MODE>
cudaError_t launch_gemm(const char* name, const Maps& maps, Shape sh, bool first, float* partial, const JoinOut& out,
                        unsigned int* status, cudaStream_t stream) {
  if (!partial_bytes(sh)) return launch_part<MODE, false>(name, maps, sh, first, status, stream);
  int64_t vectors = 0;
  for (Product& p : sh.p) {
    if (!partial_bytes(p)) continue;
    p.partial = partial;
    partial += partial_bytes(p) / sizeof(float);
    if (p.rows * (p.cols / 8) > vectors) vectors = p.rows * (p.cols / 8);
  }
  cudaError_t e = launch_part<MODE, true>(name, maps, sh, first, status, stream);
  if (e != cudaSuccess) return e;
  ProfScope prof("ffn_join", stream);
  return launch_after(ffn_join_kernel<MODE>, dim3(static_cast<unsigned>(ceil_div(vectors, 256)), MODE == kBack ? 3 : MODE == kDw ? 2 : 1),
                      stream, sh, out);
}

template <int R, bool GRAD>
cudaError_t launch_rows(const FfnParams& p, float* dg, float* du, cudaStream_t stream) {
  // warps to a row: as many as bring four CTAs to each SM, while each has 512 features to read
  int warps = 1;
  while (warps < 8 && p.F * warps / 8 < 4 * 152 && p.D >= 1024 * warps) warps *= 2;
  ProfScope prof(GRAD ? "ffn_rows_grad" : "ffn_rows", stream);
  ffn_rows_kernel<R, GRAD><<<static_cast<unsigned>(ceil_div(p.F * warps, 8)), 256, 0, stream>>>(
      reinterpret_cast<const uint4*>(p.x), reinterpret_cast<const uint4*>(p.w_gate),
      reinterpret_cast<const uint4*>(p.w_up), p.h, p.dh, dg, du, static_cast<int>(p.M), p.D, p.F, warps, p.act);
  return cudaGetLastError();
}

// The few tokens' backward: workspace of dg, du (fp32 [M][F] each), then the chunks' parts of dx.
struct RowsBack {
  int64_t chunk, chunks;   // rows of F to a CTA; CTAs along F
  size_t dg_bytes, total;
};
RowsBack rows_back(int64_t M, int64_t D, int64_t F) {
  RowsBack b;
  const int64_t d_tiles = ceil_div(D, 256);
  b.chunk = 8 * ceil_div(F, 8 * ceil_div(4 * 152, d_tiles));   // about four CTAs to each SM, whole turns of 8 warps
  if (b.chunk < 32) b.chunk = 32;
  b.chunks = ceil_div(F, b.chunk);
  b.dg_bytes = (sizeof(float) * static_cast<size_t>(M) * F + 255) / 256 * 256;
  b.total = 2 * b.dg_bytes + sizeof(float) * static_cast<size_t>(b.chunks) * M * D;
  return b;
}

template <int R>
cudaError_t launch_rows_back(const FfnParams& p, cudaStream_t stream) {
  const RowsBack b = rows_back(p.M, p.D, p.F);
  char* ws = static_cast<char*>(p.ws);
  float *dg = reinterpret_cast<float*>(ws), *du = reinterpret_cast<float*>(ws + b.dg_bytes);
  float* partial = reinterpret_cast<float*>(ws + 2 * b.dg_bytes);
  cudaError_t e = launch_rows<R, true>(p, dg, du, stream);
  if (e != cudaSuccess) return e;
  {
    ProfScope prof("ffn_rows_back", stream);
    e = launch_after(ffn_rows_back_kernel<R>,
                     dim3(static_cast<unsigned>(ceil_div(p.D, 256)), static_cast<unsigned>(b.chunks)), stream,
                     reinterpret_cast<const uint4*>(p.x), reinterpret_cast<const uint4*>(p.w_gate),
                     reinterpret_cast<const uint4*>(p.w_up), dg, du, reinterpret_cast<uint4*>(p.dw_gate),
                     reinterpret_cast<uint4*>(p.dw_up), partial, static_cast<int>(p.M), p.D, p.F, b.chunk);
    if (e != cudaSuccess) return e;
  }
  ProfScope prof("ffn_rows_join", stream);
  const int64_t pairs = p.M * p.D / 2;
  return launch_after(ffn_rows_join_kernel, dim3(static_cast<unsigned>(ceil_div(pairs, 32))), stream,
                      reinterpret_cast<const float2*>(partial), reinterpret_cast<uint32_t*>(p.dx), pairs,
                      static_cast<int>(b.chunks));
}

template <class F>
cudaError_t by_rows(int64_t M, F&& go) {
  return M == 1 ? go(std::integral_constant<int, 1>()) : M == 2 ? go(std::integral_constant<int, 2>())
                                                                : go(std::integral_constant<int, 4>());
}

// dg and du of the tiles' backward, bf16 [M][F] each at the front of its workspace.
size_t half_bytes(int64_t M, int64_t F) { return (sizeof(bf16) * static_cast<size_t>(M) * F + 255) / 256 * 256; }

}  // namespace

size_t ffn_fwd_workspace(int64_t M, int64_t D, int64_t F) {
  return few_rows(M, D, F) ? 0 : partial_bytes(one_shape(kGate, M, D, F, 0));
}

size_t ffn_bwd_workspace(int64_t M, int64_t D, int64_t F) {
  if (few_rows(M, D, F)) return rows_back(M, D, F).total;
  const size_t grad = partial_bytes(one_shape(kGateGrad, M, D, F, 0)), back = partial_bytes(back_plan(M, D, F));
  return 2 * half_bytes(M, F) + (grad > back ? grad : back);
}

cudaError_t launch_ffn_gated_fwd(const FfnParams& p, cudaStream_t stream) {
  if (few_rows(p.M, p.D, p.F))
    return by_rows(p.M, [&](auto r) { return launch_rows<decltype(r)::value, false>(p, nullptr, nullptr, stream); });
  Maps maps{};
  if (!make_map(&maps.a0, p.x, p.M, p.D, 128) || !make_map(&maps.b0, p.w_gate, p.F, p.D, 128) ||
      !make_map(&maps.b1, p.w_up, p.F, p.D, 128) || !make_map(&maps.c0, p.h, p.M, p.F, 128, 32))
    return cudaErrorInvalidValue;
  return launch_gemm<kGate>("ffn_gate", maps, one_shape(kGate, p.M, p.D, p.F, p.act), true,
                            static_cast<float*>(p.ws), JoinOut{p.h, nullptr, nullptr}, p.status, stream);
}

cudaError_t launch_ffn_gated_bwd(const FfnParams& p, cudaStream_t stream) {
  if (few_rows(p.M, p.D, p.F))
    return by_rows(p.M, [&](auto r) { return launch_rows_back<decltype(r)::value>(p, stream); });
  char* ws = static_cast<char*>(p.ws);
  bf16 *dg = reinterpret_cast<bf16*>(ws), *du = reinterpret_cast<bf16*>(ws + half_bytes(p.M, p.F));
  float* partial = reinterpret_cast<float*>(ws + 2 * half_bytes(p.M, p.F));
  Maps grad{}, back{};
  if (!make_map(&grad.a0, p.x, p.M, p.D, 128) || !make_map(&grad.b0, p.w_gate, p.F, p.D, 128) ||
      !make_map(&grad.b1, p.w_up, p.F, p.D, 128) ||
      !make_map(&grad.c0, dg, p.M, p.F, 128, 32) || !make_map(&grad.c1, du, p.M, p.F, 128, 32) ||
      !make_map(&back.a0, dg, p.M, p.F, 128) || !make_map(&back.a1, du, p.M, p.F, 128) ||
      !make_map(&back.t0, dg, p.M, p.F, 64) || !make_map(&back.t1, du, p.M, p.F, 64) ||
      !make_map(&back.b0, p.w_gate, p.F, p.D, 64) || !make_map(&back.b1, p.w_up, p.F, p.D, 64) ||
      !make_map(&back.b2, p.x, p.M, p.D, 64) || !make_map(&back.c0, p.dx, p.M, p.D, 128, 32) ||
      !make_map(&back.c1, p.dw_gate, p.F, p.D, 128, 32) || !make_map(&back.c2, p.dw_up, p.F, p.D, 128, 32))
    return cudaErrorInvalidValue;
  Shape grad_shape = one_shape(kGateGrad, p.M, p.D, p.F, p.act);
  grad_shape.dh = p.dh;
  cudaError_t e = launch_gemm<kGateGrad>("ffn_gate_grad", grad, grad_shape, true, partial, JoinOut{dg, du, nullptr},
                                         p.status, stream);
  if (e != cudaSuccess) return e;
  const BackPlan plan = back_plan(p.M, p.D, p.F);
  const JoinOut out{p.dx, p.dw_gate, p.dw_up};
  if (plan.merged) return launch_gemm<kBack>("ffn_back", back, plan.both, false, partial, out, p.status, stream);
  e = launch_gemm<kDx>("ffn_dx", back, plan.dx, false, partial, out, p.status, stream);
  return e != cudaSuccess ? e : launch_gemm<kDw>("ffn_dw", back, plan.dw, false, partial, out, p.status, stream);
}

}  // namespace dsv
