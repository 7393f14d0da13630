// C ABI of libdsv.so (declared in include/dsv.h): host-side validation, workspace
// planning and launches.  Nothing here allocates device memory.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <map>
#include <string>
#include <utility>
#include <vector>

#include "../../include/dsv.h"
#include "dsv_block.h"
#include "dsv_internal.h"

// Device status word: kernels OR in kStatusBadIndex when they meet a key index outside
// [0, N) or a repeated key in one idx row.  Read and cleared by dsv_last_device_status.
__device__ unsigned int g_dsv_status;

namespace {

thread_local char g_msg[512] = "";

dsv_status fail(dsv_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

dsv_status ok() {
  g_msg[0] = '\0';
  return DSV_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;
// Per-device address of g_dsv_status, looked up on first use with that device current (host
// threads racing on the first look-up all find the same address).
std::atomic<unsigned int*> g_status_ptr[kMaxDevices];

dsv_status status_word(unsigned int** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(DSV_ERR_CUDA, "device ordinal %d out of range", dev);
  unsigned int* ptr = g_status_ptr[dev].load(std::memory_order_acquire);
  if (!ptr) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_dsv_status);
    if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
    ptr = static_cast<unsigned int*>(p);
    g_status_ptr[dev].store(ptr, std::memory_order_release);
  }
  *out = ptr;
  return DSV_OK;
}

dsv_status check_dims(const dsv_dims* d, bool need_d, bool need_r) {
  if (!d) return fail(DSV_ERR_INVALID_ARG, "dims is NULL");
  if (d->B < 1 || d->H < 1 || d->N < 1) return fail(DSV_ERR_INVALID_ARG, "B, H, N must be >= 1");
  if (d->block != 64) return fail(DSV_ERR_UNSUPPORTED, "block must be 64 (got %lld)", (long long)d->block);
  if (d->N % d->block) return fail(DSV_ERR_INVALID_ARG, "N (%lld) must be a multiple of block", (long long)d->N);
  if (d->N > 0x7fffffffLL) return fail(DSV_ERR_INVALID_ARG, "N must fit int32 key indices");
  if (d->k < 1 || d->k > d->N) return fail(DSV_ERR_INVALID_ARG, "need 1 <= k <= N (k=%lld)", (long long)d->k);
  if (d->B * d->H > (1LL << 31) - 1) return fail(DSV_ERR_INVALID_ARG, "B*H too large");
  if (d->B * d->H * d->N > 0x7fffffffLL)
    return fail(DSV_ERR_INVALID_ARG, "B*H*N must fit int32 row coordinates (split the heads over calls)");
  if (need_d && d->d != 64 && d->d != 128)
    return fail(DSV_ERR_UNSUPPORTED, "head dim d must be 64 or 128 (got %lld)", (long long)d->d);
  if (need_r && (d->r < 16 || d->r > 64 || d->r % 16))
    return fail(DSV_ERR_UNSUPPORTED, "low-rank dim r must be 16, 32, 48 or 64 (got %lld)", (long long)d->r);
  if (!(d->scale == d->scale)) return fail(DSV_ERR_INVALID_ARG, "scale is NaN");
  return DSV_OK;
}

#define DSV_NEED_PTR(p)                                                                \
  do {                                                                                 \
    if (!(p)) return fail(DSV_ERR_INVALID_ARG, "%s is NULL", #p);                     \
    if (!aligned16(p)) return fail(DSV_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

float eff_scale(const dsv_dims* d) { return d->scale > 0.f ? d->scale : 1.0f / sqrtf(static_cast<float>(d->d)); }

// ---------------------------------------------------------------- backward workspace planning
constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct WavePlan {
  int64_t nh = 0, nblk = 0;  // heads per wave (whole-head waves) or blocks per wave (sub-head)
  bool sub = false;
};

struct Carve {
  size_t colbits, colpre, count, offsets, tsum, lists, partial, partial_dv, acc, total;
};

// pairs: the (block, key) pairs of the largest wave (-1: nh * nblk * k)
Carve carve(const dsv_dims* d, int64_t nh, int64_t nblk, bool sub, int64_t pairs = -1) {
  const int64_t W32 = (nblk + 31) / 32;
  if (pairs < 0) pairs = nh * nblk * d->k;
  Carve c;
  size_t o = 0;
  c.colbits = o; o += up(sizeof(uint32_t) * nh * W32 * d->N);
  c.colpre = o;  o += up(sizeof(uint32_t) * nh * W32 * d->N);
  c.count = o;   o += up(sizeof(uint32_t) * nh * d->N);
  c.offsets = o; o += up(sizeof(int64_t) * nh * d->N);
  c.tsum = o;    o += up(sizeof(int64_t) * nh * ((d->N + 1023) / 1024));
  c.lists = o;   o += up(sizeof(int32_t) * pairs);
  c.partial = o; o += up(sizeof(uint16_t) * d->d * pairs);       // bf16 dK half-rows
  c.partial_dv = o; o += up(sizeof(uint16_t) * d->d * pairs);    // bf16 dV half-rows
  c.acc = o;     o += sub ? up(sizeof(float) * 2 * d->d * d->N) : 0;
  c.total = o;
  return c;
}

size_t plan_bytes(const dsv_dims* d, const WavePlan& w) { return carve(d, w.nh, w.nblk, w.sub).total; }

// Largest plan that fits `budget` bytes (whole heads first, then blocks of one head).
bool plan_for(const dsv_dims* d, size_t budget, WavePlan* out) {
  const int64_t BH = d->B * d->H, NB = d->N / 64;
  for (int64_t nh = BH; nh >= 1; nh = (nh == 1 ? 0 : (nh + 1) / 2)) {
    WavePlan w{nh, NB, false};
    if (plan_bytes(d, w) <= budget) {
      // grow back towards BH while it still fits (the halving may undershoot)
      while (w.nh < BH) {
        WavePlan w2{w.nh + 1, NB, false};
        if (plan_bytes(d, w2) > budget) break;
        w = w2;
      }
      *out = w;
      return true;
    }
    if (nh == 1) break;
  }
  // blocks of one head per wave: the largest even split that fits, rounded down to whole waves of
  // the main kernel's CTAs (one per SM), so that only a head's last wave ends in a partial one
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    sms = 0;
    (void)cudaGetLastError();  // no device (a size query on a host without one): no rounding
  }
  for (int64_t s = 2; s <= NB; s = (s < 64 ? s + 1 : s + s / 8)) {
    int64_t nblk = (NB + s - 1) / s;
    WavePlan w{1, nblk, true};
    if (plan_bytes(d, w) <= budget) {
      if (sms > 0 && nblk > sms) w.nblk = nblk / sms * sms;
      *out = w;
      return true;
    }
  }
  WavePlan w{1, 1, NB > 1};
  if (plan_bytes(d, w) <= budget) { *out = w; return true; }
  return false;
}

constexpr size_t kRecommendedPartialBytes = size_t(16) << 30;

// ---------------------------------------------------------------- optional per-kernel timing
struct ProfRecord {
  const char* name;
  cudaEvent_t begin, end;
};
constexpr int kProfPool = 16384;
bool g_prof_on = false;
std::vector<cudaEvent_t> g_prof_events;   // 2 * kProfPool, created at enable time
std::vector<ProfRecord> g_prof_records;
size_t g_prof_dropped = 0;

}  // namespace

namespace dsv {
ProfScope::ProfScope(const char* name, cudaStream_t s) : slot(-1), stream(s) {
  if (!g_prof_on) return;
  const size_t n = g_prof_records.size();
  if (n >= static_cast<size_t>(kProfPool)) { ++g_prof_dropped; return; }
  ProfRecord r{name, g_prof_events[2 * n], g_prof_events[2 * n + 1]};
  if (cudaEventRecord(r.begin, s) != cudaSuccess) return;
  g_prof_records.push_back(r);
  slot = static_cast<int>(n);
}
ProfScope::~ProfScope() {
  if (slot >= 0) cudaEventRecord(g_prof_records[slot].end, stream);
}
}  // namespace dsv

extern "C" {

const char* dsv_status_string(dsv_status s) {
  switch (s) {
    case DSV_OK: return "DSV_OK";
    case DSV_ERR_INVALID_ARG: return "DSV_ERR_INVALID_ARG";
    case DSV_ERR_UNSUPPORTED: return "DSV_ERR_UNSUPPORTED";
    case DSV_ERR_WORKSPACE: return "DSV_ERR_WORKSPACE";
    case DSV_ERR_CUDA: return "DSV_ERR_CUDA";
    case DSV_ERR_DEVICE_CHECK: return "DSV_ERR_DEVICE_CHECK";
  }
  return "DSV_ERR_UNKNOWN";
}

const char* dsv_last_error_message(void) { return g_msg; }

size_t dsv_estimate_topk_workspace(const dsv_dims* dims) {
  (void)dims;
  return 0;
}

dsv_status dsv_estimate_topk(const dsv_dims* dims, const void* q_lr, const void* k_lr, int32_t* idx, void* ws,
                             size_t ws_bytes, void* stream) {
  (void)ws;
  (void)ws_bytes;
  dsv_status s = check_dims(dims, false, true);
  if (s != DSV_OK) return s;
  DSV_NEED_PTR(q_lr);
  DSV_NEED_PTR(k_lr);
  DSV_NEED_PTR(idx);
  unsigned int* status = nullptr;
  if ((s = status_word(&status)) != DSV_OK) return s;
  dsv::EstimateParams p;
  p.q_lr = static_cast<const dsv::bf16*>(q_lr);
  p.k_lr = static_cast<const dsv::bf16*>(k_lr);
  p.idx = idx;
  p.BH = dims->B * dims->H;
  p.N = dims->N;
  p.NB = dims->N / dims->block;
  p.topk = dims->k;
  p.r = static_cast<int>(dims->r);
  p.status = status;
  cudaError_t e = dsv::launch_estimate_topk(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "estimate launch: %s", cudaGetErrorString(e));
  return ok();
}

dsv_status dsv_estimate_mass_k(const dsv_dims* dims, const void* q_lr, const void* k_lr, float tau_log2,
                               uint32_t mass_num, uint32_t dense_num, int32_t* k_row, int64_t* rowptr, int32_t* order,
                               void* stream) {
  dsv_status s = check_dims(dims, false, true);
  if (s != DSV_OK) return s;
  DSV_NEED_PTR(q_lr);
  DSV_NEED_PTR(k_lr);
  if (!k_row) return fail(DSV_ERR_INVALID_ARG, "k_row is NULL");
  if (!rowptr) return fail(DSV_ERR_INVALID_ARG, "rowptr is NULL");
  if (!(tau_log2 > 0.f) || !(tau_log2 < 3.0e38f)) return fail(DSV_ERR_INVALID_ARG, "tau_log2 must be finite and > 0");
  if (mass_num < 1 || mass_num > 65536) return fail(DSV_ERR_INVALID_ARG, "mass_num must be in [1, 65536] (got %u)", mass_num);
  if (dense_num > 65536) return fail(DSV_ERR_INVALID_ARG, "dense_num must be in [0, 65536] (got %u)", dense_num);
  if (dims->N > (1LL << 20))
    return fail(DSV_ERR_UNSUPPORTED, "mass selection supports N <= 2^20 (the weight sums are 64-bit)");
  if (order && (dims->N + 127) / 128 + 1 > 4096)
    return fail(DSV_ERR_UNSUPPORTED, "a launch order needs N <= 523904");
  unsigned int* status = nullptr;
  if ((s = status_word(&status)) != DSV_OK) return s;
  dsv::MassParams p;
  p.q_lr = static_cast<const dsv::bf16*>(q_lr);
  p.k_lr = static_cast<const dsv::bf16*>(k_lr);
  p.BH = dims->B * dims->H;
  p.N = dims->N;
  p.NB = dims->N / dims->block;
  p.r = static_cast<int>(dims->r);
  p.tau_log2 = tau_log2;
  p.mass_num = mass_num;
  p.dense_num = dense_num;
  double fact = 1.0;
  for (int i = 0; i < 7; ++i) {  // Taylor coefficients of 2^f: (ln 2)^i / i!, rounded to fp32
    if (i > 0) fact *= i;
    p.coef[i] = static_cast<float>(std::pow(std::log(2.0), i) / fact);
  }
  p.krow = k_row;
  p.rowptr = rowptr;
  p.order = order;
  p.status = status;
  cudaError_t e = dsv::launch_estimate_mass_k(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "mass selection launch: %s", cudaGetErrorString(e));
  return ok();
}

dsv_status dsv_csr_launch_order(const dsv_dims* dims, const int64_t* rowptr, int32_t* order, void* stream) {
  dsv_status s = check_dims(dims, false, false);
  if (s != DSV_OK) return s;
  if (!rowptr || !order) return fail(DSV_ERR_INVALID_ARG, "rowptr and order must be non-NULL");
  if ((dims->N + 127) / 128 + 1 > 4096) return fail(DSV_ERR_UNSUPPORTED, "a launch order needs N <= 523904");
  cudaError_t e = dsv::launch_csr_order(rowptr, dims->B * dims->H * (dims->N / dims->block), dims->N, order,
                                        static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "launch order: %s", cudaGetErrorString(e));
  return ok();
}

dsv_status dsv_estimate_topk_csr(const dsv_dims* dims, const void* q_lr, const void* k_lr, const int32_t* k_row,
                                 const int64_t* rowptr, int32_t* cols, void* stream) {
  dsv_status s = check_dims(dims, false, true);
  if (s != DSV_OK) return s;
  DSV_NEED_PTR(q_lr);
  DSV_NEED_PTR(k_lr);
  if (!k_row || !rowptr || !cols) return fail(DSV_ERR_INVALID_ARG, "k_row, rowptr and cols must be non-NULL");
  unsigned int* status = nullptr;
  if ((s = status_word(&status)) != DSV_OK) return s;
  dsv::EstimateParams p;
  p.q_lr = static_cast<const dsv::bf16*>(q_lr);
  p.k_lr = static_cast<const dsv::bf16*>(k_lr);
  p.idx = cols;
  p.BH = dims->B * dims->H;
  p.N = dims->N;
  p.NB = dims->N / dims->block;
  p.topk = dims->N;
  p.r = static_cast<int>(dims->r);
  p.krow = k_row;
  p.rowptr = rowptr;
  p.status = status;
  cudaError_t e = dsv::launch_estimate_topk(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "estimate launch: %s", cudaGetErrorString(e));
  return ok();
}

// The forward needs no scratch at present (its workspace arguments are reserved).
size_t fwd_workspace_bytes(const dsv_dims*) { return 0; }

dsv_status fwd_impl(const dsv_dims* dims, const void* q, const void* k, const void* v, const int32_t* idx,
                    const int64_t* rowptr, const int32_t* order, void* o, float* lse, void* ws, size_t ws_bytes,
                    void* stream) {
  dsv_status s = check_dims(dims, true, false);
  if (s != DSV_OK) return s;
  if (ws && !aligned16(ws)) return fail(DSV_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  DSV_NEED_PTR(q);
  DSV_NEED_PTR(k);
  DSV_NEED_PTR(v);
  if (rowptr || dims->k != dims->N) DSV_NEED_PTR(idx);  // k = N: every key, idx is not read
  DSV_NEED_PTR(o);
  DSV_NEED_PTR(lse);
  unsigned int* status = nullptr;
  if ((s = status_word(&status)) != DSV_OK) return s;
  dsv::FwdParams p;
  p.q = static_cast<const dsv::bf16*>(q);
  p.k = static_cast<const dsv::bf16*>(k);
  p.v = static_cast<const dsv::bf16*>(v);
  p.idx = idx;
  p.o = static_cast<dsv::bf16*>(o);
  p.lse = lse;
  p.BH = dims->B * dims->H;
  p.N = dims->N;
  p.NB = dims->N / dims->block;
  p.topk = dims->k;
  p.d = static_cast<int>(dims->d);
  p.scale = eff_scale(dims);
  p.status = status;
  p.rowptr = rowptr;
  p.order = order;
  (void)ws_bytes;
  cudaError_t e = dsv::launch_sparse_fwd_tc(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "forward launch: %s", cudaGetErrorString(e));
  return ok();
}

size_t dsv_sparse_attn_fwd_workspace(const dsv_dims* dims) {
  if (check_dims(dims, true, false) != DSV_OK) return 0;
  return fwd_workspace_bytes(dims);
}

dsv_status dsv_sparse_attn_fwd(const dsv_dims* dims, const void* q, const void* k, const void* v, const int32_t* idx,
                               void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  return fwd_impl(dims, q, k, v, idx, nullptr, nullptr, o, lse, ws, ws_bytes, stream);
}

dsv_status dsv_sparse_attn_fwd_csr(const dsv_dims* dims, const void* q, const void* k, const void* v,
                                   const int64_t* rowptr, const int32_t* cols, const int32_t* order, void* o,
                                   float* lse, void* stream) {
  if (!rowptr) return fail(DSV_ERR_INVALID_ARG, "rowptr is NULL");
  return fwd_impl(dims, q, k, v, cols, rowptr, order, o, lse, nullptr, 0, stream);
}

// k = N (every key selected): the dense backward needs only D = rowsum(dO o O) per query row;
// no partial rows at all.
size_t dense_bwd_bytes(const dsv_dims* d) { return up(sizeof(float) * static_cast<size_t>(d->B * d->H * d->N)); }

size_t dsv_sparse_attn_bwd_workspace_min(const dsv_dims* dims) {
  if (check_dims(dims, true, false) != DSV_OK) return 0;
  if (dims->k == dims->N) return dense_bwd_bytes(dims);
  WavePlan w{1, 1, dims->N / 64 > 1};
  return plan_bytes(dims, w);
}

size_t dsv_sparse_attn_bwd_workspace(const dsv_dims* dims) {
  if (check_dims(dims, true, false) != DSV_OK) return 0;
  if (dims->k == dims->N) return dense_bwd_bytes(dims);
  // the largest plan whose partial rows stay within the recommended budget
  const size_t per_block = sizeof(uint16_t) * 2 * dims->d * dims->k;
  const int64_t BH = dims->B * dims->H, NB = dims->N / 64;
  const int64_t blocks = static_cast<int64_t>(kRecommendedPartialBytes / (per_block ? per_block : 1));
  WavePlan w;
  if (blocks >= BH * NB) w = WavePlan{BH, NB, false};
  else if (blocks >= NB) w = WavePlan{blocks / NB, NB, false};
  else {
    const int64_t nblk = blocks < 1 ? 1 : blocks;
    const int64_t s = (NB + nblk - 1) / nblk;
    w = WavePlan{1, (NB + s - 1) / s, true};
  }
  return plan_bytes(dims, w);
}

// rowptr == nullptr: k keys per block, waves planned from the workspace; otherwise CSR rows
// with total_pairs keys in all, one wave over every head (the workspace must hold it).
// parts: dsv::kBwdAll, or one of the two halves of a split backward (kBwdPrep reads idx only;
// kBwdFinish expects the workspace a kBwdPrep call filled); the halves need a single wave.
dsv_status bwd_impl(const dsv_dims* dims, const void* d_o, const void* q, const void* k, const void* v,
                    const void* o, const float* lse, const int32_t* idx, const int64_t* rowptr,
                    const int32_t* order, int64_t total_pairs, void* dq, void* dk, void* dv, void* ws,
                    size_t ws_bytes, void* stream, int parts = dsv::kBwdAll) {
  dsv_status s = check_dims(dims, true, false);
  if (s != DSV_OK) return s;
  if (rowptr || dims->k != dims->N) DSV_NEED_PTR(idx);  // k = N: every key, idx is not read
  if (parts & dsv::kBwdFinish) {
    DSV_NEED_PTR(d_o);
    DSV_NEED_PTR(q);
    DSV_NEED_PTR(k);
    DSV_NEED_PTR(v);
    DSV_NEED_PTR(o);
    DSV_NEED_PTR(lse);
    DSV_NEED_PTR(dq);
    DSV_NEED_PTR(dk);
    DSV_NEED_PTR(dv);
  }
  if (!ws) return fail(DSV_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return fail(DSV_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (!rowptr && dims->k == dims->N) {
    // every key selected: the dense backward (dK, dV key-stationary; dQ query-centric), which
    // reads no idx and writes no partial rows; the split backward's first part has nothing to do
    const size_t need = dense_bwd_bytes(dims);
    if (ws_bytes < need)
      return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu the dense backward needs", ws_bytes, need);
    if (parts == dsv::kBwdPrep) return ok();
    unsigned int* status = nullptr;
    if ((s = status_word(&status)) != DSV_OK) return s;
    dsv::BwdParams p{};
    p.d_o = static_cast<const dsv::bf16*>(d_o);
    p.q = static_cast<const dsv::bf16*>(q);
    p.k = static_cast<const dsv::bf16*>(k);
    p.v = static_cast<const dsv::bf16*>(v);
    p.o = static_cast<const dsv::bf16*>(o);
    p.lse = lse;
    p.idx = idx;
    p.dq = static_cast<dsv::bf16*>(dq);
    p.dk = static_cast<dsv::bf16*>(dk);
    p.dv = static_cast<dsv::bf16*>(dv);
    p.BH = dims->B * dims->H;
    p.N = dims->N;
    p.NB = dims->N / dims->block;
    p.topk = dims->k;
    p.d = static_cast<int>(dims->d);
    p.scale = eff_scale(dims);
    p.status = status;
    p.dense = true;
    float* delta = static_cast<float*>(ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = dsv::launch_dense_dkdv(p, delta, st);
    if (e == cudaSuccess) e = dsv::launch_bwd_main_tc(p, dsv::BwdWave{0, p.BH, 0, p.NB, true, true}, 1, st);
    if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "dense backward launch: %s", cudaGetErrorString(e));
    return ok();
  }
  WavePlan plan;
  if (rowptr) {
    plan = WavePlan{dims->B * dims->H, dims->N / 64, false};
    const size_t need = carve(dims, plan.nh, plan.nblk, false, total_pairs).total;
    if (ws_bytes < need)
      return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu the CSR backward needs", ws_bytes, need);
  } else if (!plan_for(dims, ws_bytes, &plan)) {
    return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the minimum %zu", ws_bytes,
                dsv_sparse_attn_bwd_workspace_min(dims));
  }
  if (parts != dsv::kBwdAll && (plan.sub || plan.nh < dims->B * dims->H))
    return fail(DSV_ERR_WORKSPACE, "a split backward needs a workspace that holds every head in one wave "
                "(dsv_sparse_attn_bwd_workspace)");
  unsigned int* status = nullptr;
  if ((s = status_word(&status)) != DSV_OK) return s;

  const Carve c = rowptr ? carve(dims, plan.nh, plan.nblk, false, total_pairs) : carve(dims, plan.nh, plan.nblk, plan.sub);
  uint8_t* base = static_cast<uint8_t*>(ws);
  dsv::BwdParams p;
  p.d_o = static_cast<const dsv::bf16*>(d_o);
  p.q = static_cast<const dsv::bf16*>(q);
  p.k = static_cast<const dsv::bf16*>(k);
  p.v = static_cast<const dsv::bf16*>(v);
  p.o = static_cast<const dsv::bf16*>(o);
  p.lse = lse;
  p.idx = idx;
  p.dq = static_cast<dsv::bf16*>(dq);
  p.dk = static_cast<dsv::bf16*>(dk);
  p.dv = static_cast<dsv::bf16*>(dv);
  p.BH = dims->B * dims->H;
  p.N = dims->N;
  p.NB = dims->N / dims->block;
  p.topk = dims->k;
  p.d = static_cast<int>(dims->d);
  p.scale = eff_scale(dims);
  p.status = status;
  p.colbits = reinterpret_cast<uint32_t*>(base + c.colbits);
  p.colpre = reinterpret_cast<uint32_t*>(base + c.colpre);
  p.count = reinterpret_cast<uint32_t*>(base + c.count);
  p.offsets = reinterpret_cast<int64_t*>(base + c.offsets);
  p.tsum = reinterpret_cast<int64_t*>(base + c.tsum);
  p.lists = reinterpret_cast<int32_t*>(base + c.lists);
  p.partial = reinterpret_cast<dsv::bf16*>(base + c.partial);
  p.partial_dv = reinterpret_cast<dsv::bf16*>(base + c.partial_dv);
  p.acc = plan.sub ? reinterpret_cast<float*>(base + c.acc) : nullptr;
  p.rowptr = rowptr;
  p.order = order;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  std::vector<dsv::BwdWave> waves;
  if (!plan.sub) {
    for (int64_t bh0 = 0; bh0 < p.BH; bh0 += plan.nh)
      waves.push_back(dsv::BwdWave{bh0, plan.nh < p.BH - bh0 ? plan.nh : p.BH - bh0, 0, p.NB, true, true});
  } else {
    for (int64_t bh = 0; bh < p.BH; ++bh)
      for (int64_t b0 = 0; b0 < p.NB; b0 += plan.nblk) {
        const int64_t n = plan.nblk < p.NB - b0 ? plan.nblk : p.NB - b0;
        waves.push_back(dsv::BwdWave{bh, 1, b0, n, b0 == 0, b0 + n == p.NB});
      }
  }
  for (const dsv::BwdWave& w : waves) {
    cudaError_t e = dsv::launch_bwd_wave(p, w, st, parts);
    if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "backward launch: %s", cudaGetErrorString(e));
  }
  return ok();
}

dsv_status dsv_sparse_attn_bwd(const dsv_dims* dims, const void* d_o, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const int32_t* idx, void* dq, void* dk, void* dv,
                               void* ws, size_t ws_bytes, void* stream) {
  return bwd_impl(dims, d_o, q, k, v, o, lse, idx, nullptr, nullptr, 0, dq, dk, dv, ws, ws_bytes, stream);
}

dsv_status dsv_sparse_attn_bwd_prepare(const dsv_dims* dims, const int32_t* idx, void* ws, size_t ws_bytes,
                                       void* stream) {
  return bwd_impl(dims, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, idx, nullptr, nullptr, 0, nullptr,
                  nullptr, nullptr, ws, ws_bytes, stream, dsv::kBwdPrep);
}

dsv_status dsv_sparse_attn_bwd_prepared(const dsv_dims* dims, const void* d_o, const void* q, const void* k,
                                        const void* v, const void* o, const float* lse, const int32_t* idx, void* dq,
                                        void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
  return bwd_impl(dims, d_o, q, k, v, o, lse, idx, nullptr, nullptr, 0, dq, dk, dv, ws, ws_bytes, stream,
                  dsv::kBwdFinish);
}

size_t dsv_sparse_attn_bwd_csr_workspace(const dsv_dims* dims, int64_t total_pairs) {
  if (check_dims(dims, true, false) != DSV_OK || total_pairs < 0) return 0;
  return carve(dims, dims->B * dims->H, dims->N / 64, false, total_pairs).total;
}

dsv_status dsv_sparse_attn_bwd_csr(const dsv_dims* dims, const void* d_o, const void* q, const void* k, const void* v,
                                   const void* o, const float* lse, const int64_t* rowptr, const int32_t* cols,
                                   const int32_t* order, int64_t total_pairs, void* dq, void* dk, void* dv, void* ws,
                                   size_t ws_bytes, void* stream) {
  if (!rowptr) return fail(DSV_ERR_INVALID_ARG, "rowptr is NULL");
  if (total_pairs < 0) return fail(DSV_ERR_INVALID_ARG, "total_pairs must be >= 0");
  if (total_pairs > 0x7fffffffLL) return fail(DSV_ERR_UNSUPPORTED, "total_pairs must fit int32 partial-row indices");
  return bwd_impl(dims, d_o, q, k, v, o, lse, cols, rowptr, order, total_pairs, dq, dk, dv, ws, ws_bytes, stream);
}

dsv_status dsv_profile_enable(int on) {
  if (on && !g_prof_on) {
    if (g_prof_events.empty()) {
      g_prof_events.resize(2 * kProfPool);
      for (auto& e : g_prof_events) {
        cudaError_t err = cudaEventCreate(&e);
        if (err != cudaSuccess) {
          g_prof_events.clear();
          return fail(DSV_ERR_CUDA, "cudaEventCreate: %s", cudaGetErrorString(err));
        }
      }
    }
    g_prof_records.clear();
    g_prof_dropped = 0;
  }
  if (!on) g_prof_records.clear();
  g_prof_on = on != 0;
  return ok();
}

size_t dsv_profile_read(char* buf, size_t buf_bytes) {
  std::map<std::string, std::pair<long long, double>> agg;
  for (const auto& r : g_prof_records) {
    float ms = 0.f;
    if (cudaEventSynchronize(r.end) == cudaSuccess && cudaEventElapsedTime(&ms, r.begin, r.end) == cudaSuccess) {
      auto& a = agg[r.name];
      a.first += 1;
      a.second += ms;
    }
  }
  const bool consume = buf != nullptr && buf_bytes > 0;   // a size query keeps the records
  if (consume) g_prof_records.clear();
  std::string out;
  char line[256];
  for (const auto& kv : agg) {
    snprintf(line, sizeof(line), "%s %lld %.6f\n", kv.first.c_str(), kv.second.first, kv.second.second);
    out += line;
  }
  if (g_prof_dropped) {
    snprintf(line, sizeof(line), "dropped %zu 0\n", g_prof_dropped);
    out += line;
    if (consume) g_prof_dropped = 0;
  }
  if (consume) {
    const size_t n = out.size() < buf_bytes - 1 ? out.size() : buf_bytes - 1;
    memcpy(buf, out.data(), n);
    buf[n] = '\0';
  }
  return out.size() + 1;
}

dsv_status dsv_last_device_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "stream synchronize: %s", cudaGetErrorString(e));
  unsigned int v = 0, zero = 0;
  e = cudaMemcpyFromSymbol(&v, g_dsv_status, sizeof(v));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_dsv_status, &zero, sizeof(zero));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "status word: %s", cudaGetErrorString(e));
  if (v)
    return fail(DSV_ERR_DEVICE_CHECK, "device status 0x%x:%s%s%s", v,
                (v & 1u) ? " an out-of-range or repeated key index" : "",
                (v & 2u) ? " a kernel gave up waiting on its own barrier" : "",
                (v & 4u) ? " a token position outside its axis' table" : "");
  return ok();
}

// ---------------------------------------------------------------- fused AdaLN
static dsv_status check_adaln(const dsv_adaln_dims* d) {
  if (!d) return fail(DSV_ERR_INVALID_ARG, "dims is NULL");
  if (d->B < 1 || d->N < 1) return fail(DSV_ERR_INVALID_ARG, "B and N must be >= 1");
  if (d->D < 8 || d->D > 8192 || d->D % 8)
    return fail(DSV_ERR_INVALID_ARG, "D must be a multiple of 8 in [8, 8192] (got %lld)", (long long)d->D);
  if (d->B * d->N > (1LL << 40)) return fail(DSV_ERR_INVALID_ARG, "B*N too large");
  if (!(d->eps >= 0.f) || d->eps > 3.0e38f) return fail(DSV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return DSV_OK;
}

dsv_status dsv_adaln_fwd(const dsv_adaln_dims* dims, const void* x, const void* scale, const void* shift, void* y,
                         void* stream) {
  dsv_status s = check_adaln(dims);
  if (s != DSV_OK) return s;
  DSV_NEED_PTR(x);
  DSV_NEED_PTR(scale);
  DSV_NEED_PTR(shift);
  DSV_NEED_PTR(y);
  dsv::AdalnParams p{};
  p.x = x;
  p.scale = scale;
  p.shift = shift;
  p.y = y;
  p.B = dims->B;
  p.N = dims->N;
  p.D = dims->D;
  p.eps = dims->eps;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_adaln_fwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "adaln forward launch: %s", cudaGetErrorString(e));
  return ok();
}

size_t dsv_adaln_bwd_workspace(const dsv_adaln_dims* dims) {
  if (check_adaln(dims) != DSV_OK) return 0;
  return up(dsv::adaln_tiling(dims->B, dims->N, dims->D, true).workspace_bytes);
}

dsv_status dsv_adaln_bwd(const dsv_adaln_dims* dims, const void* x, const void* scale, const void* dy, void* dx,
                         float* d_scale, float* d_shift, void* ws, size_t ws_bytes, void* stream) {
  dsv_status s = check_adaln(dims);
  if (s != DSV_OK) return s;
  DSV_NEED_PTR(x);
  DSV_NEED_PTR(scale);
  DSV_NEED_PTR(dy);
  DSV_NEED_PTR(dx);
  DSV_NEED_PTR(d_scale);
  DSV_NEED_PTR(d_shift);
  const size_t need = dsv::adaln_tiling(dims->B, dims->N, dims->D, true).workspace_bytes;
  if (!ws) return fail(DSV_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return fail(DSV_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu needed", ws_bytes, need);
  dsv::AdalnParams p{};
  p.x = x;
  p.scale = scale;
  p.dy = dy;
  p.dx = dx;
  p.d_scale = d_scale;
  p.d_shift = d_shift;
  p.partial = static_cast<float*>(ws);
  p.B = dims->B;
  p.N = dims->N;
  p.D = dims->D;
  p.eps = dims->eps;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_adaln_bwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "adaln backward launch: %s", cudaGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- rotary positions, qk norm
static dsv_status check_rope(const dsv_rope_dims* d, dsv::RopeGeom* g) {
  if (!d) return fail(DSV_ERR_INVALID_ARG, "dims is NULL");
  constexpr int64_t kMax = 0x7fffffffLL;
  if (d->B < 1 || d->H < 1 || d->N < 1) return fail(DSV_ERR_INVALID_ARG, "B, H, N must be >= 1");
  // (64 short of 2^31: a tile's tokens are counted past the last one in 32 bits)
  if (d->B > kMax || d->H > kMax || d->N > kMax || d->B * d->H > kMax || d->B * d->H * d->N > kMax - 64)
    return fail(DSV_ERR_INVALID_ARG, "B*H*N must fit int32 row coordinates (split the heads over calls)");
  if (d->d != 64 && d->d != 128)
    return fail(DSV_ERR_UNSUPPORTED, "head dim d must be 64 or 128 (got %lld)", (long long)d->d);
  if (d->pairing != DSV_PAIRS_INTERLEAVED && d->pairing != DSV_PAIRS_HALVES)
    return fail(DSV_ERR_INVALID_ARG, "pairing must be DSV_PAIRS_INTERLEAVED or DSV_PAIRS_HALVES (got %d)", d->pairing);
  int64_t rotated = 0, entries = 0;
  for (int a = 0; a < 3; ++a) {
    if (d->rot[a] < 0 || d->rot[a] % 2 || d->rot[a] > d->d)
      return fail(DSV_ERR_INVALID_ARG, "rot[%d] must be even and in [0, d] (got %lld)", a, (long long)d->rot[a]);
    if (d->rot[a] > 0 && (d->len[a] < 1 || d->len[a] > kMax))
      return fail(DSV_ERR_INVALID_ARG, "len[%d] must be >= 1 and fit int32 (got %lld)", a, (long long)d->len[a]);
    rotated += d->rot[a];
    g->axis_pairs[a] = static_cast<int>(d->rot[a] / 2);
    g->len[a] = d->rot[a] > 0 ? d->len[a] : 0;
    g->table_off[a] = entries;
    entries += g->len[a] * g->axis_pairs[a];
  }
  if (rotated > d->d) return fail(DSV_ERR_INVALID_ARG, "rot must sum to at most d (got %lld)", (long long)rotated);
  if (entries > kMax) return fail(DSV_ERR_INVALID_ARG, "the table must hold at most 2^31 - 1 (cos, sin) pairs");
  if (d->pairing == DSV_PAIRS_HALVES && rotated % 16)
    return fail(DSV_ERR_UNSUPPORTED, "pairs in halves need rot to sum to a multiple of 16 (got %lld)",
                (long long)rotated);
  if (!(d->eps >= 0.f) || d->eps > 3.0e38f) return fail(DSV_ERR_INVALID_ARG, "eps must be finite and >= 0");
  g->B = d->B;
  g->H = d->H;
  g->N = d->N;
  g->pos_batch = d->pos_batched ? d->N : 0;
  g->pairs = static_cast<int>(rotated / 2);
  return DSV_OK;
}

// A view's strides and the bytes it spans; an output's elements must be distinct.
struct ViewSpan {
  const char *lo, *hi;
};
static dsv_status check_view(const dsv_rope_dims* d, const char* name, const void* p, const dsv_view_strides* s,
                             bool output, dsv::RopeView* view, ViewSpan* span) {
  if (!p) return fail(DSV_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(DSV_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  const int64_t n[3] = {d->B, d->H, d->N};
  int64_t st[3] = {s ? s->b : d->H * d->N * d->d, s ? s->h : d->N * d->d, s ? s->n : d->d};
  int64_t last = d->d - 1;
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) st[i] = 0;   // a single entry: its stride is never used
    if (st[i] < 0 || st[i] % 8 || st[i] > (1LL << 40))
      return fail(DSV_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements in [0, 2^40] (got %lld)", name,
                  (long long)st[i]);
    if (n[i] > (1LL << 48) / (st[i] + 1) || last + (n[i] - 1) * st[i] > (1LL << 48))
      return fail(DSV_ERR_INVALID_ARG, "%s: the view spans too much memory", name);
    last += (n[i] - 1) * st[i];
  }
  if (output) {   // innermost to outermost: each stride must pass what the inner ones span
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (st[order[j]] > st[order[j + 1]]) std::swap(order[j], order[j + 1]);
    int64_t extent = d->d;
    for (int i = 0; i < 3; ++i) {
      const int a = order[i];
      if (n[a] == 1) continue;
      if (st[a] < extent) return fail(DSV_ERR_INVALID_ARG, "%s: the output's strides let its elements overlap", name);
      extent += (n[a] - 1) * st[a];
    }
  }
  view->p = static_cast<dsv::bf16*>(const_cast<void*>(p));
  view->sb = st[0];
  view->sh = st[1];
  view->sn = st[2];
  span->lo = static_cast<const char*>(p);
  span->hi = span->lo + (last + 1) * 2;
  return DSV_OK;
}
static bool apart(const ViewSpan& a, const ViewSpan& b) { return a.hi <= b.lo || b.hi <= a.lo; }

// Whether delta = i st[0] + j st[1] + .. + t has a solution with every |i| < n of its stride and |t| < d, strides
// falling and each past what the smaller ones span (so that only two i of each stride come into question).
static bool reaches(int64_t delta, const int64_t* st, const int64_t* n, int dims, int64_t d) {
  if (dims == 0) return delta > -d && delta < d;
  if (n[0] == 1) return reaches(delta, st + 1, n + 1, dims - 1, d);
  int64_t i = delta / st[0];
  if (delta < 0 && delta % st[0]) --i;
  for (int64_t c = i; c <= i + 1; ++c)
    if (c > -n[0] && c < n[0] && reaches(delta - c * st[0], st + 1, n + 1, dims - 1, d)) return true;
  return false;
}
// Two outputs that share no element: apart, or interleaved views of one layout.
static bool distinct(const dsv_rope_dims* d, const dsv::RopeView& a, const ViewSpan& as, const dsv::RopeView& b,
                     const ViewSpan& bs) {
  if (apart(as, bs)) return true;
  if (a.sb != b.sb || a.sh != b.sh || a.sn != b.sn) return false;
  int64_t st[3] = {a.sb, a.sh, a.sn}, n[3] = {d->B, d->H, d->N};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (st[j] < st[j + 1]) {
        std::swap(st[j], st[j + 1]);
        std::swap(n[j], n[j + 1]);
      }
  return !reaches((bs.lo - as.lo) / 2, st, n, 3, d->d);
}

static size_t rope_table_bytes(const dsv::RopeGeom& g) {
  size_t n = 0;
  for (int a = 0; a < 3; ++a) n += static_cast<size_t>(g.len[a]) * g.axis_pairs[a];
  return n * 2 * sizeof(float);
}

// What a call reads besides its views: the weights, and with anything to rotate the positions and the table.
struct RopeSmall {
  const char* name[4];
  ViewSpan span[4];
  int n = 0;
  void add(const char* what, const void* p, size_t bytes) {
    name[n] = what;
    span[n].lo = static_cast<const char*>(p);
    span[n++].hi = static_cast<const char*>(p) + bytes;
  }
};
static dsv_status check_rope_small(const dsv_rope_dims* d, const dsv::RopeGeom& g, const void* wq, const void* wk,
                                   const int32_t* pos, const float* table, RopeSmall* small) {
  const size_t w_bytes = static_cast<size_t>(d->d) * sizeof(dsv::bf16);
  if (wq) {
    DSV_NEED_PTR(wq);
    small->add("wq", wq, w_bytes);
  }
  if (wk) {
    DSV_NEED_PTR(wk);
    small->add("wk", wk, w_bytes);
  }
  if (!g.pairs) return DSV_OK;
  DSV_NEED_PTR(pos);
  DSV_NEED_PTR(table);
  small->add("pos", pos, static_cast<size_t>(d->pos_batched ? d->B : 1) * d->N * 3 * sizeof(int32_t));
  small->add("table", table, rope_table_bytes(g));
  return DSV_OK;
}
// An output lies over none of them.
static dsv_status apart_from_small(const RopeSmall& small, const char* name, const ViewSpan& out) {
  for (int i = 0; i < small.n; ++i)
    if (!apart(small.span[i], out)) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", name, small.name[i]);
  return DSV_OK;
}

size_t dsv_rope3d_table_bytes(const dsv_rope_dims* dims) {
  dsv::RopeGeom g{};
  if (check_rope(dims, &g) != DSV_OK) return 0;
  return rope_table_bytes(g);
}

dsv_status dsv_rope3d_table(const dsv_rope_dims* dims, const double theta[3], float* table, void* stream) {
  dsv::RopeGeom g{};
  dsv_status s = check_rope(dims, &g);
  if (s != DSV_OK) return s;
  if (!g.pairs) return ok();
  if (!theta) return fail(DSV_ERR_INVALID_ARG, "theta is NULL");
  double th[3] = {1.0, 1.0, 1.0};
  for (int a = 0; a < 3; ++a) {
    if (!g.axis_pairs[a]) continue;
    if (!(theta[a] > 0.0) || theta[a] > 1e300) return fail(DSV_ERR_INVALID_ARG, "theta[%d] must be finite and > 0", a);
    th[a] = theta[a];
  }
  DSV_NEED_PTR(table);
  cudaError_t e = dsv::launch_rope3d_table(g, th, table, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "rope table launch: %s", cudaGetErrorString(e));
  return ok();
}

static dsv_status rope3d_impl(const dsv_rope_dims* dims, const void* x, const dsv_view_strides* xs, const int32_t* pos,
                              const float* table, void* y, const dsv_view_strides* ys, bool backward, void* stream) {
  dsv::RopeParams p{};
  dsv_status s = check_rope(dims, &p.g);
  if (s != DSV_OK) return s;
  ViewSpan a, b;
  if ((s = check_view(dims, backward ? "dy" : "x", x, xs, false, &p.q, &a)) != DSV_OK) return s;
  if ((s = check_view(dims, backward ? "dx" : "y", y, ys, true, &p.qo, &b)) != DSV_OK) return s;
  const bool in_place = p.q.p == p.qo.p && p.q.sb == p.qo.sb && p.q.sh == p.qo.sh && p.q.sn == p.qo.sn;
  if (!in_place && !apart(a, b))
    return fail(DSV_ERR_INVALID_ARG, "the output overlaps the input (in place needs the same pointer and strides)");
  RopeSmall small;
  if ((s = check_rope_small(dims, p.g, nullptr, nullptr, pos, table, &small)) != DSV_OK) return s;
  if ((s = apart_from_small(small, backward ? "dx" : "y", b)) != DSV_OK) return s;
  p.d = static_cast<int>(dims->d);
  p.half = dims->pairing == DSV_PAIRS_HALVES;
  p.backward = backward;
  p.pos = pos;
  p.table = table;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_rope3d(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "rope3d launch: %s", cudaGetErrorString(e));
  return ok();
}

dsv_status dsv_rope3d_fwd(const dsv_rope_dims* dims, const void* x, const dsv_view_strides* x_strides,
                          const int32_t* pos, const float* table, void* y, const dsv_view_strides* y_strides,
                          void* stream) {
  return rope3d_impl(dims, x, x_strides, pos, table, y, y_strides, false, stream);
}

dsv_status dsv_rope3d_bwd(const dsv_rope_dims* dims, const void* dy, const dsv_view_strides* dy_strides,
                          const int32_t* pos, const float* table, void* dx, const dsv_view_strides* dx_strides,
                          void* stream) {
  return rope3d_impl(dims, dy, dy_strides, pos, table, dx, dx_strides, true, stream);
}

dsv_status dsv_qk_norm_rope_fwd(const dsv_rope_dims* dims, const void* q, const void* k, const void* v,
                                const dsv_view_strides strides[3], const void* wq, const void* wk,
                                const int32_t* pos, const float* table, void* q_out, void* k_out, void* v_out,
                                void* stream) {
  dsv::RopeParams p{};
  dsv_status s = check_rope(dims, &p.g);
  if (s != DSV_OK) return s;
  if (!v != !v_out) return fail(DSV_ERR_INVALID_ARG, "v and v_out must both be given, or both be NULL");
  const int nt = v ? 3 : 2;
  const char* in_name[3] = {"q", "k", "v"};
  const char* out_name[3] = {"q_out", "k_out", "v_out"};
  const void* in[3] = {q, k, v};
  void* out[3] = {q_out, k_out, v_out};
  dsv::RopeView* iv[3] = {&p.q, &p.k, &p.v};
  dsv::RopeView* ov[3] = {&p.qo, &p.ko, &p.vo};
  ViewSpan is[3], os[3];
  for (int i = 0; i < nt; ++i) {
    if ((s = check_view(dims, in_name[i], in[i], strides ? strides + i : nullptr, false, iv[i], &is[i])) != DSV_OK)
      return s;
    if ((s = check_view(dims, out_name[i], out[i], nullptr, true, ov[i], &os[i])) != DSV_OK) return s;
  }
  for (int i = 0; i < nt; ++i)
    for (int j = 0; j < nt; ++j) {
      if (!apart(is[i], os[j])) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", out_name[j], in_name[i]);
      if (i < j && !apart(os[i], os[j])) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", out_name[j], out_name[i]);
    }
  RopeSmall small;
  if ((s = check_rope_small(dims, p.g, wq, wk, pos, table, &small)) != DSV_OK) return s;
  for (int i = 0; i < nt; ++i)
    if ((s = apart_from_small(small, out_name[i], os[i])) != DSV_OK) return s;
  p.d = static_cast<int>(dims->d);
  p.half = dims->pairing == DSV_PAIRS_HALVES;
  p.eps = dims->eps;
  p.wq = static_cast<const dsv::bf16*>(wq);
  p.wk = static_cast<const dsv::bf16*>(wk);
  p.pos = pos;
  p.table = table;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_qk_norm_rope_fwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "qk_norm_rope forward launch: %s", cudaGetErrorString(e));
  return ok();
}

static size_t qk_norm_rope_ws(const dsv::RopeGeom& g, const dsv_rope_dims* d) {
  const dsv::RopeGeom plan = dsv::rope_plan(g, static_cast<int>(d->d), true);
  const int64_t rows = dsv::rope_bwd_ctas(plan);
  return up(static_cast<size_t>(rows) * 2 * d->d * sizeof(float));
}

size_t dsv_qk_norm_rope_bwd_workspace(const dsv_rope_dims* dims) {
  dsv::RopeGeom g{};
  if (check_rope(dims, &g) != DSV_OK) return 0;
  return qk_norm_rope_ws(g, dims);
}

dsv_status dsv_qk_norm_rope_bwd(const dsv_rope_dims* dims, const void* d_q_out, const void* d_k_out,
                                const void* d_v_out, const void* q, const void* k, const dsv_view_strides strides[2],
                                const void* wq, const void* wk, const int32_t* pos, const float* table, void* dq,
                                void* dk, void* dv, const dsv_view_strides d_strides[3], float* dwq, float* dwk,
                                void* ws, size_t ws_bytes, void* stream) {
  dsv::RopeParams p{};
  dsv_status s = check_rope(dims, &p.g);
  if (s != DSV_OK) return s;
  if (!d_v_out != !dv) return fail(DSV_ERR_INVALID_ARG, "d_v_out and dv must both be given, or both be NULL");
  const int nt = dv ? 3 : 2;
  const char* in_name[5] = {"d_q_out", "d_k_out", "q", "k", "d_v_out"};
  const void* in[5] = {d_q_out, d_k_out, q, k, d_v_out};
  dsv::RopeView* iv[5] = {&p.qo, &p.ko, &p.q, &p.k, &p.vo};
  const char* out_name[3] = {"dq", "dk", "dv"};
  void* out[3] = {dq, dk, dv};
  dsv::RopeView* ov[3] = {&p.dq, &p.dk, &p.dv};
  ViewSpan is[5], os[3];
  const int ni = dv ? 5 : 4;
  for (int i = 0; i < ni; ++i) {
    const dsv_view_strides* st = (i == 2 || i == 3) && strides ? strides + (i - 2) : nullptr;
    if ((s = check_view(dims, in_name[i], in[i], st, false, iv[i], &is[i])) != DSV_OK) return s;
  }
  for (int i = 0; i < nt; ++i)
    if ((s = check_view(dims, out_name[i], out[i], d_strides ? d_strides + i : nullptr, true, ov[i], &os[i])) !=
        DSV_OK)
      return s;
  for (int j = 0; j < nt; ++j) {
    for (int i = 0; i < ni; ++i)
      if (!apart(is[i], os[j])) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", out_name[j], in_name[i]);
    for (int i = 0; i < j; ++i)   // the views of a packed gradient interleave
      if (!distinct(dims, *ov[i], os[i], *ov[j], os[j]))
        return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", out_name[j], out_name[i]);
  }
  if (dwq) DSV_NEED_PTR(dwq);
  if (dwk) DSV_NEED_PTR(dwk);
  RopeSmall small;
  if ((s = check_rope_small(dims, p.g, wq, wk, pos, table, &small)) != DSV_OK) return s;
  for (int i = 0; i < nt; ++i)
    if ((s = apart_from_small(small, out_name[i], os[i])) != DSV_OK) return s;
  if (dwq || dwk) {
    const size_t need = qk_norm_rope_ws(p.g, dims);
    if (!ws) return fail(DSV_ERR_WORKSPACE, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(ws) % kAlign)
      return fail(DSV_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < need)
      return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu needed", ws_bytes, need);
    const char* sum_name[3] = {"dwq", "dwk", "ws"};
    const void* sum[3] = {dwq, dwk, ws};
    ViewSpan ss[3];
    for (int j = 0; j < 3; ++j) {
      ss[j].lo = static_cast<const char*>(sum[j]);
      ss[j].hi = ss[j].lo + (!sum[j] ? 0 : j < 2 ? dims->d * 4 : static_cast<int64_t>(need));
      for (int i = 0; i < ni + nt + j && sum[j]; ++i) {
        const ViewSpan& t = i < ni ? is[i] : i < ni + nt ? os[i - ni] : ss[i - ni - nt];
        const char* name = i < ni ? in_name[i] : i < ni + nt ? out_name[i - ni] : sum_name[i - ni - nt];
        if (!apart(t, ss[j])) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", sum_name[j], name);
      }
      if (sum[j] && (s = apart_from_small(small, sum_name[j], ss[j])) != DSV_OK) return s;
    }
  }
  p.d = static_cast<int>(dims->d);
  p.half = dims->pairing == DSV_PAIRS_HALVES;
  p.eps = dims->eps;
  p.wq = static_cast<const dsv::bf16*>(wq);
  p.wk = static_cast<const dsv::bf16*>(wk);
  p.dwq = dwq;
  p.dwk = dwk;
  p.partial = static_cast<float*>(ws);
  p.pos = pos;
  p.table = table;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_qk_norm_rope_bwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "qk_norm_rope backward launch: %s", cudaGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- gated feed-forward
static dsv_status check_ffn(const dsv_ffn_dims* d) {
  if (!d) return fail(DSV_ERR_INVALID_ARG, "dims is NULL");
  if (d->M < 1 || d->M > 0x7fffffffLL - 256) return fail(DSV_ERR_INVALID_ARG, "M must be in [1, 2^31 - 257] (got %lld)", (long long)d->M);
  if (d->D < 8 || d->D % 8 || d->D > (1 << 20) || d->F < 8 || d->F % 8 || d->F > (1 << 20))
    return fail(DSV_ERR_INVALID_ARG, "D and F must be multiples of 8 in [8, 2^20] (got %lld, %lld)", (long long)d->D,
                (long long)d->F);
  if (d->act != DSV_ACT_SILU && d->act != DSV_ACT_GELU_TANH)
    return fail(DSV_ERR_INVALID_ARG, "act must be DSV_ACT_SILU or DSV_ACT_GELU_TANH (got %d)", d->act);
  return DSV_OK;
}

// Checks a call's tensors: not NULL, aligned, no output over an input or another output.
struct NamedSpan {
  const char* name;
  const void* p;
  int64_t elements;
};
static dsv_status check_spans(const NamedSpan* in, int n_in, const NamedSpan* out, int n_out) {
  auto span = [](const NamedSpan& t) {
    const char* lo = static_cast<const char*>(t.p);
    return ViewSpan{lo, lo + 2 * t.elements};
  };
  for (int i = 0; i < n_in + n_out; ++i) {
    const NamedSpan& t = i < n_in ? in[i] : out[i - n_in];
    if (!t.p) return fail(DSV_ERR_INVALID_ARG, "%s is NULL", t.name);
    if (!aligned16(t.p)) return fail(DSV_ERR_INVALID_ARG, "%s is not 16-byte aligned", t.name);
  }
  for (int j = 0; j < n_out; ++j)
    for (int i = 0; i < n_in + j; ++i) {
      const NamedSpan& t = i < n_in ? in[i] : out[i - n_in];
      if (!apart(span(t), span(out[j]))) return fail(DSV_ERR_INVALID_ARG, "%s overlaps %s", out[j].name, t.name);
    }
  return DSV_OK;
}

static dsv_status check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(DSV_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return fail(DSV_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < need) return fail(DSV_ERR_WORKSPACE, "workspace of %zu bytes is below the %zu needed", ws_bytes, need);
  return DSV_OK;
}

size_t dsv_ffn_gated_fwd_workspace(const dsv_ffn_dims* dims) {
  if (check_ffn(dims) != DSV_OK) return 0;
  return up(dsv::ffn_fwd_workspace(dims->M, dims->D, dims->F));
}

dsv_status dsv_ffn_gated_fwd(const dsv_ffn_dims* dims, const void* x, const void* w_gate, const void* w_up, void* h,
                             void* ws, size_t ws_bytes, void* stream) {
  dsv_status s = check_ffn(dims);
  if (s != DSV_OK) return s;
  const int64_t M = dims->M, D = dims->D, F = dims->F;
  const size_t need = up(dsv::ffn_fwd_workspace(M, D, F));
  if (need && (s = check_workspace(ws, ws_bytes, need)) != DSV_OK) return s;
  const NamedSpan in[3] = {{"x", x, M * D}, {"w_gate", w_gate, F * D}, {"w_up", w_up, F * D}};
  const NamedSpan out[2] = {{"h", h, M * F}, {"ws", ws, static_cast<int64_t>(need / 2)}};
  if ((s = check_spans(in, 3, out, need ? 2 : 1)) != DSV_OK) return s;
  dsv::FfnParams p{};
  p.M = M;
  p.D = D;
  p.F = F;
  p.act = dims->act;
  p.x = static_cast<const dsv::bf16*>(x);
  p.w_gate = static_cast<const dsv::bf16*>(w_gate);
  p.w_up = static_cast<const dsv::bf16*>(w_up);
  p.h = static_cast<dsv::bf16*>(h);
  p.ws = ws;
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_ffn_gated_fwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "ffn forward launch: %s", cudaGetErrorString(e));
  return ok();
}

size_t dsv_ffn_gated_bwd_workspace(const dsv_ffn_dims* dims) {
  if (check_ffn(dims) != DSV_OK) return 0;
  return up(dsv::ffn_bwd_workspace(dims->M, dims->D, dims->F));
}

dsv_status dsv_ffn_gated_bwd(const dsv_ffn_dims* dims, const void* dh, const void* x, const void* w_gate,
                             const void* w_up, void* dx, void* dw_gate, void* dw_up, void* ws, size_t ws_bytes,
                             void* stream) {
  dsv_status s = check_ffn(dims);
  if (s != DSV_OK) return s;
  const int64_t M = dims->M, D = dims->D, F = dims->F;
  const size_t need = dsv_ffn_gated_bwd_workspace(dims);
  const NamedSpan in[4] = {{"dh", dh, M * F}, {"x", x, M * D}, {"w_gate", w_gate, F * D}, {"w_up", w_up, F * D}};
  const NamedSpan out[4] = {{"dx", dx, M * D}, {"dw_gate", dw_gate, F * D}, {"dw_up", dw_up, F * D},
                            {"ws", ws, static_cast<int64_t>(need / 2)}};
  if ((s = check_workspace(ws, ws_bytes, need)) != DSV_OK) return s;
  if ((s = check_spans(in, 4, out, 4)) != DSV_OK) return s;
  dsv::FfnParams p{};
  p.M = M;
  p.D = D;
  p.F = F;
  p.act = dims->act;
  p.x = static_cast<const dsv::bf16*>(x);
  p.w_gate = static_cast<const dsv::bf16*>(w_gate);
  p.w_up = static_cast<const dsv::bf16*>(w_up);
  p.dh = static_cast<const dsv::bf16*>(dh);
  p.ws = ws;
  p.dx = static_cast<dsv::bf16*>(dx);
  p.dw_gate = static_cast<dsv::bf16*>(dw_gate);
  p.dw_up = static_cast<dsv::bf16*>(dw_up);
  if ((s = status_word(&p.status)) != DSV_OK) return s;
  cudaError_t e = dsv::launch_ffn_gated_bwd(p, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "ffn backward launch: %s", cudaGetErrorString(e));
  return ok();
}

// ---------------------------------------------------------------- backward with library-held scratch
// For callers that cannot allocate device memory (see include/dsv.h).  The scratch is a
// fixed device array; host code only ever uses the address looked up per device below.
}  // extern "C"

namespace {
static __device__ __align__(256) unsigned char g_noalloc_scratch[DSV_NOALLOC_SCRATCH_BYTES];
// Per-device address of g_noalloc_scratch, looked up once per device.  Several host threads may
// race on the first look-up; they all find the same address, and the atomic makes the store and
// the loads well defined.
std::atomic<void*> g_noalloc_ptr[kMaxDevices];
}  // namespace

extern "C" {

dsv_status dsv_sparse_attn_bwd_noalloc(const dsv_dims* dims, const void* d_o, const void* q, const void* k,
                                       const void* v, const void* o, const float* lse, const int32_t* idx,
                                       void* dq, void* dk, void* dv, void* stream) {
  dsv_status s = check_dims(dims, true, false);
  if (s != DSV_OK) return s;
  const size_t need = dsv_sparse_attn_bwd_workspace_min(dims);
  if (need > DSV_NOALLOC_SCRATCH_BYTES)
    return fail(DSV_ERR_WORKSPACE,
                "this backward needs at least %zu bytes of scratch but the no-allocation variant holds %zu; "
                "call dsv_sparse_attn_bwd with a caller workspace instead",
                need, static_cast<size_t>(DSV_NOALLOC_SCRATCH_BYTES));
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(DSV_ERR_CUDA, "device ordinal %d out of range", dev);
  void* scratch = g_noalloc_ptr[dev].load(std::memory_order_acquire);
  if (!scratch) {  // set-up, once per device, with that device current
    e = cudaGetSymbolAddress(&scratch, g_noalloc_scratch);
    if (e != cudaSuccess) return fail(DSV_ERR_CUDA, "cudaGetSymbolAddress(scratch): %s", cudaGetErrorString(e));
    g_noalloc_ptr[dev].store(scratch, std::memory_order_release);
  }
  // Every word of the scratch that the backward reads in a wave is written earlier in the same
  // wave (the bitmap kernel writes all of its words, zeros included; the scans, lists, partial
  // rows and the accumulator are written before they are read), so what an earlier call left
  // there is never used and nothing needs clearing.
  return dsv_sparse_attn_bwd(dims, d_o, q, k, v, o, lse, idx, dq, dk, dv, scratch, DSV_NOALLOC_SCRATCH_BYTES,
                             stream);
}

}  // extern "C"
