// extern "C" entry points declared in include/mm.h.
//
// Each entry point validates its arguments on the host (plan.cpp) before any
// HIP call, checks once per device that it runs on gfx950, then enqueues the
// kernels on the caller's stream without synchronising.
#include <hip/hip_runtime.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "../../include/mm.h"
#include "kernels.h"
#include "plan.h"

using namespace qsg;

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_device_ok[kMaxDevices];   // 0 unknown, 1 gfx950, -1 other

int check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return MM_ERR_HIP;
  if (dev < 0 || dev >= kMaxDevices) return MM_ERR_DEVICE;
  int state = g_device_ok[dev].load(std::memory_order_relaxed);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return MM_ERR_HIP;
    state = strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    g_device_ok[dev].store(state, std::memory_order_relaxed);
  }
  return state == 1 ? MM_OK : MM_ERR_DEVICE;
}

int hip_status(hipError_t e) { return e == hipSuccess ? MM_OK : MM_ERR_HIP; }

// Workspace of mm_mul_mat_q4_0_f32_noalloc: a file-scope device array, one
// copy per GPU, held until the process ends.  In host code `scratch` names a
// host-side stand-in, not device memory: its device address on the current
// GPU comes from hipGetSymbolAddress, looked up once per device (with that
// device current) and kept in g_scratch_ptr; only that pointer is ever
// passed to a kernel.
static __device__ __align__(256) uint8_t scratch[kNoAllocScratchBytes];
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// Device address of `scratch` on the current device (looked up on the first
// call on each device), or NULL with *st set on failure.
void* scratch_ptr(int* st) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) { *st = MM_ERR_HIP; return nullptr; }
  if (dev < 0 || dev >= kMaxDevices) { *st = MM_ERR_DEVICE; return nullptr; }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) {
      *st = MM_ERR_HIP;
      return nullptr;
    }
    g_scratch_ptr[dev] = ptr;
  }
  *st = MM_OK;
  return g_scratch_ptr[dev];
}

Q4Args q4_args(const Plan& p, const void* src0, float* dst, int32_t* dots, int64_t M,
               int64_t N, int64_t K, int64_t n0, int64_t n1, void* ws) {
  uint8_t* base = (uint8_t*)ws;
  Q4Args a;
  a.w = (const uint8_t*)src0;
  a.aq = (const int8_t*)(base + p.off_aq);
  a.ad = (const float*)(base + p.off_ad);
  a.ab = (const int32_t*)(base + p.off_ab);
  a.sq = p.off_sq ? (const uint8_t*)(base + p.off_sq) : nullptr;
  a.ss = p.off_ss ? (const float*)(base + p.off_ss) : nullptr;
  a.sk_phases = (int)p.sk_phases;
  a.sq_bytes = (int)(p.sk_rows * p.sk_phases * 256);
  a.ss_bytes = (int)(p.sk_rows * p.sk_phases * 32);
  a.dst = dst;
  a.part = p.split > 1 ? (float*)(base + p.off_part) : nullptr;
  a.M = (int)M; a.N = (int)N; a.K = (int)K;
  a.dots = dots; a.n0 = (int)n0; a.n1 = (int)n1;
  return a;
}

// INIT: src1 -> Q8_0 wdata in the workspace.
int q4_init(const Plan& p, const float* src1, int64_t M, int64_t K, void* ws, hipStream_t s) {
  uint8_t* base = (uint8_t*)ws;
  if (p.off_sq)
    return hip_status(launch_quantize_q8_0_skinny(
        src1, M, K, (int8_t*)(base + p.off_aq), (float*)(base + p.off_ad),
        (int32_t*)(base + p.off_ab), base + p.off_sq, (float*)(base + p.off_ss), p.sk_rows,
        p.sk_phases, p.mt == 8, s));
  return hip_status(launch_quantize_q8_0(src1, M, K, nullptr, (int8_t*)(base + p.off_aq),
                                         (float*)(base + p.off_ad), (int32_t*)(base + p.off_ab), s));
}

Q4Mats single_mat(const void* src0, float* dst, int64_t N) {
  Q4Mats m;
  for (int i = 0; i < kMaxGroup; ++i) { m.w[i] = nullptr; m.dst[i] = nullptr; }
  for (int i = 0; i <= kMaxGroup; ++i) m.row0[i] = (int)N;
  m.w[0] = (const uint8_t*)src0;
  m.dst[0] = dst;
  m.row0[0] = 0;
  m.count = 1;
  return m;
}

// The product kernel (x != NULL: INIT fused), then the split-K reduction.
int q4_product(const Plan& p, const Q4Args& a, const float* x, hipStream_t s) {
  // Q8_0 weights have no staged-chunk fallback for the skinny plan
  if (p.type == MM_TYPE_Q8_0 && p.kind == KK_Q4_MMA && !(a.sq && q4_skinny_ok(a.K, a.w)))
    return MM_ERR_ARG;
  hipError_t e = p.kind == KK_Q4_NARROW    ? launch_q4_narrow(p, a, single_mat(a.w, a.dst, a.N), x, s)
                 : p.kind == KK_Q4_MMA     ? (a.sq && q4_skinny_ok(a.K, a.w) ? launch_q4_skinny(p, a, s)
                                                                       : launch_q4_mma(p, a, s))
                 : p.kind == KK_Q4R_SKINNY ? launch_q4r_skinny(p, a, s)
                                           : launch_q4_wide_i8(p, a, s);
  if (e == hipSuccess && p.split > 1)
    e = launch_splitk_reduce(a.part, a.dst, (int64_t)a.M * a.N, p.split, s);
  return hip_status(e);
}

int run_q4_0(const Plan& p, const void* src0, const float* src1, float* dst, int32_t* dots,
             int64_t M, int64_t N, int64_t K, int64_t n0, int64_t n1, void* ws, hipStream_t s) {
  const Q4Args a = q4_args(p, src0, dst, dots, M, N, K, n0, n1, ws);
  if (p.kind == KK_Q4_NARROW && p.fuse) return q4_product(p, a, src1, s);
  const int st = q4_init(p, src1, M, K, ws, s);
  if (st != MM_OK) return st;
  return q4_product(p, a, nullptr, s);
}

// Skinny F16 / F32 product: the MFMA kernel, one launch; operands that it
// cannot take (not 16-byte aligned, K off its step) take the narrow kernel's
// plan for the same shape instead.
int run_f_mma(const Plan& p, int type, const void* src0, const float* src1, float* dst,
              int64_t M, int64_t N, int64_t K, hipStream_t s) {
  if (!f_mma_ok(type, src0, src1, K)) {
    Plan q;
    const int st = make_plan(type, M, N, K, 1, &q);
    if (st != MM_OK) return st;
    return hip_status(launch_f_narrow(q, type, src0, src1, dst, (int)M, (int)N, (int)K, s));
  }
  return hip_status(launch_f_mma(p, type, src0, src1, dst, (int)M, (int)N, (int)K, s));
}

int mul_mat(int type, const void* src0, const float* src1, float* dst, int32_t* dots,
            int64_t M, int64_t N, int64_t K, int64_t n0, int64_t n1, int variant, void* ws,
            size_t ws_bytes, void* stream) {
  Plan p;
  int st = make_plan(type, M, N, K, variant, &p);
  if (st != MM_OK) return st;
  st = validate_mul_mat(type, src0, src1, dst, M, N, K, ws, ws_bytes, p);
  if (st != MM_OK) return st;
  if (p.kind == KK_NONE) return MM_OK;
  st = check_device();
  if (st != MM_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  switch (p.kind) {
    case KK_ZERO: return hip_status(launch_zero(dst, M * N, s));
    case KK_Q4_NARROW:
    case KK_Q4_MMA:
    case KK_Q4R_SKINNY:
    case KK_Q4_WIDE: return run_q4_0(p, src0, src1, dst, dots, M, N, K, n0, n1, ws, s);
    case KK_F_NARROW:
      return hip_status(launch_f_narrow(p, type, src0, src1, dst, (int)M, (int)N, (int)K, s));
    case KK_F_MMA: return run_f_mma(p, type, src0, src1, dst, M, N, K, s);
    case KK_F16_WIDE:
      return hip_status(launch_f16_wide(p, (const uint16_t*)src0, src1, dst, (int)M, (int)N,
                                        (int)K, ws, s));
    default: return MM_ERR_ARG;
  }
}

int quantize(int out_type, const float* x, void* y, int64_t nrows, int64_t k, void* stream) {
  int st = validate_quantize(out_type, x, y, nrows, k);
  if (st != MM_OK) return st;
  if (nrows == 0 || k == 0) return MM_OK;
  st = check_device();
  if (st != MM_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  if (out_type == MM_TYPE_Q4_0) return hip_status(launch_quantize_q4_0(x, nrows, k, (uint8_t*)y, s));
  return hip_status(launch_quantize_q8_0(x, nrows, k, (uint8_t*)y, nullptr, nullptr, nullptr, s));
}

// Q4_0 <-> repacked Q4_0: plain rows are 2-byte aligned, the repacked
// buffer 16-byte aligned; the two must not overlap.
int repack(const void* src, void* dst, int64_t N, int64_t K, bool to_repacked, void* stream) {
  const int64_t rb = repacked_bytes(N, K);
  if (rb < 0) return MM_ERR_SHAPE;
  if (N == 0 || K == 0) return MM_OK;
  if (!src || !dst) return MM_ERR_NULL;
  const void* plain = to_repacked ? src : dst;
  const void* packed = to_repacked ? dst : src;
  if ((uintptr_t)plain % 2 || (uintptr_t)packed % 16) return MM_ERR_ALIGN;
  const uintptr_t p0 = (uintptr_t)plain, p1 = (uintptr_t)packed;
  const size_t pb = (size_t)N * (size_t)row_bytes(MM_TYPE_Q4_0, K);
  if (p0 < p1 + (size_t)rb && p1 < p0 + pb) return MM_ERR_ALIAS;
  const int st = check_device();
  if (st != MM_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  return hip_status(to_repacked
                        ? launch_repack_q4_0((const uint8_t*)src, (uint8_t*)dst, N, K, s)
                        : launch_unpack_q4_0((const uint8_t*)src, (uint8_t*)dst, N, K, s));
}

// Product with e4m3 weights: src1 as f32 (x) or as codes and scales (a, asc).
int f8_product(const void* src0, const float* scale0, const float* x, const void* a,
               const float* asc, float* dst, int64_t M, int64_t N, int64_t K, void* ws,
               size_t ws_bytes, void* stream, bool given) {
  F8Plan p;
  int st = make_f8_plan(M, N, K, given, &p);
  if (st != MM_OK) return st;
  st = validate_f8(src0, scale0, given ? a : (const void*)x, asc, dst, M, N, K, given, ws, ws_bytes, p);
  if (st != MM_OK) return st;
  if (p.kind == F8_NONE) return MM_OK;
  st = check_device();
  if (st != MM_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  if (p.kind == F8_ZERO) return hip_status(launch_zero(dst, M * N, s));
  return hip_status(launch_f8_product(p, (const uint8_t*)src0, scale0, x, (const uint8_t*)a, asc,
                                      dst, (int)M, (int)N, (int)K, ws, s));
}

// Product with MXFP4 weights: src1 as f32 (x) or as codes and scales (a, asc).
int mx4_product(const void* src0, const void* scale0, const float* x, const void* a, const void* asc,
                float* dst, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream,
                bool given) {
  Mx4Plan p;
  int st = make_mx4_plan(M, N, K, given, &p);
  if (st != MM_OK) return st;
  st = validate_mx4(src0, scale0, given ? a : (const void*)x, asc, dst, M, N, K, given, ws, ws_bytes, p);
  if (st != MM_OK) return st;
  if (p.kind == MX4_NONE) return MM_OK;
  st = check_device();
  if (st != MM_OK) return st;
  hipStream_t s = (hipStream_t)stream;
  if (p.kind == MX4_ZERO) return hip_status(launch_zero(dst, M * N, s));
  return hip_status(launch_mx4_product(p, (const uint8_t*)src0, (const uint8_t*)scale0, x,
                                       (const uint8_t*)a, (const uint8_t*)asc, dst, (int)M, (int)N,
                                       (int)K, ws, s));
}

}  // namespace

// Status codes travel as int inside the library; the C entry points return
// them as the header's enum.
inline mm_status as_status(int st) { return static_cast<mm_status>(st); }

extern "C" {

mm_status mm_quantize_q4_0(const float* x, void* y, int64_t nrows, int64_t k, void* stream) {
  return as_status(quantize(MM_TYPE_Q4_0, x, y, nrows, k, stream));
}

mm_status mm_quantize_q8_0(const float* x, void* y, int64_t nrows, int64_t k, void* stream) {
  return as_status(quantize(MM_TYPE_Q8_0, x, y, nrows, k, stream));
}

mm_status mm_mul_mat_q4_0_f32(const void* src0, const float* src1, float* dst,
                              int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                              void* stream) {
  return as_status(
      mul_mat(MM_TYPE_Q4_0, src0, src1, dst, nullptr, M, N, K, 0, 0, 0, ws, ws_bytes, stream));
}

mm_status mm_mul_mat_q4_0_f32_noalloc(const void* src0, const float* src1, float* dst, int64_t M,
                                      int64_t N, int64_t K, void* stream) {
  // the plan first: a shape whose workspace does not fit the array is
  // rejected before any HIP call
  Plan p;
  int st = make_plan(MM_TYPE_Q4_0, M, N, K, 0, &p);
  if (st != MM_OK) return as_status(st);
  if (p.ws_bytes > kNoAllocScratchBytes) return MM_ERR_WORKSPACE;
  if (p.kind == KK_NONE) return MM_OK;
  st = validate_mul_mat(MM_TYPE_Q4_0, src0, src1, dst, M, N, K, nullptr, 0, p, STAGE_ALL,
                        /*check_ws=*/false);
  if (st != MM_OK) return as_status(st);
  st = check_device();
  if (st != MM_OK) return as_status(st);
  void* ws = scratch_ptr(&st);
  if (!ws) return as_status(st);
  return as_status(mul_mat(MM_TYPE_Q4_0, src0, src1, dst, nullptr, M, N, K, 0, 0, 0, ws,
                 kNoAllocScratchBytes, stream));
}

mm_status mm_mul_mat_q8_0_f32(const void* src0, const float* src1, float* dst,
                              int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                              void* stream) {
  return as_status(
      mul_mat(MM_TYPE_Q8_0, src0, src1, dst, nullptr, M, N, K, 0, 0, 0, ws, ws_bytes, stream));
}

mm_status mm_mul_mat_q4_0r_f32(const void* src0r, const float* src1, float* dst,
                               int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                               void* stream) {
  return as_status(
      mul_mat(MM_TYPE_Q4_0R, src0r, src1, dst, nullptr, M, N, K, 0, 0, 0, ws, ws_bytes, stream));
}

int64_t mm_repacked_q4_0_bytes(int64_t N, int64_t K) { return repacked_bytes(N, K); }

mm_status mm_repack_q4_0(const void* src0, void* dst, int64_t N, int64_t K, void* stream) {
  return as_status(repack(src0, dst, N, K, /*to_repacked=*/true, stream));
}

mm_status mm_unpack_q4_0(const void* src0r, void* dst, int64_t N, int64_t K, void* stream) {
  return as_status(repack(src0r, dst, N, K, /*to_repacked=*/false, stream));
}

mm_status mm_mul_mat_f16_f32(const uint16_t* src0, const float* src1, float* dst, int64_t M,
                             int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream) {
  return as_status(
      mul_mat(MM_TYPE_F16, src0, src1, dst, nullptr, M, N, K, 0, 0, 0, ws, ws_bytes, stream));
}

mm_status mm_quantize_f8(const float* x, void* codes, float* scales, int64_t nrows, int64_t k,
                         int block_rows, void* stream) {
  int st = validate_f8_quantize(x, codes, scales, nrows, k, block_rows);
  if (st != MM_OK || nrows == 0 || k == 0) return as_status(st);
  st = check_device();
  if (st != MM_OK) return as_status(st);
  return as_status(hip_status(
      launch_f8_quantize(x, (uint8_t*)codes, scales, nrows, k, block_rows, (hipStream_t)stream)));
}

mm_status mm_mul_mat_f8_f32(const void* src0, const float* scale0, const float* src1, float* dst,
                            int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                            void* stream) {
  return as_status(f8_product(src0, scale0, src1, nullptr, nullptr, dst, M, N, K, ws, ws_bytes,
                              stream, false));
}

mm_status mm_mul_mat_f8_f8(const void* src0, const float* scale0, const void* src1,
                           const float* scale1, float* dst, int64_t M, int64_t N, int64_t K,
                           void* ws, size_t ws_bytes, void* stream) {
  return as_status(f8_product(src0, scale0, nullptr, src1, scale1, dst, M, N, K, ws, ws_bytes,
                              stream, true));
}

size_t mm_mul_mat_f8_workspace_size(int64_t M, int64_t N, int64_t K, int src1_quantized) {
  F8Plan p;
  if (make_f8_plan(M, N, K, src1_quantized != 0, &p) != MM_OK) return 0;
  return p.ws_bytes;
}

mm_status mm_quantize_mxfp4(const float* x, void* codes, void* scales, int64_t nrows, int64_t k,
                            void* stream) {
  int st = validate_mx4_quantize(x, codes, scales, nrows, k);
  if (st != MM_OK || nrows == 0 || k == 0) return as_status(st);
  st = check_device();
  if (st != MM_OK) return as_status(st);
  return as_status(hip_status(launch_mx4_quantize(x, (uint8_t*)codes, (uint8_t*)scales, nrows, k,
                                                  (hipStream_t)stream)));
}

mm_status mm_dequantize_mxfp4(const void* codes, const void* scales, float* y, int64_t nrows, int64_t k,
                              void* stream) {
  int st = validate_mx4_quantize(y, codes, scales, nrows, k);
  if (st != MM_OK || nrows == 0 || k == 0) return as_status(st);
  st = check_device();
  if (st != MM_OK) return as_status(st);
  return as_status(hip_status(launch_mx4_dequantize((const uint8_t*)codes, (const uint8_t*)scales, y,
                                                    nrows, k, (hipStream_t)stream)));
}

mm_status mm_mul_mat_mxfp4_f32(const void* src0, const void* scale0, const float* src1, float* dst,
                               int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                               void* stream) {
  return as_status(mx4_product(src0, scale0, src1, nullptr, nullptr, dst, M, N, K, ws, ws_bytes,
                               stream, false));
}

mm_status mm_mul_mat_mxfp4_mxfp4(const void* src0, const void* scale0, const void* src1,
                                 const void* scale1, float* dst, int64_t M, int64_t N, int64_t K,
                                 void* ws, size_t ws_bytes, void* stream) {
  return as_status(mx4_product(src0, scale0, nullptr, src1, scale1, dst, M, N, K, ws, ws_bytes,
                               stream, true));
}

size_t mm_mul_mat_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K, int src1_quantized) {
  Mx4Plan p;
  if (make_mx4_plan(M, N, K, src1_quantized != 0, &p) != MM_OK) return 0;
  return p.ws_bytes;
}

mm_status mm_mul_mat_f32(const float* src0, const float* src1, float* dst,
                         int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                         void* stream) {
  return as_status(
      mul_mat(MM_TYPE_F32, src0, src1, dst, nullptr, M, N, K, 0, 0, 0, ws, ws_bytes, stream));
}

mm_status mm_q4_0_init(const float* src1, void* ws, int64_t M, int64_t N, int64_t K,
                       size_t ws_bytes, void* stream) {
  Plan p;
  int st = make_plan(MM_TYPE_Q4_0, M, N, K, 0, &p);
  if (st != MM_OK) return as_status(st);
  st = validate_mul_mat(MM_TYPE_Q4_0, nullptr, src1, nullptr, M, N, K, ws, ws_bytes, p, STAGE_INIT);
  if (st != MM_OK) return as_status(st);
  if (p.kind == KK_NONE || p.kind == KK_ZERO) return MM_OK;
  st = check_device();
  if (st != MM_OK) return as_status(st);
  return as_status(q4_init(p, src1, M, K, ws, (hipStream_t)stream));
}

mm_status mm_q4_0_compute(const void* src0, float* dst, int64_t M, int64_t N, int64_t K,
                          const void* ws, size_t ws_bytes, void* stream) {
  Plan p;
  int st = make_plan(MM_TYPE_Q4_0, M, N, K, 0, &p);
  if (st != MM_OK) return as_status(st);
  st = validate_mul_mat(MM_TYPE_Q4_0, src0, nullptr, dst, M, N, K, ws, ws_bytes, p, STAGE_COMPUTE);
  if (st != MM_OK) return as_status(st);
  if (p.kind == KK_NONE) return MM_OK;
  st = check_device();
  if (st != MM_OK) return as_status(st);
  hipStream_t s = (hipStream_t)stream;
  if (p.kind == KK_ZERO) return as_status(hip_status(launch_zero(dst, M * N, s)));
  return as_status(
      q4_product(p, q4_args(p, src0, dst, nullptr, M, N, K, 0, 0, (void*)ws), nullptr, s));
}

namespace {

bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

// Plan of a grouped product: narrow -> one launch over the concatenated rows
// (no split); wide -> one plan per matrix, sharing the wdata at the front of
// the workspace.  Returns the workspace size through *ws.
int group_plan(int count, const int64_t* Ns, int64_t M, int64_t K, Plan* whole, int64_t* ntot,
               size_t* ws) {
  if (count < 1 || count > kMaxGroup) return MM_ERR_ARG;
  if (!Ns) return MM_ERR_NULL;
  int64_t tot = 0;
  for (int i = 0; i < count; ++i) {
    if (Ns[i] < 0) return MM_ERR_SHAPE;
    tot += Ns[i];
  }
  if (tot > 0x7fffffff) return MM_ERR_SHAPE;
  *ntot = tot;
  int st = make_plan(MM_TYPE_Q4_0, M, tot, K, 0, whole, /*allow_split=*/false);
  if (st != MM_OK) return st;
  size_t need = whole->ws_bytes;
  if (whole->kind == KK_Q4_WIDE || whole->kind == KK_Q4_MMA) {
    // every member takes the group's kernel (one INIT writes the wdata
    // layout of that kernel for all of them)
    for (int i = 0; i < count; ++i) {
      Plan pi;
      st = make_plan(MM_TYPE_Q4_0, M, Ns[i], K, whole->variant, &pi);
      if (st != MM_OK) return st;
      if (pi.ws_bytes > need) need = pi.ws_bytes;
    }
  }
  *ws = need;
  return MM_OK;
}

// Bytes of one of the layer's matrices (all experts), and of its scales.
size_t moe_matrix_bytes(const mm_moe_layer& l, int64_t rows, int64_t K) {
  return (size_t)l.E * (size_t)(l.type == MM_TYPE_Q4_0R ? repacked_bytes(rows, K)
                                                        : rows * row_bytes(l.type, K));
}
size_t moe_scale_bytes(const mm_moe_layer& l, int64_t rows, int64_t K) {
  if (l.type == MM_TYPE_MXFP4)
    return (size_t)l.E * (size_t)rows * 4 * (size_t)((K + kMx4Group - 1) / kMx4Group);
  if (l.type != MM_TYPE_F8) return 0;
  return (size_t)l.E * (size_t)((rows + kF8Block - 1) / kF8Block) *
         (size_t)((K + kF8Block - 1) / kF8Block) * 4;
}

}  // namespace

namespace {

// The layer, with its own router (ids and weights are outputs, may be NULL) or,
// `routed`, for a choice that is given (ids and weights are inputs).
int moe(const mm_moe_layer* layer, const float* x, float* dst, int32_t* ids, float* weights,
        bool routed, int64_t T, void* ws, size_t ws_bytes, void* stream) {
  if (!layer) return MM_ERR_NULL;
  const mm_moe_layer& l = *layer;
  MoePlan p;
  int st = make_moe_plan(l.type, T, l.D, l.F, l.E, l.top_k, &p, routed);
  if (st != MM_OK) return st;
  if (T == 0) return MM_OK;
  const bool scaled = l.type == MM_TYPE_F8 || l.type == MM_TYPE_MXFP4;
  if (!x || !dst || !l.gate || !l.up || !l.down) return MM_ERR_NULL;
  if (routed ? !ids || !weights : !l.router) return MM_ERR_NULL;
  if (scaled && (!l.gate_scale || !l.up_scale || !l.down_scale)) return MM_ERR_NULL;
  const void* const router = routed ? nullptr : l.router;
  const auto off = [](const void* v, uintptr_t a) { return (uintptr_t)v % a != 0; };
  if (off(x, 16) || off(router, 16) || off(l.gate, 16) || off(l.up, 16) || off(l.down, 16) ||
      off(dst, 4) || off(ids, 4) || off(weights, 4))
    return MM_ERR_ALIGN;
  if (scaled && (off(l.gate_scale, 4) || off(l.up_scale, 4) || off(l.down_scale, 4))) return MM_ERR_ALIGN;
  if (!ws || ws_bytes < p.ws_bytes) return MM_ERR_WORKSPACE;
  if (off(ws, 256)) return MM_ERR_ALIGN;
  const size_t xb = (size_t)(T * l.D) * 4, kb = (size_t)(T * l.top_k) * 4;
  const struct { const void* p; size_t n; } in[10] = {
      {x, xb}, {router, (size_t)(l.E * l.D) * 4},
      {l.gate, moe_matrix_bytes(l, l.F, l.D)}, {l.up, moe_matrix_bytes(l, l.F, l.D)},
      {l.down, moe_matrix_bytes(l, l.D, l.F)},
      {scaled ? l.gate_scale : nullptr, moe_scale_bytes(l, l.F, l.D)},
      {scaled ? l.up_scale : nullptr, moe_scale_bytes(l, l.F, l.D)},
      {scaled ? l.down_scale : nullptr, moe_scale_bytes(l, l.D, l.F)},
      {routed ? ids : nullptr, kb}, {routed ? weights : nullptr, kb}};
  const struct { const void* p; size_t n; } out[4] = {
      {dst, xb}, {ws, p.ws_bytes}, {routed ? nullptr : ids, kb}, {routed ? nullptr : weights, kb}};
  for (int i = 0; i < 4; ++i) {
    for (const auto& v : in)
      if (ranges_overlap(out[i].p, out[i].n, v.p, v.n)) return MM_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MM_ERR_ALIAS;
  }
  st = check_device();
  if (st != MM_OK) return st;
  uint8_t* const b = (uint8_t*)ws;
  MoeArgs a;
  a.x = x;
  a.router = l.router;
  a.gate = (const uint8_t*)l.gate; a.up = (const uint8_t*)l.up; a.down = (const uint8_t*)l.down;
  a.gate_scale = l.gate_scale; a.up_scale = l.up_scale; a.down_scale = l.down_scale;
  a.dst = dst;
  a.logits = (double*)(b + p.off_logits);
  a.ids = ids && !routed ? ids : (int*)(b + p.off_ids);
  a.weights = weights && !routed ? weights : (float*)(b + p.off_weights);
  a.given_ids = routed ? ids : nullptr;
  a.given_weights = routed ? weights : nullptr;
  a.xp = b + p.off_xp; a.xs = (float*)(b + p.off_xs);
  a.hp = b + p.off_hp; a.hs = (float*)(b + p.off_hs);
  a.T = (int)T; a.D = (int)l.D; a.F = (int)l.F; a.E = (int)l.E;
  a.top_k = l.top_k; a.norm = l.norm != 0;
  a.fold = p.fold;
  a.up_groups = p.up_groups;
  return hip_status(launch_moe(l.type, p, a, (float*)(b + p.off_part), (hipStream_t)stream));
}

}  // namespace

size_t mm_moe_workspace_size(const mm_moe_layer* layer, int64_t T) {
  MoePlan p;
  if (!layer || make_moe_plan(layer->type, T, layer->D, layer->F, layer->E, layer->top_k, &p) != MM_OK)
    return 0;
  return p.ws_bytes;
}

mm_status mm_moe_f32(const mm_moe_layer* layer, const float* x, float* dst, int32_t* ids,
                     float* weights, int64_t T, void* ws, size_t ws_bytes, void* stream) {
  return as_status(moe(layer, x, dst, ids, weights, false, T, ws, ws_bytes, stream));
}

size_t mm_moe_routed_workspace_size(const mm_moe_layer* layer, int64_t T) {
  MoePlan p;
  if (!layer || make_moe_plan(layer->type, T, layer->D, layer->F, layer->E, layer->top_k, &p, true) != MM_OK)
    return 0;
  return p.ws_bytes;
}

mm_status mm_moe_routed_f32(const mm_moe_layer* layer, const float* x, const int32_t* ids,
                            const float* weights, float* dst, int64_t T, void* ws, size_t ws_bytes,
                            void* stream) {
  return as_status(moe(layer, x, dst, const_cast<int32_t*>(ids), const_cast<float*>(weights), true, T,
                       ws, ws_bytes, stream));
}

mm_status mm_route_f32(const mm_router* router, const float* logits, int32_t* ids, float* weights,
                       int64_t T, void* stream) {
  if (!router) return MM_ERR_NULL;
  const mm_router& r = *router;
  if ((r.score != MM_SCORE_SOFTMAX && r.score != MM_SCORE_SIGMOID) || r.group_top < 1 || r.group_top > 2)
    return MM_ERR_ARG;
  if (T < 0 || T > kRouteMaxTokens || r.E < 1 || r.E > kRouteMaxExperts || r.top_k < 1 ||
      r.top_k > kRouteMaxTopK || r.top_k > r.E || r.groups < 1 || r.groups > 64 || r.E % r.groups ||
      r.group_k < 1 || r.group_k > r.groups)
    return MM_ERR_SHAPE;
  if (T == 0) return MM_OK;
  if (!logits || !ids || !weights) return MM_ERR_NULL;
  const auto off = [](const void* v) { return (uintptr_t)v % 4 != 0; };
  if (off(logits) || off(r.bias) || off(ids) || off(weights)) return MM_ERR_ALIGN;
  const size_t lb = (size_t)T * (size_t)r.E * 4, kb = (size_t)T * (size_t)r.top_k * 4;
  if (ranges_overlap(ids, kb, logits, lb) || ranges_overlap(weights, kb, logits, lb) ||
      ranges_overlap(ids, kb, r.bias, (size_t)r.E * 4) || ranges_overlap(weights, kb, r.bias, (size_t)r.E * 4) ||
      ranges_overlap(ids, kb, weights, kb))
    return MM_ERR_ALIAS;
  const int st = check_device();
  if (st != MM_OK) return as_status(st);
  RouteArgs a;
  a.logits = logits; a.bias = r.bias; a.ids = ids; a.weights = weights;
  a.T = T; a.E = (int)r.E; a.top_k = r.top_k;
  // every group taken: no groups
  a.groups = r.group_k < r.groups ? r.groups : 1;
  a.group_k = r.group_k; a.group_top = r.group_top;
  a.lanes_per_group = 1;
  while (2 * a.lanes_per_group * a.groups <= 64) a.lanes_per_group *= 2;
  a.softmax = r.score == MM_SCORE_SOFTMAX; a.norm = r.norm != 0; a.scale = r.scale;
  return as_status(hip_status(launch_route(a, (hipStream_t)stream)));
}

mm_status mm_rms_norm_f32(const float* x, const float* residual, const float* weight, float eps,
                          float* sum, int out_type, void* y, void* scales, int64_t T, int64_t D,
                          void* stream) {
  if (out_type != MM_TYPE_F32 && out_type != MM_TYPE_F8 && out_type != MM_TYPE_MXFP4) return MM_ERR_ARG;
  if (!(eps >= 0.0f)) return MM_ERR_ARG;
  const bool scaled = out_type != MM_TYPE_F32;
  if (T < 0 || D < 0 || D > kNormMaxDim || (scaled && D % kQK)) return MM_ERR_SHAPE;
  if (T == 0 || D == 0) return MM_OK;
  int waves, rows;
  norm_shape(T, D, &waves, &rows);
  if (T > kF8MaxK * 256 || (T + rows - 1) / rows * (64 * waves * rows) > 0xffffffffll) return MM_ERR_SHAPE;
  if (!x || !y || (scaled && !scales)) return MM_ERR_NULL;
  const auto off = [](const void* v, uintptr_t a) { return (uintptr_t)v % a != 0; };
  if (off(x, 4) || off(residual, 4) || off(weight, 4) || off(sum, 4) || off(y, scaled ? 16 : 4) ||
      (scaled && off(scales, 4)))
    return MM_ERR_ALIGN;
  const size_t n = (size_t)T * (size_t)D, xb = n * 4, wb = (size_t)D * 4;
  const size_t yb = out_type == MM_TYPE_F32 ? xb : out_type == MM_TYPE_F8 ? n : n / 2;
  const size_t sb = scaled ? (size_t)T * (size_t)((D + 127) / 128) * 4 : 0;
  // the sum may take the place of x or of the residual, nothing else may overlap
  if ((sum != x && ranges_overlap(sum, xb, x, xb)) || (sum != residual && ranges_overlap(sum, xb, residual, xb)) ||
      ranges_overlap(sum, xb, weight, wb) || ranges_overlap(sum, xb, y, yb) || ranges_overlap(sum, xb, scales, sb))
    return MM_ERR_ALIAS;
  const struct { const void* p; size_t n; } in[3] = {{x, xb}, {residual, xb}, {weight, wb}};
  for (const auto& v : in)
    if (ranges_overlap(y, yb, v.p, v.n) || ranges_overlap(scales, sb, v.p, v.n)) return MM_ERR_ALIAS;
  if (ranges_overlap(y, yb, scales, sb)) return MM_ERR_ALIAS;
  const int st = check_device();
  if (st != MM_OK) return as_status(st);
  NormArgs a;
  a.x = x; a.residual = residual; a.weight = weight; a.sum = sum; a.y = y; a.scales = scales;
  a.T = T; a.D = (int)D; a.eps = eps;
  return as_status(hip_status(launch_rms_norm(out_type, a, (hipStream_t)stream)));
}

size_t mm_mul_mat_q4_0_group_workspace_size(int count, const int64_t* Ns, int64_t M, int64_t K) {
  Plan p;
  int64_t tot;
  size_t ws = 0;
  if (group_plan(count, Ns, M, K, &p, &tot, &ws) != MM_OK) return 0;
  return ws;
}

mm_status mm_mul_mat_q4_0_f32_group(int count, const void* const* src0s, float* const* dsts,
                                    const int64_t* Ns, const float* src1, int64_t M, int64_t K,
                                    void* ws, size_t ws_bytes, void* stream) {
  Plan whole;
  int64_t ntot = 0;
  size_t need = 0;
  int st = group_plan(count, Ns, M, K, &whole, &ntot, &need);
  if (st != MM_OK) return as_status(st);
  if (!src0s || !dsts) return MM_ERR_NULL;
  if (M == 0 || ntot == 0) return MM_OK;
  // each product on its own, then the group as a whole
  const int64_t rbytes = row_bytes(MM_TYPE_Q4_0, K);
  for (int i = 0; i < count; ++i) {
    if (Ns[i] == 0) continue;
    Plan pi = whole;
    pi.ws_bytes = need;
    st = validate_mul_mat(MM_TYPE_Q4_0, src0s[i], src1, dsts[i], M, Ns[i], K, ws, ws_bytes, pi);
    if (st != MM_OK) return as_status(st);
    for (int j = 0; j < count; ++j) {
      if (j == i || Ns[j] == 0) continue;
      if (ranges_overlap(dsts[i], (size_t)M * Ns[i] * 4, dsts[j], (size_t)M * Ns[j] * 4) ||
          (K > 0 && ranges_overlap(dsts[i], (size_t)M * Ns[i] * 4, src0s[j], (size_t)Ns[j] * rbytes)))
        return MM_ERR_ALIAS;
    }
  }
  st = check_device();
  if (st != MM_OK) return as_status(st);
  hipStream_t s = (hipStream_t)stream;
  if (K == 0) {
    for (int i = 0; i < count; ++i) {
      if (Ns[i] == 0) continue;
      st = hip_status(launch_zero(dsts[i], M * Ns[i], s));
      if (st != MM_OK) return as_status(st);
    }
    return MM_OK;
  }
  if (whole.kind == KK_Q4_NARROW) {
    Q4Mats mats;
    int row = 0, c = 0;
    for (int i = 0; i < kMaxGroup; ++i) { mats.w[i] = nullptr; mats.dst[i] = nullptr; }
    for (int i = 0; i < count; ++i) {
      if (Ns[i] == 0) continue;
      mats.w[c] = (const uint8_t*)src0s[i];
      mats.dst[c] = dsts[i];
      mats.row0[c] = row;
      row += (int)Ns[i];
      ++c;
    }
    for (int i = c; i <= kMaxGroup; ++i) mats.row0[i] = row;
    mats.count = c;
    const Q4Args a = q4_args(whole, mats.w[0], mats.dst[0], nullptr, M, ntot, K, 0, 0, ws);
    if (!whole.fuse) {
      st = q4_init(whole, src1, M, K, ws, s);
      if (st != MM_OK) return as_status(st);
    }
    return as_status(hip_status(launch_q4_narrow(whole, a, mats, whole.fuse ? src1 : nullptr, s)));
  }
  // wide and skinny MFMA: one INIT, then one product per matrix (same wdata
  // layout at the front of every per-matrix plan)
  st = q4_init(whole, src1, M, K, ws, s);
  if (st != MM_OK) return as_status(st);
  for (int i = 0; i < count; ++i) {
    if (Ns[i] == 0) continue;
    Plan pi;
    make_plan(MM_TYPE_Q4_0, M, Ns[i], K, whole.variant, &pi);
    st = q4_product(pi, q4_args(pi, src0s[i], dsts[i], nullptr, M, Ns[i], K, 0, 0, ws), nullptr, s);
    if (st != MM_OK) return as_status(st);
  }
  return MM_OK;
}

size_t mm_mul_mat_workspace_size(int type, int64_t M, int64_t N, int64_t K) {
  if (type == MM_TYPE_F8) return mm_mul_mat_f8_workspace_size(M, N, K, 0);
  if (type == MM_TYPE_MXFP4) return mm_mul_mat_mxfp4_workspace_size(M, N, K, 0);
  Plan p;
  if (make_plan(type, M, N, K, 0, &p) != MM_OK) return 0;
  return p.ws_bytes;
}

size_t mm_debug_workspace_size(int type, int64_t M, int64_t N, int64_t K, int variant) {
  Plan p;
  if (make_plan(type, M, N, K, variant, &p) != MM_OK) return 0;
  return p.ws_bytes;
}

int64_t mm_row_bytes(int type, int64_t K) { return row_bytes(type, K); }

mm_status mm_dispatch(int type, int64_t M, int64_t N, int64_t K, int* out) {
  Plan p;
  const int st = make_plan(type, M, N, K, 0, &p);
  if (st != MM_OK) return as_status(st);
  if (out) {
    out[0] = p.variant;
    out[1] = p.split;
    const bool tiled = p.variant == 2;
    out[2] = tiled ? p.bm : p.mt;
    out[3] = tiled ? p.bn : p.variant == 3 ? p.waves : p.kind == KK_Q4_NARROW && p.fuse ? p.fuse_rpw : p.rpw;
    const bool q4 = p.type == MM_TYPE_Q4_0 || p.type == MM_TYPE_Q4_0R || p.type == MM_TYPE_Q8_0;
    // INIT (quantized kinds, unless fused), the src1 pre-pass of the wide
    // F16 kernel, the product, the split-K reduce
    const int init = (q4 && !(p.kind == KK_Q4_NARROW && p.fuse)) ? 1 : 0;
    const int pre = p.kind == KK_F16_WIDE ? 1 : 0;
    out[4] = init + pre + 1 + (p.split > 1 ? 1 : 0);
  }
  return MM_OK;
}

mm_status mm_debug_mul_mat(int type, const void* src0, const float* src1, float* dst, int32_t* dots,
                           int64_t M, int64_t N, int64_t K, int64_t n0, int64_t n1, int variant,
                           void* ws, size_t ws_bytes, void* stream) {
  if (variant < 0 || variant > 3) return MM_ERR_ARG;
  if (n0 < 0 || n1 < n0 || n1 > N) return MM_ERR_SHAPE;
  if ((type != MM_TYPE_Q4_0 && type != MM_TYPE_Q4_0R && type != MM_TYPE_Q8_0) || n1 == n0)
    dots = nullptr;
  else if (!dots) return MM_ERR_NULL;
  if (type == MM_TYPE_Q8_0 && dots) {
    // Q8_0 weights: only the wide kernel writes block dots
    Plan p;
    const int st = make_plan(type, M, N, K, variant, &p);
    if (st != MM_OK) return as_status(st);
    if (p.kind == KK_Q4_NARROW) return MM_ERR_ARG;
  }
  return as_status(
      mul_mat(type, src0, src1, dst, dots, M, N, K, n0, n1, variant, ws, ws_bytes, stream));
}

const char* mm_status_string(int status) {
  switch (status) {
    case MM_OK: return "ok";
    case MM_ERR_NULL: return "a required pointer is NULL";
    case MM_ERR_SHAPE: return "invalid shape (negative size, K not a multiple of 32 for a block type, or too large)";
    case MM_ERR_ALIGN: return "pointer not aligned as required";
    case MM_ERR_WORKSPACE:
      return "workspace missing or smaller than mm_mul_mat_workspace_size() (for "
             "mm_mul_mat_q4_0_f32_noalloc: the shape needs more than its fixed 64 MiB array)";
    case MM_ERR_ALIAS: return "output or workspace overlaps another operand";
    case MM_ERR_DEVICE: return "current device is not gfx950 (MI355X)";
    case MM_ERR_HIP: return "HIP runtime error";
    case MM_ERR_ARG: return "unknown type or variant";
    default: return "unknown status";
  }
}

}  // extern "C"
