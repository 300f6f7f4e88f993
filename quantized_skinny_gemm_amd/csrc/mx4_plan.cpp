// Host-only plan, workspace layout and argument checks of the MXFP4 quantizer
// and product, and the norm's launch shape.
#include <stdint.h>

#include "../../include/mm.h"
#include "plan.h"

namespace qsg {

namespace {

constexpr int64_t kMaxDim = 0x7fffff00;      // the ends of tiles stay below 2^31
constexpr int64_t kMaxTiles = (1 << 23) - 1; // workgroups x 512 threads stay below 2^32

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

size_t scale_bytes(int64_t rows, int64_t K) { return (size_t)rows * 4 * (size_t)ceil_div(K, kMx4Group); }

}  // namespace

int make_mx4_plan(int64_t M, int64_t N, int64_t K, bool given, Mx4Plan* p) {
  *p = Mx4Plan();
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kF8MaxK || K % kQK)
    return MM_ERR_SHAPE;
  if (M == 0 || N == 0) return MM_OK;
  if (K == 0) { p->kind = MX4_ZERO; return MM_OK; }
  const int64_t ng = ceil_div(K, kMx4Group), tiles16 = ceil_div(N, 16);
  if (!given && M <= 16 && M * ng <= 256) {
    p->kind = MX4_FUSED;
    const int64_t groups = M * ng;
    p->nt = groups <= 32 ? 1 : groups <= 64 ? 2 : groups <= 128 ? 4 : 8;
    const int64_t most = 3 * kCUs;
    p->grid_n = tiles16 < most ? tiles16 : most;
    p->lds = (size_t)(M * (ng * kMx4Group / 2 + 16)) + align_up((size_t)groups * 4, 16) + (size_t)M * 512;
    return MM_OK;
  }
  size_t off = 0;
  if (!given) {
    p->off_a = off; off = align_up(off + (size_t)M * (size_t)(K / 2), 256);
    p->off_as = off; off = align_up(off + scale_bytes(M, K), 256);
  }
  if (M <= 32) {
    p->kind = MX4_SKINNY;
    p->nt = M <= 16 ? 1 : 2;
    p->waves = 8;
    while (p->waves > 1 && (p->waves - 1) * 4 >= ng) p->waves /= 2;
    p->grid_n = tiles16;
    if (p->grid_n * p->waves > kMaxTiles * 8) return MM_ERR_SHAPE;
    p->lds = (size_t)p->waves * 1024 * p->nt;
  } else {
    p->kind = MX4_WIDE;
    const bool low = M <= 64;
    p->bm = low ? 64 : M <= 128 ? 128 : 128;
    p->bn = low ? 128 : M <= 256 ? 128 : 256;
    if (M > 256 && N > 16384) p->bm = 256;
    p->tiles_m = ceil_div(M, p->bm);
    p->tiles_n = ceil_div(N, p->bn);
    const int64_t tiles = p->tiles_m * p->tiles_n, nst = ceil_div(K, 256);
    if (tiles > kMaxTiles) return MM_ERR_SHAPE;
    int64_t split = 1;
    if (tiles < kCUs) {
      split = kCUs / tiles;
      if (split > nst / 4) split = nst / 4;
      if (split > 16) split = 16;
      if (split < 1) split = 1;
    }
    p->kchunk = ceil_div(nst, split);
    p->split = (int)ceil_div(nst, p->kchunk);
    if (p->split > 1) {
      p->off_part = off;
      off = align_up(off + (size_t)p->split * (size_t)M * (size_t)N * 4, 256);
    }
  }
  p->ws_bytes = off;
  return MM_OK;
}

int validate_mx4(const void* src0, const void* scale0, const void* src1, const void* scale1,
                 const void* dst, int64_t M, int64_t N, int64_t K, bool given, const void* ws,
                 size_t ws_bytes, const Mx4Plan& p) {
  if (p.kind == MX4_NONE) return MM_OK;
  if (!dst) return MM_ERR_NULL;
  if ((uintptr_t)dst % 4) return MM_ERR_ALIGN;
  if (K == 0) return MM_OK;
  if (!src0 || !scale0 || !src1 || (given && !scale1)) return MM_ERR_NULL;
  if ((uintptr_t)src0 % 16 || (uintptr_t)scale0 % 4 || (uintptr_t)src1 % 16 ||
      (given && (uintptr_t)scale1 % 4))
    return MM_ERR_ALIGN;
  if (p.ws_bytes > 0) {
    if (!ws || ws_bytes < p.ws_bytes) return MM_ERR_WORKSPACE;
    if ((uintptr_t)ws % 256) return MM_ERR_ALIGN;
  }
  const struct { const void* p; size_t n; } in[4] = {
      {src0, (size_t)N * (size_t)(K / 2)},
      {scale0, scale_bytes(N, K)},
      {src1, given ? (size_t)M * (size_t)(K / 2) : (size_t)M * (size_t)K * 4},
      {given ? scale1 : nullptr, scale_bytes(M, K)}};
  const size_t db = (size_t)M * (size_t)N * 4;
  for (const auto& i : in)
    if (overlaps(dst, db, i.p, i.n) || (p.ws_bytes > 0 && overlaps(ws, p.ws_bytes, i.p, i.n)))
      return MM_ERR_ALIAS;
  if (p.ws_bytes > 0 && overlaps(ws, p.ws_bytes, dst, db)) return MM_ERR_ALIAS;
  return MM_OK;
}

int validate_mx4_quantize(const void* x, const void* codes, const void* scales, int64_t nrows,
                          int64_t k) {
  if (nrows < 0 || k < 0 || nrows > kMaxDim || k > kF8MaxK || k % kQK) return MM_ERR_SHAPE;
  if (nrows == 0 || k == 0) return MM_OK;
  if (!x || !codes || !scales) return MM_ERR_NULL;
  if ((uintptr_t)x % 16 || (uintptr_t)codes % 16 || (uintptr_t)scales % 4) return MM_ERR_ALIGN;
  const size_t xb = (size_t)nrows * (size_t)k * 4, cb = (size_t)nrows * (size_t)(k / 2);
  const size_t sb = scale_bytes(nrows, k);
  if (overlaps(x, xb, codes, cb) || overlaps(x, xb, scales, sb) || overlaps(codes, cb, scales, sb))
    return MM_ERR_ALIAS;
  return MM_OK;
}

void norm_shape(int64_t T, int64_t D, int* waves, int* rows) {
  // As many waves as have a piece of 8 values for each lane while rows are few
  // (one row's latency is what counts), else so few that a lane holds four.
  const int64_t pieces = ceil_div(D, 8), each = T < 2 * kCUs ? 1 : 4;
  *waves = 1;
  while (*waves < 16 && (int64_t)*waves * 64 * each < pieces) *waves *= 2;
  *rows = *waves < 4 ? 4 / *waves : 1;
}

}  // namespace qsg
