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

  // Up to 8 rounds of 32 groups of 128: every workgroup quantizes src1 itself, in
  // less time than an INIT launch takes (us per call, fused / INIT and product: 4096 x
  // 4096, M = 1, 4, 8 4.3 / 6.8, 5.1 / 7.0, 6.3 / 7.2; 14336 x 4096, M = 8 11.7 / 11.3).
  const int64_t groups = M * ng;
  if (!given && M <= 16 && groups <= 256) {
    p->kind = MX4_FUSED;
    p->nt = groups <= 32 ? 1 : groups <= 64 ? 2 : groups <= 128 ? 4 : 8;
    // workgroups, each walking tiles of 16 weight rows (14336 x 4096, 256 / 512 / 768
    // workgroups: M = 1 9.1 / 7.9 / 8.6 us, M = 4 10.1 / 10.9 / 11.0, M = 8 11.7 / 12.8 / 14.9)
    const int64_t most = M <= 2 ? 2 * kCUs : kCUs;
    p->grid_n = tiles16 < most ? tiles16 : most;
    p->lds = (size_t)(M * (ng * kMx4Group / 2 + 16)) + align_up((size_t)groups * 4, 16) + (size_t)M * 512;
    return MM_OK;
  }
  size_t off = 0;
  if (!given) {
    p->off_a = off; off = align_up(off + (size_t)M * (size_t)(K / 2), 256);
    p->off_as = off; off = align_up(off + scale_bytes(M, K), 256);
  }
  // Few src1 rows on few weight rows: 16 weight rows per workgroup fill the device
  // sooner than the tiled kernel's 32 or 64 (us, skinny / tiled: 4096 x 4096, M = 16
  // 4.9 / 5.1, M = 32 6.2 / 5.0; 1000 x 4128, M = 32 4.4 / 5.4; 14336 x 4096, M = 4, 16
  // 9.3 / 8.0, 11.8 / 8.0; 4096 x 14336, M = 16, 32 10.2 / 13.1, 14.9 / 13.1).
  if ((M <= 16 && tiles16 <= 2 * kCUs) || (M <= 32 && tiles16 <= kCUs / 2)) {
    p->kind = MX4_SKINNY;
    p->nt = M <= 16 ? 1 : 2;
    p->waves = 8;
    while (p->waves > 1 && (p->waves / 2) * 4 >= ng) p->waves /= 2;
    p->grid_n = tiles16;
    p->lds = (size_t)p->waves * 1024 * p->nt;
    p->ws_bytes = off;
    return MM_OK;
  }
  // Tiled: the tile, and the split of K over workgroups (with a second launch to join
  // it), of the least time by what a workgroup of each takes per stage of 256 k where
  // it has a CU to itself (hundredths of a us; fitted to calls of at most 256 workgroups
  // at K = 4096, which take 5, 6 to 8, 7 to 10, 9.6 to 14, 12 to 17, 18 to 25 and 27
  // to 34 us from few workgroups to 256).  256 workgroups run at a time; those that share
  // a CU take as long as one after the other.  The tile chosen and the best of all, in us:
  // 64 x 14336 x 4096 8.3 (64 x 64, the best), 128 x 14336 x 4096 11.3 (64 x 128, the best),
  // 256 x 14336 x 4096 16.5 (128 x 128, the best; 64 x 64 25.3, 256 x 128 24.2), 512 x
  // 14336 x 4096 25.5 (256 x 128, the best; 256 x 256 34.1, 128 x 128 34.2), 1024 x 14336 x
  // 4096 39 (256 x 256, the best; 256 x 128 53), 2048 x 4096 x 14336 80 (256 x 128, the best;
  // 256 x 256 94), 512 x 128256 x 4096 182 (256 x 256, the best; 256 x 128 222), 256 x
  // 4096 x 4096 7.9 (64 x 64, the best), 512 x 4096 x 4096 10.8 (64 x 128, the best).
  // The 32 x 64 tile (two sets of waves, each with half of K) has half a us to join its
  // sums: 32 x 14336 x 4096 8.3 (64 x 64 9.4, 32 x 32 8.9), 64 x 8192 x 4096 6.6 (7.6, 7.3),
  // 128 x 4096 x 4096 6.3 (7.6, 7.1), but 20 x 16000 x 1056 5.3 (4.9, 5.3).
  static const struct { int bm, bn, cost, fixed; } kTiles[] = {
      {32, 32, 19}, {32, 64, 24, 50}, {64, 64, 31}, {64, 128, 44}, {128, 128, 63}, {256, 128, 90}, {256, 256, 155}};
  const int64_t nst = ceil_div(K, 256);
  int64_t best = -1;
  p->kind = MX4_WIDE;
  for (const auto& t : kTiles) {
    const int64_t tm = ceil_div(M, t.bm), tn = ceil_div(N, t.bn);
    if (tm > kMaxTiles || tm * tn > kMaxTiles) continue;
    for (int64_t split = 1; split <= 16; split *= 2) {
      // a split: at least 4 stages each, no second round; the join takes about 7 us and
      // what writing and reading the partial sums does (us, split / not: 64 x 4096 x 28672
      // 15.7 / 20.6, 300 x 300 x 65536 15 / 40, 128 x 4096 x 14336 14.2 / 18.8, 33 x 512 x
      // 14336 12.5 / 11.0; of the largest tile that fills the device 8 times, which a cost
      // without the bytes takes: 1024 x 1024 x 8192 24 / 12, 384 x 4096 x 14336 34 / 26)
      if (split > 1 && (nst < 4 * split || tm * tn * split > kCUs)) break;
      const int64_t time = ceil_div(tm * tn * split, kCUs) * ceil_div(nst, split) * t.cost + t.fixed + (split > 1 ? 700 + split * M * N / 6000 : 0);
      if (best >= 0 && time >= best) continue;
      best = time;
      p->bm = t.bm; p->bn = t.bn;
      p->tiles_m = tm; p->tiles_n = tn;
      p->kchunk = ceil_div(nst, split);
      p->split = (int)ceil_div(nst, p->kchunk);
    }
  }
  if (best < 0) return MM_ERR_SHAPE;
  if (p->split > 1) {
    p->off_part = off;
    off = align_up(off + (size_t)p->split * (size_t)M * (size_t)N * 4, 256);
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
