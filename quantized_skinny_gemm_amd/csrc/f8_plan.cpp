// Host-only plan, workspace layout and argument checks of the e4m3 (F8)
// quantizer and product.
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

}  // namespace

int make_f8_plan(int64_t M, int64_t N, int64_t K, bool given, F8Plan* p) {
  *p = F8Plan();
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kF8MaxK || K % kQK)
    return MM_ERR_SHAPE;
  if (M == 0 || N == 0) return MM_OK;
  if (K == 0) { p->kind = F8_ZERO; return MM_OK; }
  const int64_t nkb = ceil_div(K, kF8Block);

  // Up to 8 rounds of 32 blocks of 128: every workgroup quantizes src1 itself
  // (at M = 8 and K = 4096 in about the time of an INIT launch).  Below 32 blocks
  // of K its waves idle in part, and the join of every 16 rows shows: a workgroup
  // takes about 7 us per group at any K, the tiled kernel the time of the bytes.
  // So K bounds the rows (us per call, fused / tiled, M = 1: 12500 x 1024 10.8 / 10.7,
  // 18944 x 1024 13.3 / 11.1, 65536 x 1024 36 / 20; 12500 x 2048 11.4 / 12.9, 24000 x
  // 2048 16.4 / 16.6, 30000 x 2048 22.3 / 17.8; 18944 x 2560 14.1 / 18.7, 65536 x 2560
  // 43.1 / 42.3, 152064 x 2560 96.0 / 94.6; 18944 x 3584 15.1 / 23.8, 65536 x 3584 47.7 /
  // 55.1, 65536 x 4096 52.1 / 69.1).
  const int64_t blocks = M * nkb, groups = ceil_div(N, 16);
  if (!given && M <= 16 && blocks <= 256 && (nkb >= 20 || groups <= (nkb >= 16 ? 6 : 3) * kCUs)) {
    p->kind = F8_FUSED;
    p->nt = blocks <= 32 ? 1 : blocks <= 64 ? 2 : blocks <= 128 ? 4 : 8;
    // workgroups along N, each walking groups of 16 rows (us per call, 14336 x
    // 4096, 512 / 768 workgroups: M = 1 15.1 / 14.3, M = 8 18.5 / 20.1)
    const int64_t most = M <= 2 ? 3 * kCUs : 2 * kCUs;
    p->grid_n = groups < most ? groups : most;
    p->lds = (size_t)(M * (nkb * kF8Block + 16)) + align_up((size_t)blocks * 4, 16) + (size_t)M * 512;
    return MM_OK;
  }
  // Few src1 rows: the skinny kernel, which has 16 weight rows per workgroup and
  // no split of K across them; else the tiled one.  The most rows for it (us per
  // call without INIT, skinny / tiled):
  // - Over 8192 weight rows a third workgroup of it shares a CU and its time steps
  //   up; the shorter K is, the sooner the tiled kernel is ahead (M = 1, 4, 8: 8200 x
  //   1024 8.7 / 8.0, 9.8 / 8.1, 11.3 / 8.0; 12500 x 2560 12.7 / 12.6, 14.4 / 12.5, 15.7 /
  //   12.6; 18944 x 2816 15.9 / 17.6, 17.4 / 17.8, 18.9 / 17.7; 18944 x 3584 16.6 / 21.2,
  //   17.7 / 21.4, 19.2 / 21.4; 65536 x 3584, M = 1, 8 53.4 / 53.8, 61.2 / 53.9; 65536 x
  //   4096 58.2 / 67.0, 66.0 / 68.0; of 8192 rows M = 1 at K = 1024 / 3968 8.0 / 11.7,
  //   8.3 / 13.4).
  // - Up to 2048 weight rows most CUs have none, and the longer K is, the more the
  //   tiled kernel's K split gains (M = 1, 8, 16, 24: 1024 x 4096 7 / 10, 7 / 10, 7 / 10,
  //   9 / 10; 1024 x 8192 7 / 10, 9 / 10, 11 / 10, 15 / 10; 1024 x 14336 12 / 10, 16 / 10,
  //   20 / 10, 26 / 10; 1024 x 28672 20 / 13, 26 / 14, 33 / 14, 44 / 14; 2048 x 14336 12 / 12,
  //   16 / 13, 20 / 13, 26 / 13).
  // - Between: 8 on matrices of 32 MiB or more (4096 x 14336, M = 4, 8, 16 14 / 16, 16 /
  //   17, 20 / 17; 14336 x 4096, M = 16 with INIT 24.7 / 19.8), else 24, where the two
  //   tiles of 16 src1 rows past 16 are worth it (M = 16, 24: 4096 x 4096 8 / 12, 10 / 12;
  //   3200 x 8192 12 / 12, 15 / 13; 7000 x 3200 10.8 / 12.2, 15.2 / 12.2; 8192 x 1024 11.3 /
  //   11.7, 15.6 / 11.8).
  const bool large = N * K >= ((int64_t)1 << 25);
  const int64_t skinny_rows = groups > 2 * kCUs    ? (nkb < 22 ? 0 : nkb < 32 ? 4 : 8)
                              : groups <= kCUs / 2 ? (nkb >= 96 ? 0 : nkb >= 64 ? 8 : 24)
                              : large              ? 8
                                                   : (groups <= kCUs && nkb < 64 ? 24 : 16);
  const bool wide = M > skinny_rows;
  // Output tile by M (us per call with INIT, 64 x 128, 128 x 128 and 128 x 256 tiles:
  // 14336 x 4096, M = 128 29.0 / 32.9 / 37.1, M = 256 53.8 / 44.3 / 51.4, M = 512 102.5 /
  // 84.8 / 72.1; 4096 x 14336, M = 128 30.6 / 33.1 / 38.2, M = 256 52.1 / 49.0 / 51.5,
  // M = 600 157.3 / 120.7 / 94.5).  Below 32 MiB a small tile also where that gives
  // each CU at most one (4096 x 4096, M = 256 23.0 / 27.8 / 31.5, M = 512 31.4 / 35.3 /
  // 39.7, M = 1024 57.6 / 49.8 / 56.0, M = 2048 113.2 / 97.9 / 81.7), and 64 x 64 up to
  // M = 128 (M = 64 / 128 14.9 / 17.4 against 17.1 / 18.9).
  const auto fits = [&](int bm, int bn) { return ceil_div(M, bm) * ceil_div(N, bn) <= kCUs; };
  const bool low = M <= 128 || (!large && fits(64, 128));
  const bool mid = M <= 256 || (!large && fits(128, 128));
  p->bm = low ? 64 : 128;
  p->bn = !low && !mid ? 256 : !large && M <= 128 ? 64 : 128;
  // src1 codes where INIT makes them, or where K ends inside a block and the
  // tiled kernel needs rows of whole blocks
  size_t off = 0;
  if (!given || (wide && K % kF8Block)) {
    p->off_a = off;
    off = align_up(off + (size_t)M * (wide ? (size_t)nkb * kF8Block : (size_t)K), 256);
  }
  if (!given) {
    p->off_as = off; off = align_up(off + (size_t)M * (size_t)nkb * 4, 256);
  }
  if (!wide) {
    p->kind = F8_SKINNY;
    p->nt = M <= 16 ? 1 : 2;
    p->waves = 8;
    while (p->waves > 1 && p->waves > nkb) p->waves /= 2;
    p->grid_n = ceil_div(N, 16);
    if (p->grid_n * p->waves > kMaxTiles * 8) return MM_ERR_SHAPE;
    p->lds = (size_t)p->waves * 1024 * p->nt;
  } else {
    p->kind = F8_WIDE;
    p->tiles_m = ceil_div(M, p->bm);
    p->tiles_n = ceil_div(N, p->bn);
    const int64_t tiles = p->tiles_m * p->tiles_n;
    if (tiles > kMaxTiles) return MM_ERR_SHAPE;
    int64_t split = 1;
    if (tiles < kCUs) {
      split = kCUs / tiles;
      if (split > nkb / 4) split = nkb / 4;
      if (split > 16) split = 16;
      if (split < 1) split = 1;
    }
    p->kchunk = ceil_div(nkb, split);
    p->split = (int)ceil_div(nkb, p->kchunk);
    if (p->split > 1) {
      p->off_part = off;
      off = align_up(off + (size_t)p->split * (size_t)M * (size_t)N * 4, 256);
    }
  }
  p->ws_bytes = off;
  return MM_OK;
}

int validate_f8(const void* src0, const void* scale0, const void* src1, const void* scale1,
                const void* dst, int64_t M, int64_t N, int64_t K, bool given, const void* ws,
                size_t ws_bytes, const F8Plan& p) {
  if (p.kind == F8_NONE) return MM_OK;
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
  const size_t nkb = (size_t)ceil_div(K, kF8Block);
  const struct { const void* p; size_t n; } in[4] = {
      {src0, (size_t)N * (size_t)K},
      {scale0, (size_t)ceil_div(N, kF8Block) * nkb * 4},
      {src1, (size_t)M * (size_t)K * (given ? 1 : 4)},
      {given ? scale1 : nullptr, (size_t)M * nkb * 4}};
  const size_t db = (size_t)M * (size_t)N * 4;
  for (const auto& i : in)
    if (overlaps(dst, db, i.p, i.n) || (p.ws_bytes > 0 && overlaps(ws, p.ws_bytes, i.p, i.n)))
      return MM_ERR_ALIAS;
  if (p.ws_bytes > 0 && overlaps(ws, p.ws_bytes, dst, db)) return MM_ERR_ALIAS;
  return MM_OK;
}

int validate_f8_quantize(const void* x, const void* codes, const void* scales, int64_t nrows,
                         int64_t k, int block_rows) {
  if (block_rows != 1 && block_rows != kF8Block) return MM_ERR_ARG;
  if (nrows < 0 || k < 0 || nrows > kMaxDim || k > kF8MaxK || k % kQK) return MM_ERR_SHAPE;
  if (nrows == 0 || k == 0) return MM_OK;
  const int64_t nkb = ceil_div(k, kF8Block), nrb = ceil_div(nrows, block_rows);
  if (block_rows != 1 && nrb * nkb > kMaxTiles) return MM_ERR_SHAPE;
  if (!x || !codes || !scales) return MM_ERR_NULL;
  if ((uintptr_t)x % 16 || (uintptr_t)codes % 16 || (uintptr_t)scales % 4) return MM_ERR_ALIGN;
  const size_t xb = (size_t)nrows * (size_t)k * 4, cb = (size_t)nrows * (size_t)k;
  const size_t sb = (size_t)nrb * (size_t)nkb * 4;
  if (overlaps(x, xb, codes, cb) || overlaps(x, xb, scales, sb) || overlaps(codes, cb, scales, sb))
    return MM_ERR_ALIAS;
  return MM_OK;
}

}  // namespace qsg
