// 8-bit floating point (OCP e4m3) with one fp32 scale per block of 128: the
// quantizer and the product, for gfx950.
//
// Codec: per block (1 x 128 for activations, 128 x 128 for weights)
//   d = max(fl32(amax / 448), 2^-126), id = fl32(1 / d),
//   code = e4m3(fl32(x * id)), round to nearest even; value = d * code.
// 448 is the largest e4m3 value and |x * id| <= 448 (1 + 2^-22), which still
// rounds to it, so no code saturates; the lower limit of d keeps id finite.
//
// Product: dst[m][n] = sum_b ds[m][b] * dw[n / 128][b] * S_b[m][n] with the
// block dot S_b = sum over the 128 k of block b of two e4m3 codes' products,
// on the binary16 matrix cores: an e4m3 code is exact in binary16 and the
// products of two are exact in fp32.  The matrix cores' own 8-bit
// instructions (16x16x128_f8f6f4, 16x16x32_fp8_fp8; the first at twice the
// rate) are not used: they drop the bits of a product that lie about 2^-17
// below the largest one of the sum (measured: 448 * 448 + 0.5 gives 200704,
// and normal codes give S_b with a relative error of 1.7e-5 in the mean, up to
// 4e-5), which is past the 1e-5 that the quantized products keep; binary16
// measures 3e-9.  S_b enters the fp32 sum with one fma by fl32(ds * dw).
// With the weights as operand A every output register of a lane belongs to
// one src1 row, so that scale is one value per lane and block.
//
// In every operand the 16-byte piece at k offset 16 g of a block's first
// half and the one at 64 + 16 g belong to lane group g (the tiled kernel has
// its own map below): the matrix core only needs both operands to agree on
// where a k lies, and this choice lets each load instruction cover whole
// 64-byte segments.
#include "f8.h"
#include "kernels.h"

namespace qsg {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBlk = kF8Block;          // 128

// Eight e4m3 codes as binary16 (exact; a NaN code becomes a NaN).
__device__ __forceinline__ v8h widen(uint32_t lo, uint32_t hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return (v8h){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// ---------------------------------------------------------------- quantizer

// 1 x 128 blocks: 16 lanes per block, one 32-byte load and one 8-byte store
// per lane; rows of codes `pitch` apart (K, or whole blocks).  Bound: HBM (5 bytes per value).
__global__ __launch_bounds__(256) void k_f8_quantize_rows(const float* __restrict__ x,
                                                          uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int K,
                                                          int pitch, int nkb, int64_t nblocks) {
  const int i = threadIdx.x & 15;
  for (int64_t blk = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); blk < nblocks;
       blk += (int64_t)gridDim.x * 16) {            // whole groups of 16 lanes
    const int64_t row = blk / nkb;
    const int k = (int)(blk - row * nkb) * kBlk + 8 * i;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (k < K) {                                    // K % 32 == 0: all 8 values or none
      const float4* p = reinterpret_cast<const float4*>(x + row * K + k);
      a = p[0]; b = p[1];
    }
    float d;
    const uint2 c = f8_row_block(a, b, d);
    if (k < pitch) *reinterpret_cast<uint2*>(codes + row * pitch + k) = c;   // past K: zeros
    if (i == 0) scales[blk] = d;
  }
}

// Codes given by the caller as rows of whole blocks, zeros past K, 16 bytes
// per thread (for the tiled product, where K ends inside a block).
__global__ __launch_bounds__(256) void k_f8_pad(const uint8_t* __restrict__ codes,
                                                uint8_t* __restrict__ rows, int K, int nkb,
                                                int64_t pieces) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += 256 * (int64_t)gridDim.x) {
    const int64_t row = i / (8 * nkb);
    const int k = (int)(i - row * 8 * nkb) * 16;
    *reinterpret_cast<uint4*>(rows + 16 * i) =
        k < K ? *reinterpret_cast<const uint4*>(codes + row * K + k) : make_uint4(0, 0, 0, 0);
  }
}

// 128 x 128 blocks: one workgroup per block, 64 values per thread held in
// registers between the maximum and the codes, so x is read once.
__global__ __launch_bounds__(256) void k_f8_quantize_tiles(const float* __restrict__ x,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales, int64_t N,
                                                           int K, int nkb) {
  __shared__ float part[4];
  const int64_t tn = blockIdx.x / nkb;
  const int kb = (int)(blockIdx.x - tn * nkb);
  const int tid = threadIdx.x;
  const int k = kb * kBlk + 4 * (tid & 31);
  const int64_t r0 = tn * kBlk + (tid >> 5);
  float4 v[16];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t r = r0 + 8 * i;
    if (r < N && k < K) v[i] = *reinterpret_cast<const float4*>(x + r * K + k);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
  amax = row16_max(amax);
  amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
  amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
  if ((tid & 63) == 0) part[tid >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  float d, id;
  f8_scale(amax, d, id);
  if (tid == 0) scales[blockIdx.x] = d;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + 8 * i;
    if (r < N && k < K)
      *reinterpret_cast<uint32_t*>(codes + r * K + k) = f8_pack4(v[i].x, v[i].y, v[i].z, v[i].w, id);
  }
}

// ---------------------------------------------------------------- product, few src1 rows

// A lane's two 16-byte pieces of block kb of a row; pieces past K are zero
// (both operands' are: an e4m3 NaN times zero is not zero).
__device__ __forceinline__ void load_block(const uint8_t* __restrict__ row, int kb, int g, int K,
                                           uint4& lo, uint4& hi) {
  const int k0 = kb * kBlk + 16 * g;
  const uint4 z = make_uint4(0, 0, 0, 0);
  if ((kb + 1) * kBlk <= K) {                       // uniform: a whole block
    lo = *reinterpret_cast<const uint4*>(row + k0);
    hi = *reinterpret_cast<const uint4*>(row + k0 + 64);
  } else {
    lo = z; hi = z;
    if (k0 < K) lo = *reinterpret_cast<const uint4*>(row + k0);
    if (k0 + 64 < K) hi = *reinterpret_cast<const uint4*>(row + k0 + 64);
  }
}

__device__ __forceinline__ void widen_block(const uint4& lo, const uint4& hi, v8h (&v)[4]) {
  v[0] = widen(lo.x, lo.y);
  v[1] = widen(lo.z, lo.w);
  v[2] = widen(hi.x, hi.y);
  v[3] = widen(hi.z, hi.w);
}

// acc += s * (the block dot of 16 weight rows and 16 src1 rows).
__device__ __forceinline__ void block_fma(const v8h (&w)[4], const v8h (&a)[4], float s, v4f& acc) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i], a[i], c, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(c[e], s, acc[e]);
}

// Each workgroup takes 16 weight rows and all src1 rows, at most NT tiles of 16
// (codes and scales as INIT or the caller left them), its waves the K blocks
// wave, wave + W, ... (together they read W * 128 consecutive bytes of each
// weight row); the waves' partial tiles are added in LDS in wave order.  32
// weight rows per workgroup, sharing each src1 operand, measured slower (4096 x
// 4096, M = 5 / 16: 11.9 / 13.2 us against 10.0 / 11.3).
template <int NT>
__global__ __launch_bounds__(512) void k_f8_skinny(
    const uint8_t* __restrict__ w, const float* __restrict__ wsc, const uint8_t* __restrict__ a,
    const float* __restrict__ asc, int M, int N, int K, float* __restrict__ dst) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int U = 4;                              // blocks in flight per wave
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int W = blockDim.x >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int nkb = (K + kBlk - 1) / kBlk;
  const int n0 = blockIdx.x * 16;

  const uint8_t* const wrow = w + (int64_t)min(n0 + i16, N - 1) * K;
  const float* const wscr = wsc + (int64_t)(n0 / kBlk) * nkb;
  const uint8_t* arow[NT];
  const float* ascr[NT];
  bool live[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = 16 * t + i16;
    live[t] = m < M;
    arow[t] = a + (int64_t)(live[t] ? m : 0) * K;
    ascr[t] = asc + (int64_t)(live[t] ? m : 0) * nkb;
  }

  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = (v4f){0.f, 0.f, 0.f, 0.f};

  for (int kb0 = wave; kb0 < nkb; kb0 += W * U) {
    uint4 wl[U], wh[U], al[U][NT], ah[U][NT];
    float sa[U][NT], sw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(kb0 + u * W, nkb - 1);       // valid addresses throughout
      load_block(wrow, kb, g, K, wl[u], wh[u]);
      sw[u] = wscr[kb];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        al[u][t] = ah[u][t] = make_uint4(0, 0, 0, 0);
        sa[u][t] = 0.0f;
        if (live[t]) {
          load_block(arow[t], kb, g, K, al[u][t], ah[u][t]);
          sa[u][t] = ascr[t][kb];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb0 + u * W >= nkb) continue;                // uniform
      v8h wv[4];
      widen_block(wl[u], wh[u], wv);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v8h av[4];
        widen_block(al[u][t], ah[u][t], av);
        block_fma(wv, av, sw[u] * sa[u][t], acc[t]);
      }
    }
  }

  // join the waves' partial tiles: [wave][m][n], n fastest
  float* const part = reinterpret_cast<float*>(lds);
  constexpr int TILE = 256 * NT;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    *reinterpret_cast<v4f*>(part + wave * TILE + (16 * t + i16) * 16 + 4 * g) = acc[t];
  __syncthreads();
  for (int e = tid; e < TILE; e += blockDim.x) {
    float s = part[e];
    for (int v = 1; v < W; ++v) s += part[v * TILE + e];
    const int m = e / 16, n = n0 + e % 16;
    if (m < M && n < N) dst[(int64_t)m * N + n] = s;
  }
}

// A few src1 rows given as f32: every workgroup quantizes them into LDS itself
// (16 lanes per block; no INIT launch, no workspace), then walks groups of
// 16 weight rows, blockIdx.x, blockIdx.x + gridDim.x, ...  The first group's
// weights are requested before the quantization waits for src1, each next
// round's before the current one is computed; the barriers wait for LDS only,
// so that these loads stay under way.  Rounds of U blocks per wave.
template <int ROUNDS>
__global__ __launch_bounds__(512) void k_f8_fused(
    const float* __restrict__ x, const uint8_t* __restrict__ w, const float* __restrict__ wsc,
    float* __restrict__ dst, int M, int N, int K, int groups) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int U = 4, W = 8;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int nkb = (K + kBlk - 1) / kBlk, pitch = nkb * kBlk + 16;   // 16: rows in different banks
  // codes [M][pitch], scales [M][nkb], the waves' partial tiles
  float* const sscale = reinterpret_cast<float*>(lds + M * pitch);
  float* const part = reinterpret_cast<float*>(lds + M * pitch + (M * nkb * 4 + 15) / 16 * 16);

  // src1: M * nkb <= 32 ROUNDS blocks of 128, all requested at once
  const int total = M * nkb;
  float4 p[ROUNDS], q[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int b = min((tid >> 4) + 32 * r, total - 1), m = b / nkb;
    const int k = (b - m * nkb) * kBlk + 8 * i16;
    p[r] = q[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < K) {
      const float4* s = reinterpret_cast<const float4*>(x + (int64_t)m * K + k);
      p[r] = s[0]; q[r] = s[1];
    }
  }
  struct Round { uint4 lo[U], hi[U]; float s[U]; };
  const auto load = [&](Round& r, int group, int kb0) {
    const uint8_t* const row = w + (int64_t)min(16 * group + i16, N - 1) * K;
    const float* const sc = wsc + (int64_t)(16 * group / kBlk) * nkb;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(kb0 + wave + u * W, nkb - 1);
      load_block(row, kb, g, K, r.lo[u], r.hi[u]);
      r.s[u] = sc[kb];
    }
  };
  int group = blockIdx.x, kb0 = 0;
  Round cur;
  load(cur, group, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int b = (tid >> 4) + 32 * r;
    float d;
    const uint2 c = f8_row_block(p[r], q[r], d);
    if (b < total) {
      const int m = b / nkb;
      *reinterpret_cast<uint2*>(lds + m * pitch + (b - m * nkb) * kBlk + 8 * i16) = c;
      if (i16 == 0) sscale[b] = d;
    }
  }
  lds_barrier();

  v4f acc = {0.f, 0.f, 0.f, 0.f};
  while (group < groups) {
    const bool last = kb0 + W * U >= nkb;
    const int ngroup = last ? group + (int)gridDim.x : group, nkb0 = last ? 0 : kb0 + W * U;
    Round next;
    if (ngroup < groups) load(next, ngroup, nkb0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + wave + u * W;
      if (kb >= nkb) continue;                         // uniform
      uint4 al = make_uint4(0, 0, 0, 0), ah = al;
      float sa = 0.0f;
      if (i16 < M) {
        const uint8_t* const c = lds + i16 * pitch + kb * kBlk + 16 * g;
        al = *reinterpret_cast<const uint4*>(c);
        ah = *reinterpret_cast<const uint4*>(c + 64);
        sa = sscale[i16 * nkb + kb];
      }
      v8h wv[4], av[4];
      widen_block(cur.lo[u], cur.hi[u], wv);
      widen_block(al, ah, av);
      block_fma(wv, av, cur.s[u] * sa, acc);
    }
    if (last) {
      if (i16 < M) *reinterpret_cast<v4f*>(part + (wave * M + i16) * 16 + 4 * g) = acc;
      lds_barrier();
      for (int e = tid; e < 16 * M; e += 512) {
        float s = part[e];
#pragma unroll
        for (int v = 1; v < W; ++v) s += part[v * 16 * M + e];
        const int n = 16 * group + e % 16;
        if (n < N) dst[(int64_t)(e / 16) * N + n] = s;
      }
      lds_barrier();                                   // the partial tiles are read
      acc = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    cur = next;
    group = ngroup;
    kb0 = nkb0;
  }
}

// ---------------------------------------------------------------- product, many src1 rows

// Output tile of BN weight rows x BM src1 rows per workgroup, one block of 128 k
// per stage, STAGES stages in LDS, both operands copied there straight from
// memory as codes and widened in registers.  (src1 widened once by INIT,
// binary16 in LDS, spares the widening and costs twice the copies' bytes: about
// 3% slower.  Stages of half a block, twice as many: twice the barriers and
// 64-byte rows in the copies, 14336 x 4096, M = 128 / 512 39.3 / 78.8 us against
// 31.6 / 75.5.  More stages: no faster.)
//
// A block is eight steps of 16 k (q); each MFMA adds to the block dot c, and the
// fp32 sums take c * (dw * ds).  Operands are read two steps at a time, ahead of
// the products.  The one barrier per stage stands before its last q's MFMAs:
// there every wave has read the whole stage, so the copy of the stage STAGES
// further can start, and the next stage has arrived, so its first operands are
// read behind those MFMAs.
//
// In LDS a row's eight 16-byte chunks are permuted by (row / 2) % 8, so that the
// 16 rows of an operand read lie in different banks.  Lane half h of an MFMA
// holds k 32 p + 16 h + 8 (q % 2) .. + 7, p = q / 2: one chunk serves two q.
//
// What bounds it, at 512 x 128256 x 4096 (128 x 256 tiles): 613 us, 880 TFLOP/s.
// Without the copies, the widening, the scaling and the barriers the same MFMAs
// take 407 us (1320 TFLOP/s, what the card's power leaves of the matrix cores; a
// library product of 8192^3 in binary16 reaches 1285), with LDS reads and
// barriers 490 to 520.  The copies (48 KB per workgroup and block, 85% L2 hits)
// keep the address units 58% busy.
template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, 1) void k_f8_wide(
    const uint8_t* __restrict__ w, const float* __restrict__ wsc, const uint8_t* __restrict__ a,
    const float* __restrict__ asc, int M, int N, int K, float* __restrict__ dst, int tiles_m,
    int tiles, int split, int kchunk) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  constexpr int TM = WTM / 32, TN = WTN / 32;
  constexpr int kA = BN * kBlk, kS = kA + BM * kBlk;           // stage: weights, src1, its scales
  constexpr int STAGE = kS + BM * 4;
  constexpr int WL = BN / 8 / NW, AL = BM / 8 / NW;            // pieces of 8 rows, 1 KB, per wave
  constexpr int kCopies = WL + AL + 1;
  static_assert((STAGES - 1) * kCopies < 64, "wait counts");
  static_assert(kBlk % WTN == 0, "one weight scale per wave and stage");
  static_assert(BN % (8 * NW) == 0 && BM % (8 * NW) == 0 && BM % 64 == 0 && NW % 2 == 0, "whole pieces");
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WAVES_M, wn = wave / WAVES_M;
  const int h = lane >> 5, l32 = lane & 31;
  const int nkb = (K + kBlk - 1) / kBlk;
  const int t = xcd_remap(blockIdx.x, tiles * split);
  const int z = t / tiles, tt = t - z * tiles;
  const int tm = tt % tiles_m, tn = tt / tiles_m;    // m fastest: same weight tile adjacent
  const int m0 = tm * BM, n0 = tn * BN;
  const int kb0 = z * kchunk, kb1 = min(kb0 + kchunk, nkb);
  const int s1 = kb1 - kb0;                          // stages

  // this lane's part of each piece
  const uint8_t* const wbase = w + (int64_t)n0 * K;
  const uint8_t* const abase = a + (int64_t)m0 * nkb * kBlk;
  const int chunk = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
  uint32_t woff[WL], aoff[AL];
#pragma unroll
  for (int i = 0; i < WL; ++i)
    woff[i] = (uint32_t)min((i * NW + wave) * 8 + (lane >> 3), N - 1 - n0) * (uint32_t)K;
#pragma unroll
  for (int i = 0; i < AL; ++i)
    aoff[i] = (uint32_t)min((i * NW + wave) * 8 + (lane >> 3), M - 1 - m0) * (uint32_t)nkb * kBlk;
  // every wave issues the same number of copies (the rows' scales are copied
  // by several waves, to the same place)
  const int sm = (wave % (BM / 64)) * 64;
  const float* const sbase = asc + (int64_t)m0 * nkb;
  const uint32_t soff = (uint32_t)min(sm + lane, M - 1 - m0) * (uint32_t)nkb;
  const uint32_t lds0 = lds_offset(lds);
  auto copy_stage = [&](int s, int buf) {
    const uint32_t base = lds0 + buf * STAGE;
    // past a weight row: its own first codes, which meet the zeros that src1
    // is padded with (if one is a NaN, so is the whole row's result)
    const uint32_t ka = (kb0 + s) * kBlk + chunk * 16, kw = (int)ka < K ? ka : 0;
#pragma unroll
    for (int i = 0; i < WL; ++i) copy16(base + (i * NW + wave) * 1024, wbase, woff[i] + kw);
#pragma unroll
    for (int i = 0; i < AL; ++i) copy16(base + kA + (i * NW + wave) * 1024, abase, aoff[i] + ka);
    copy4(base + kS + 4 * sm, sbase, 4 * (soff + kb0 + s));
  };
  const int nrow = min(n0 + wn * WTN, N - 1);
  const float* const wscr = wsc + (int64_t)(nrow / kBlk) * nkb;

  float acc[TN][TM][16];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int wrow = (wn * WTN + l32) * kBlk, arow = kA + (wm * WTM + l32) * kBlk;
  const int x8 = (l32 >> 1) & 7;
  uint4 wr[2][TN], ar[2][TM];
  // the operands of steps 2 p and 2 p + 1 (p = 0..3) into register set p % 2
  auto read = [&](const uint8_t* base, int p) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
      wr[p % 2][i] = *reinterpret_cast<const uint4*>(base + wrow + 32 * i * kBlk + 16 * ((2 * p + h) ^ x8));
#pragma unroll
    for (int j = 0; j < TM; ++j)
      ar[p % 2][j] = *reinterpret_cast<const uint4*>(base + arow + 32 * j * kBlk + 16 * ((2 * p + h) ^ x8));
  };

#pragma unroll
  for (int s = 0; s < STAGES; ++s)
    if (s < s1) copy_stage(s, s);
  if (s1 >= STAGES) wait_copies<(STAGES - 1) * kCopies>();
  else wait_copies<0>();
  __builtin_amdgcn_s_barrier();
  read(lds, 0);

  float sw = wscr[kb0];
  int buf = 0;
  for (int s = 0; s < s1; ++s) {
    const uint8_t* const base = lds + buf * STAGE;
    const int next = buf + 1 == STAGES ? 0 : buf + 1;
    v16f c[TN][TM];
    float sc[TM];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q % 2 == 1 && q < 7) read(base, q / 2 + 1);
      if (q == 7) {
        // the next stage is here and this wave's reads of this one are done
        if (s + STAGES - 1 < s1) wait_copies<(STAGES - 2) * kCopies>();
        else wait_copies<0>();
        __builtin_amdgcn_s_barrier();
        if (s + STAGES < s1) copy_stage(s + STAGES, buf);
        read(lds + next * STAGE, 0);
      }
      __builtin_amdgcn_sched_barrier(0);             // the reads stay ahead of the products
      if (q == 1) {
        const float* const ss = reinterpret_cast<const float*>(base + kS) + wm * WTM + l32;
#pragma unroll
        for (int j = 0; j < TM; ++j) sc[j] = sw * ss[32 * j];
        sw = wscr[min(kb0 + s + 1, nkb - 1)];
      }
      v8h av[TM];
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const uint4 v = ar[(q / 2) % 2][j];
        av[j] = q % 2 == 0 ? widen(v.x, v.y) : widen(v.z, v.w);
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const uint4 v = wr[(q / 2) % 2][i];
        const v8h wv = q % 2 == 0 ? widen(v.x, v.y) : widen(v.z, v.w);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
          if (q == 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) c[i][j][r] = 0.0f;
          }
          c[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wv, av[j], c[i][j], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(c[i][j][r], sc[j], acc[i][j][r]);
    buf = next;
  }

  // lane: src1 row of column l32, weight rows 8 q + 4 h + 0..3
  float* const out = dst + (int64_t)z * M * N;
  const bool vec = N % 4 == 0 && (uintptr_t)dst % 16 == 0;
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int m = m0 + wm * WTM + 32 * j + l32;
      if (m >= M) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = n0 + wn * WTN + 32 * i + 8 * q + 4 * h;
        float* const p = out + (int64_t)m * N + n;
        if (vec && n < N) {
          *reinterpret_cast<float4*>(p) = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                      acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < N) p[e] = acc[i][j][4 * q + e];
        }
      }
    }
}

// dst = the sum of its slices, in order; the loads of four slices are under way at once.
template <bool kVec>
__global__ __launch_bounds__(256) void k_join_slices(const float* __restrict__ part,
                                                     float* __restrict__ dst, int64_t n, int slices) {
  constexpr int V = kVec ? 4 : 1;
  typedef float vec __attribute__((ext_vector_type(V)));
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i * V < n; i += (int64_t)gridDim.x * 256) {
    vec s = *reinterpret_cast<const vec*>(part + i * V);
    for (int z0 = 1; z0 < slices; z0 += 4) {
      vec v[4];
#pragma unroll
      for (int z = 0; z < 4; ++z)
        v[z] = *reinterpret_cast<const vec*>(part + (int64_t)min(z0 + z, slices - 1) * n + i * V);
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (z0 + z < slices) s += v[z];
    }
    *reinterpret_cast<vec*>(dst + i * V) = s;
  }
}

}  // namespace

hipError_t launch_join_slices(const float* part, float* dst, int64_t n, int slices, hipStream_t s) {
  const bool vec = n % 4 == 0 && (uintptr_t)dst % 16 == 0;       // part is 256-byte aligned
  const int64_t items = vec ? n / 4 : n, grid = (items + 255) / 256;
  const dim3 g((unsigned)(grid < 4096 ? grid : 4096));
  if (vec) hipLaunchKernelGGL((k_join_slices<true>), g, dim3(256), 0, s, part, dst, n, slices);
  else hipLaunchKernelGGL((k_join_slices<false>), g, dim3(256), 0, s, part, dst, n, slices);
  return hipGetLastError();
}

hipError_t launch_f8_quantize(const float* x, uint8_t* codes, float* scales, int64_t nrows,
                              int64_t k, int block_rows, hipStream_t s, int64_t pitch) {
  const int64_t nkb = (k + kBlk - 1) / kBlk;
  if (block_rows == 1) {
    const int64_t nblocks = nrows * nkb;
    const int64_t grid = (nblocks + 15) / 16;
    hipLaunchKernelGGL(k_f8_quantize_rows, dim3((unsigned)(grid < kMaxGridX ? grid : kMaxGridX)),
                       dim3(256), 0, s, x, codes, scales, (int)k, (int)(pitch ? pitch : k), (int)nkb,
                       nblocks);
  } else {
    const int64_t grid = (nrows + kBlk - 1) / kBlk * nkb;
    hipLaunchKernelGGL(k_f8_quantize_tiles, dim3((unsigned)grid), dim3(256), 0, s, x, codes,
                       scales, nrows, (int)k, (int)nkb);
  }
  return hipGetLastError();
}

namespace {

template <int NT>
hipError_t skinny(const F8Plan& p, const uint8_t* w, const float* wsc, const uint8_t* a,
                  const float* asc, float* dst, int M, int N, int K, hipStream_t s) {
  if (M > 16 * NT) return hipErrorInvalidValue;       // the plan gives it no more rows
  hipLaunchKernelGGL((k_f8_skinny<NT>), dim3((unsigned)p.grid_n),
                     dim3(64 * p.waves), p.lds, s, w, wsc, a, asc, M, N, K, dst);
  return hipGetLastError();
}

template <int ROUNDS>
hipError_t fused(const F8Plan& p, const float* x, const uint8_t* w, const float* wsc, float* dst,
                 int M, int N, int K, hipStream_t s) {
  hipLaunchKernelGGL((k_f8_fused<ROUNDS>), dim3((unsigned)p.grid_n), dim3(512), p.lds, s, x, w,
                     wsc, dst, M, N, K, (N + 15) / 16);
  return hipGetLastError();
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES>
hipError_t wide(const F8Plan& p, const uint8_t* w, const float* wsc, const uint8_t* a,
                const float* asc, float* dst, int M, int N, int K, void* ws, hipStream_t s) {
  constexpr int kLds = STAGES * ((BN + BM) * kBlk + BM * 4);
  auto* const kern = k_f8_wide<BM, BN, WAVES_M, WAVES_N, STAGES>;
  if (kLds > 65536) {
    static std::atomic<uint64_t> raised{0};          // devices whose limit is set already
    const hipError_t e = raise_lds(reinterpret_cast<const void*>(kern), kLds, raised);
    if (e != hipSuccess) return e;
  }
  float* const out = p.split > 1 ? reinterpret_cast<float*>((uint8_t*)ws + p.off_part) : dst;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles_m * p.tiles_n * p.split)),
                     dim3(64 * WAVES_M * WAVES_N), kLds, s, w, wsc, a, asc, M, N, K, out,
                     (int)p.tiles_m, (int)(p.tiles_m * p.tiles_n), p.split, (int)p.kchunk);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.split > 1) e = launch_join_slices(out, dst, (int64_t)M * N, p.split, s);
  return e;
}

}  // namespace

hipError_t launch_f8_product(const F8Plan& p, const uint8_t* w, const float* wsc, const float* x,
                             const uint8_t* a, const float* asc, float* dst, int M, int N, int K,
                             void* ws, hipStream_t s) {
  if (p.kind == F8_FUSED) {
    if (p.nt == 1) return fused<1>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 2) return fused<2>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 4) return fused<4>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 8) return fused<8>(p, x, w, wsc, dst, M, N, K, s);
    return hipErrorInvalidValue;
  }
  if (p.kind == F8_WIDE) {
    uint8_t* const rows = (uint8_t*)ws + p.off_a;
    const int64_t nkb = (K + kBlk - 1) / kBlk;
    hipError_t e = hipSuccess;
    if (x) {                                          // INIT
      float* const scales = reinterpret_cast<float*>((uint8_t*)ws + p.off_as);
      e = launch_f8_quantize(x, rows, scales, M, K, 1, s, nkb * kBlk);
      a = rows;
      asc = scales;
    } else if (K % kBlk) {
      const int64_t pieces = 8 * (int64_t)M * nkb, grid = (pieces + 255) / 256;
      hipLaunchKernelGGL(k_f8_pad, dim3((unsigned)(grid < kMaxGridX ? grid : kMaxGridX)), dim3(256),
                         0, s, a, rows, K, (int)nkb, pieces);
      e = hipGetLastError();
      a = rows;
    }
    if (e != hipSuccess) return e;
    if (p.bm == 128 && p.bn == 256) return wide<128, 256, 2, 4, 3>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    if (p.bm == 128 && p.bn == 128) return wide<128, 128, 2, 4, 4>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    if (p.bm == 64 && p.bn == 128) return wide<64, 128, 2, 4, 4>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    if (p.bm == 64 && p.bn == 64) return wide<64, 64, 2, 2, 4>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    return hipErrorInvalidValue;
  }
  if (x) {                                            // INIT
    uint8_t* codes = (uint8_t*)ws + p.off_a;
    float* scales = reinterpret_cast<float*>((uint8_t*)ws + p.off_as);
    const hipError_t e = launch_f8_quantize(x, codes, scales, M, K, 1, s);
    if (e != hipSuccess) return e;
    a = codes;
    asc = scales;
  }
  if (p.nt == 1) return skinny<1>(p, w, wsc, a, asc, dst, M, N, K, s);
  if (p.nt == 2) return skinny<2>(p, w, wsc, a, asc, dst, M, N, K, s);
  return hipErrorInvalidValue;
}

}  // namespace qsg
