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
#include "device.h"
#include "kernels.h"

namespace qsg {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kBlk = kF8Block;          // 128

// Correctly rounded d and 1 / d of a block from its largest magnitude.
__device__ __forceinline__ void f8_scale(float amax, float& d, float& id) {
  d = fmaxf(amax / 448.0f, __builtin_bit_cast(float, 0x00800000u));   // 2^-126
  id = 1.0f / d;
}

// Four e4m3 codes of fl32(v * id), little endian.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float id) {
#pragma clang fp contract(off)
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * id, b * id, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * id, d * id, w, true);
  return (uint32_t)w;
}

__device__ __forceinline__ float amax8(const float4& a, const float4& b) {
  return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
               fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
}

// Maximum over the 16 lanes of a DPP row, in every lane of it.
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, dpp_f<0xB1>(v));     // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp_f<0x4E>(v));     // quad_perm [2,3,0,1]
  v = fmaxf(v, dpp_f<0x141>(v));    // row_half_mirror
  v = fmaxf(v, dpp_f<0x140>(v));    // row_mirror
  return v;
}

// One 1 x 128 block by 16 lanes, 8 values each: lane i (0..15) passes the
// values at 8 i .. 8 i + 7 and gets their codes and the block's scale.
__device__ __forceinline__ uint2 f8_row_block(const float4& a, const float4& b, float& d) {
  float id;
  f8_scale(row16_max(amax8(a, b)), d, id);
  return make_uint2(f8_pack4(a.x, a.y, a.z, a.w, id), f8_pack4(b.x, b.y, b.z, b.w, id));
}

// ---------------------------------------------------------------- quantizer

// 1 x 128 blocks: 16 lanes per block, one 32-byte load and one 8-byte store
// per lane.  Bound: HBM (5 bytes per value).
__global__ __launch_bounds__(256) void k_f8_quantize_rows(const float* __restrict__ x,
                                                          uint8_t* __restrict__ codes,
                                                          float* __restrict__ scales, int K,
                                                          int nkb, int64_t nblocks) {
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
    if (k < K) *reinterpret_cast<uint2*>(codes + row * K + k) = c;
    if (i == 0) scales[blk] = d;
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

// Eight e4m3 codes as binary16 (exact; a NaN code becomes a NaN).
__device__ __forceinline__ v8h widen(uint32_t lo, uint32_t hi) {
  const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return (v8h){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

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

// Each wave takes 16 RT weight rows and NT tiles of 16 src1 rows over the K
// blocks wave, wave + W, ... (the workgroup together reads W * 128
// consecutive bytes of each weight row); the waves' partial tiles are added
// in LDS in wave order.  Weights go from memory to the matrix core's
// operand registers as loaded.  kFused: src1 is f32 and every workgroup
// quantizes it into LDS first (16 lanes per block), which saves the INIT
// launch while M is small.
template <int NT, int RT, bool kFused>
__global__ __launch_bounds__(512) void k_f8_skinny(
    const uint8_t* __restrict__ w, const float* __restrict__ wsc, const uint8_t* __restrict__ a,
    const float* __restrict__ asc, int M, int N, int K, float* __restrict__ dst) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int U = RT * NT >= 4 ? 2 : 4;           // blocks in flight per wave
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int W = blockDim.x >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int nkb = (K + kBlk - 1) / kBlk;
  const int n0 = blockIdx.x * 16 * RT, m0 = blockIdx.y * 16 * NT;

  const uint8_t* wrow[RT];
  const float* wscr[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int n = n0 + 16 * r + i16;
    wrow[r] = w + (int64_t)(n < N ? n : N - 1) * K;
    const int nt = n0 + 16 * r;
    wscr[r] = wsc + (int64_t)((nt < N ? nt : N - 1) / kBlk) * nkb;
  }

  // kFused: codes [m][nkb * 128] then scales [m][nkb], M <= 16 rows
  const int pitch = nkb * kBlk;
  float* const sscale = reinterpret_cast<float*>(lds + M * pitch);
  if constexpr (kFused) {
    const float* x = reinterpret_cast<const float*>(a);
    const int total = M * nkb;
    for (int b0 = (tid >> 4); b0 < total; b0 += blockDim.x >> 4) {
      const int m = b0 / nkb, kb = b0 - m * nkb;
      const int k = kb * kBlk + 8 * i16;
      float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
      if (k < K) {
        const float4* s = reinterpret_cast<const float4*>(x + (int64_t)m * K + k);
        p = s[0]; q = s[1];
      }
      float d;
      const uint2 c = f8_row_block(p, q, d);
      *reinterpret_cast<uint2*>(lds + m * pitch + k) = c;
      if (i16 == 0) sscale[b0] = d;
    }
  }

  const uint8_t* arow[NT];
  const float* ascr[NT];
  bool live[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = m0 + 16 * t + i16;
    live[t] = m < M;
    arow[t] = a + (int64_t)(live[t] ? m : 0) * K;
    ascr[t] = asc + (int64_t)(live[t] ? m : 0) * nkb;
  }

  v4f acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = (v4f){0.f, 0.f, 0.f, 0.f};

  // every wave runs the same number of rounds: the barrier inside is met by all
  for (int r0 = 0; r0 < nkb; r0 += W * U) {
    const int kb0 = r0 + wave;
    uint4 wl[U][RT], wh[U][RT], al[U][NT], ah[U][NT];
    float sa[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(kb0 + u * W, nkb - 1);       // valid addresses throughout
#pragma unroll
      for (int r = 0; r < RT; ++r) load_block(wrow[r], kb, g, K, wl[u][r], wh[u][r]);
      if constexpr (!kFused) {
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
    }
    if (kFused && r0 == 0) lds_barrier();             // the first weights are on their way by now
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + u * W;
      if (kb >= nkb) continue;                       // uniform
      if constexpr (kFused) {
        al[u][0] = ah[u][0] = make_uint4(0, 0, 0, 0);
        sa[u][0] = 0.0f;
        if (i16 < M) {
          const uint8_t* p = lds + i16 * pitch + kb * kBlk + 16 * g;
          al[u][0] = *reinterpret_cast<const uint4*>(p);
          ah[u][0] = *reinterpret_cast<const uint4*>(p + 64);
          sa[u][0] = sscale[i16 * nkb + kb];
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const v8h w0 = widen(wl[u][r].x, wl[u][r].y), w1 = widen(wl[u][r].z, wl[u][r].w);
        const v8h w2 = widen(wh[u][r].x, wh[u][r].y), w3 = widen(wh[u][r].z, wh[u][r].w);
        const float sw = wscr[r][kb];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          v4f s = {0.f, 0.f, 0.f, 0.f};
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w0, widen(al[u][t].x, al[u][t].y), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w1, widen(al[u][t].z, al[u][t].w), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w2, widen(ah[u][t].x, ah[u][t].y), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_f16(w3, widen(ah[u][t].z, ah[u][t].w), s, 0, 0, 0);
          const float sc = sw * sa[u][t];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(s[e], sc, acc[r][t][e]);
        }
      }
    }
  }

  // join the waves' partial tiles: [wave][tile][m][n], n fastest
  __syncthreads();                                   // kFused: the codes are done with
  float* const part = reinterpret_cast<float*>(lds);
  constexpr int TILE = 256 * RT * NT;
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<v4f*>(part + wave * TILE + (16 * t + i16) * 16 * RT + 16 * r + 4 * g) = acc[r][t];
  __syncthreads();
  for (int e = tid; e < TILE; e += blockDim.x) {
    float s = part[e];
    for (int v = 1; v < W; ++v) s += part[v * TILE + e];
    const int m = m0 + e / (16 * RT), n = n0 + e % (16 * RT);
    if (m < M && n < N) dst[(int64_t)m * N + n] = s;
  }
}

// ---------------------------------------------------------------- product, many src1 rows

typedef __attribute__((address_space(1))) const void gvoid;
typedef __attribute__((address_space(3))) void lvoid;

// Output tile of BN weight rows x BM src1 rows per workgroup,
// one block of 128 k per stage.  Both operands' stages go from memory
// straight into LDS (16 bytes per lane), kStages buffers deep, the rows'
// eight 16-byte chunks permuted by the row's low three bits so that the
// operand reads (32 rows at one chunk) spread over the banks.
template <int BM, int BN, int WAVES_M, int WAVES_N, int kStages>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, 1) void k_f8_wide(
    const uint8_t* __restrict__ w, const float* __restrict__ wsc, const uint8_t* __restrict__ a,
    const float* __restrict__ asc, int M, int N, int K, float* __restrict__ dst, int tiles_m,
    int tiles, int split, int kchunk) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  constexpr int TM = WTM / 32, TN = WTN / 32;
  static_assert(kBlk % WTN == 0, "one weight scale per wave and stage");
  constexpr int ROWS = BM + BN;
  constexpr int STAGE = ROWS * kBlk + BM * 4;        // codes, then the src1 rows' scales
  constexpr int LOADS = ROWS / 8 / NW;               // 8-row pieces per wave and stage
  static_assert(ROWS % (8 * NW) == 0 && BM % 64 == 0, "whole pieces");
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

  // this lane's part of each 8-row piece: row base + lane / 8, the chunk that
  // belongs at position lane % 8
  const uint8_t* const wbase = w + (int64_t)n0 * K;
  const uint8_t* const abase = a + (int64_t)m0 * K;
  const int chunk = (lane & 7) ^ (lane >> 3);
  uint32_t off[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int r = (i * NW + wave) * 8 + (lane >> 3);
    const int rr = r < BN ? min(r, N - 1 - n0) : min(r - BN, M - 1 - m0);
    off[i] = (uint32_t)rr * (uint32_t)K;
  }

  auto load = [&](int kb, int buf) {
    uint8_t* const base = lds + buf * STAGE;
    int k = kb * kBlk + chunk * 16;
    if (k >= K) k = 0;                               // past the row: any valid bytes, zeroed below
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = (i * NW + wave) * 8;             // uniform
      const uint8_t* const src = (r < BN ? wbase : abase) + (off[i] + (uint32_t)k);
      __builtin_amdgcn_global_load_lds((gvoid*)src, (lvoid*)(base + r * kBlk), 16, 0, 0);
    }
    if (wave < BM / 64) {
      const int m = min(m0 + 64 * wave + lane, M - 1);
      __builtin_amdgcn_global_load_lds((gvoid*)(asc + (int64_t)m * nkb + kb),
                                       (lvoid*)(base + ROWS * kBlk + 256 * wave), 4, 0, 0);
    }
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

  const int ksteps = kb1 - kb0;
  for (int s = 0; s < kStages - 1; ++s)
    if (s < ksteps) load(kb0 + s, s);

  int buf = 0;
  for (int s = 0; s < ksteps; ++s) {
    const int kb = kb0 + s;
    __syncthreads();
    const int next = s + kStages - 1;
    if (next < ksteps) load(kb0 + next, buf == 0 ? kStages - 1 : buf - 1);
    uint8_t* const base = lds + buf * STAGE;
    if ((kb + 1) * kBlk > K) {                       // the chunks past K become zero in both operands
      const int valid = (K - kb * kBlk) / 16;
      for (int r = tid; r < ROWS; r += 64 * NW)
        for (int c = valid; c < 8; ++c)
          *reinterpret_cast<uint4*>(base + r * kBlk + 16 * (c ^ (r & 7))) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    const float sw = wscr[kb];
    // lane half h holds chunk 2 q + h of its row: 8 k for each of two MFMAs
    auto operand_at = [&](int row, int q, v8h& x, v8h& y) {
      const uint4 v = *reinterpret_cast<const uint4*>(base + row * kBlk + 16 * ((2 * q + h) ^ (row & 7)));
      x = widen(v.x, v.y);
      y = widen(v.z, v.w);
    };
    v8h av[TM][8];
    float sc[TM];
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int row = wm * WTM + 32 * j + l32;
#pragma unroll
      for (int q = 0; q < 4; ++q) operand_at(BN + row, q, av[j][2 * q], av[j][2 * q + 1]);
      sc[j] = sw * *reinterpret_cast<const float*>(base + ROWS * kBlk + 4 * row);
    }
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      v8h wv[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) operand_at(wn * WTN + 32 * i + l32, q, wv[2 * q], wv[2 * q + 1]);
      v16f c[TM];
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) c[j][r] = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q)
#pragma unroll
        for (int j = 0; j < TM; ++j)
          c[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(wv[q], av[j][q], c[j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(c[j][r], sc[j], acc[i][j][r]);
    }
    buf = buf + 1 == kStages ? 0 : buf + 1;
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

}  // namespace

hipError_t launch_f8_quantize(const float* x, uint8_t* codes, float* scales, int64_t nrows,
                              int64_t k, int block_rows, hipStream_t s) {
  const int64_t nkb = (k + kBlk - 1) / kBlk;
  if (block_rows == 1) {
    const int64_t nblocks = nrows * nkb;
    const int64_t grid = (nblocks + 15) / 16;
    hipLaunchKernelGGL(k_f8_quantize_rows, dim3((unsigned)(grid < kMaxGridX ? grid : kMaxGridX)),
                       dim3(256), 0, s, x, codes, scales, (int)k, (int)nkb, nblocks);
  } else {
    const int64_t grid = (nrows + kBlk - 1) / kBlk * nkb;
    hipLaunchKernelGGL(k_f8_quantize_tiles, dim3((unsigned)grid), dim3(256), 0, s, x, codes,
                       scales, nrows, (int)k, (int)nkb);
  }
  return hipGetLastError();
}

namespace {

template <int NT, int RT, bool kFused>
hipError_t skinny(const F8Plan& p, const uint8_t* w, const float* wsc, const uint8_t* a,
                  const float* asc, float* dst, int M, int N, int K, hipStream_t s) {
  hipLaunchKernelGGL((k_f8_skinny<NT, RT, kFused>), dim3((unsigned)p.grid_n, (unsigned)p.grid_m),
                     dim3(64 * p.waves), p.lds, s, w, wsc, a, asc, M, N, K, dst);
  return hipGetLastError();
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int kStages>
hipError_t wide(const F8Plan& p, const uint8_t* w, const float* wsc, const uint8_t* a,
                const float* asc, float* dst, int M, int N, int K, void* ws, hipStream_t s) {
  constexpr int kLds = kStages * ((BM + BN) * kBlk + BM * 4);
  auto* const kern = k_f8_wide<BM, BN, WAVES_M, WAVES_N, kStages>;
  if (kLds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  float* const out = p.split > 1 ? reinterpret_cast<float*>((uint8_t*)ws + p.off_part) : dst;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles_m * p.tiles_n * p.split)),
                     dim3(64 * WAVES_M * WAVES_N), kLds, s, w, wsc, a, asc, M, N, K, out,
                     (int)p.tiles_m, (int)(p.tiles_m * p.tiles_n), p.split, (int)p.kchunk);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.split > 1) e = launch_splitk_reduce(out, dst, (int64_t)M * N, p.split, s);
  return e;
}

}  // namespace

hipError_t launch_f8_product(const F8Plan& p, const uint8_t* w, const float* wsc, const float* x,
                             const uint8_t* a, const float* asc, float* dst, int M, int N, int K,
                             void* ws, hipStream_t s) {
  if (p.kind == F8_FUSED)
    return p.rt == 2 ? skinny<1, 2, true>(p, w, wsc, (const uint8_t*)x, nullptr, dst, M, N, K, s)
                     : skinny<1, 1, true>(p, w, wsc, (const uint8_t*)x, nullptr, dst, M, N, K, s);
  if (x) {                                            // INIT
    uint8_t* codes = (uint8_t*)ws + p.off_a;
    float* scales = reinterpret_cast<float*>((uint8_t*)ws + p.off_as);
    const hipError_t e = launch_f8_quantize(x, codes, scales, M, K, 1, s);
    if (e != hipSuccess) return e;
    a = codes;
    asc = scales;
  }
  if (p.kind == F8_WIDE) {
    if (p.bm == 128 && p.bn == 256) return wide<128, 256, 2, 4, 3>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    if (p.bm == 128 && p.bn == 128) return wide<128, 128, 2, 2, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    if (p.bm == 64 && p.bn == 128) return wide<64, 128, 1, 4, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
    return hipErrorInvalidValue;
  }
#define QSG_F8(NT_, RT_) \
  if (p.nt == NT_ && p.rt == RT_) return skinny<NT_, RT_, false>(p, w, wsc, a, asc, dst, M, N, K, s);
  QSG_F8(1, 1) QSG_F8(1, 2) QSG_F8(2, 1) QSG_F8(2, 2) QSG_F8(4, 1) QSG_F8(4, 2)
#undef QSG_F8
  return hipErrorInvalidValue;
}

}  // namespace qsg
