// Microscaled 4-bit floating point (MXFP4): quantizer, its inverse and the
// product, for gfx950.
//
// Product: dst[m][n] = sum_b 2^(ea[m][b] + ew[n][b]) S_b[m][n], S_b the dot of the
// 32 code pairs of block b, on the scaled matrix instructions
// (v_mfma_scale_f32_16x16x128_f8f6f4 and 32x32x64, both operands e2m1), which
// take the blocks' scale bytes as they are stored.  Code products are multiples
// of 1/4 up to 36, so S_b is exact in 13 bits; an instruction's sum and the fp32
// accumulation are exact too while the blocks' scales lie within a few binades
// (measured: 0 with scales within 2^4 of each other, 1e-7 to 2.6e-7 in the
// 2-norm, K up to 16384, with scales spread over 2^24).  src1 is operand A and the
// weights operand B, so that 16 or 32 neighbouring lanes hold neighbouring
// outputs of one row.
//
// A lane's operand is one whole block: 16 consecutive bytes of codes and one
// byte of scale.
#include <type_traits>

#include "kernels.h"
#include "mx4.h"

namespace qsg {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kGrp = kMx4Group;         // 128: four blocks, one dword of scale bytes

// Sums that are complete here: the compiler may move a scaled matrix instruction
// down to its result's first use, into a branch that leaves out lanes whose operands
// it needs.
template <class T>
__device__ __forceinline__ void settle(T& sums) {
  asm volatile("" : "+v"(sums));
}

__device__ __forceinline__ v8i operand(const uint4& c) {
  return (v8i){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}

// ---------------------------------------------------------------- quantizer

// 16 lanes per group of 128 values: one 32-byte load, one 4-byte store of codes
// per lane.  Bound: HBM (4.53 bytes per value): 11008 x 4096 46 us, 4.4 TB/s; 511 x 4096
// 3.1 us.
__global__ __launch_bounds__(256) void k_mx4_quantize(const float* __restrict__ x,
                                                      uint8_t* __restrict__ codes,
                                                      uint32_t* __restrict__ scales, int K, int ng,
                                                      int64_t groups) {
  const int lane = threadIdx.x & 63, i = lane & 15;
  for (int64_t at = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); at < groups;
       at += (int64_t)gridDim.x * 16) {              // whole groups of 16 lanes
    const int64_t row = at / ng;
    const int k = (int)(at - row * ng) * kGrp + 8 * i;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (k < K) {                                     // K % 32 == 0: all 8 values or none
      const float4* p = reinterpret_cast<const float4*>(x + row * K + k);
      a = p[0]; b = p[1];
    }
    uint32_t bytes;
    const uint32_t c = mx4_group(a, b, k < K, lane, bytes);
    if (k < K) *reinterpret_cast<uint32_t*>(codes + (row * K + k) / 2) = c;
    if (i == 0) scales[at] = bytes;
  }
}

// Eight values per lane.  Bound: HBM: 11008 x 4096 33 us (6.2 TB/s, part of the codes
// from the last-level cache).
__global__ __launch_bounds__(256) void k_mx4_dequantize(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales,
                                                        float* __restrict__ y, int K, int ng,
                                                        int64_t pieces) {
  const int per = K / 8;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < pieces;
       at += (int64_t)gridDim.x * 256) {
    const int64_t row = at / per;
    const int p = (int)(at - row * per);
    const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + 4 * at);
    const int byte = scales[row * 4 * ng + p / 4];
    v2f v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = __builtin_amdgcn_ldexpf(v[j / 2][j % 2], byte - 127);
      if (byte == 255) f[j] = __builtin_nanf("");
    }
    float4* const out = reinterpret_cast<float4*>(y + 8 * at);
    out[0] = make_float4(f[0], f[1], f[2], f[3]);
    out[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// ---------------------------------------------------------------- product, few src1 rows

// A unit is 4 groups of 128 k of a row: lane group g holds block g of each, and the
// row's 16 scale bytes (one load: an access of a few bytes per row costs the address
// units as much as one of 64).
constexpr int kUnit = 4;
typedef uint32_t v4u __attribute__((ext_vector_type(4), aligned(4)));
struct Unit {
  uint4 c[kUnit];
  v4u s;
};

// Groups kb0 .. kb0 + 3 of a row; those past its end repeat the last one, blocks
// past K are zeros (what is stored there is not read).
__device__ __forceinline__ Unit load_unit(const uint8_t* __restrict__ codes,
                                          const uint8_t* __restrict__ scales, int kb0, int g, int K, int ng) {
  Unit r;
  const uint32_t* const sc = reinterpret_cast<const uint32_t*>(scales);
  if ((kb0 + kUnit) * kGrp <= K) {                    // uniform: a whole unit
#pragma unroll
    for (int u = 0; u < kUnit; ++u)
      r.c[u] = *reinterpret_cast<const uint4*>(codes + (kb0 + u) * (kGrp / 2) + 16 * g);
    r.s = *reinterpret_cast<const v4u*>(sc + kb0);
  } else {
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      const int kb = min(kb0 + u, ng - 1), k = kb * kGrp + 32 * g;
      r.c[u] = make_uint4(0, 0, 0, 0);
      r.s[u] = 0x7f7f7f7fu;
      if (k < K) {
        r.c[u] = *reinterpret_cast<const uint4*>(codes + k / 2);
        r.s[u] = sc[kb];
      }
    }
  }
  return r;
}

// Each workgroup takes 16 weight rows and all src1 rows, at most NT tiles of 16;
// its waves take units of 4 groups in turn (a wave's loads cover 256 consecutive
// bytes of each row); the waves' partial tiles are added in LDS in
// wave order.  Bound: latency (16 x 4096 x 4096 4.9 us a call, 32 x 1000 x 4128 4.4).
template <int NT>
__global__ __launch_bounds__(512) void k_mx4_skinny(
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ wsc, const uint8_t* __restrict__ a,
    const uint8_t* __restrict__ asc, int M, int N, int K, float* __restrict__ dst) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int W = blockDim.x >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int ng = (K + kGrp - 1) / kGrp;
  const int n0 = blockIdx.x * 16;

  const int64_t wr = min(n0 + i16, N - 1);
  const uint8_t* const wrow = w + wr * (K / 2);
  const uint8_t* const wsr = wsc + wr * 4 * ng;
  const uint8_t* arow[NT];
  const uint8_t* asr[NT];
  bool live[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int m = 16 * t + i16;
    live[t] = m < M;
    arow[t] = a + (int64_t)(live[t] ? m : 0) * (K / 2);
    asr[t] = asc + (int64_t)(live[t] ? m : 0) * 4 * ng;
  }
  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = (v4f){0.f, 0.f, 0.f, 0.f};

  for (int kb0 = wave * kUnit; kb0 < ng; kb0 += W * kUnit) {
    Unit ab[NT];
    const Unit wb = load_unit(wrow, wsr, kb0, g, K, ng);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      ab[t].s = (v4u){0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu};
#pragma unroll
      for (int u = 0; u < kUnit; ++u) ab[t].c[u] = make_uint4(0, 0, 0, 0);
      if (live[t]) ab[t] = load_unit(arow[t], asr[t], kb0, g, K, ng);
    }
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      if (kb0 + u >= ng) continue;                    // uniform
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            operand(ab[t].c[u]), operand(wb.c[u]), acc[t], 4, 4, 0, (int)(ab[t].s[u] >> (8 * g)), 0,
            (int)(wb.s[u] >> (8 * g)));
    }
  }

  // join the waves' partial tiles: [wave][m][n], n fastest
  float* const part = reinterpret_cast<float*>(lds);
  constexpr int TILE = 256 * NT;
#pragma unroll
  for (int t = 0; t < NT; ++t) settle(acc[t]);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave * TILE + (16 * t + 4 * g + e) * 16 + i16] = acc[t][e];
  __syncthreads();
  for (int e = tid; e < TILE; e += blockDim.x) {
    float s = part[e];
    for (int v = 1; v < W; ++v) s += part[v * TILE + e];
    const int m = e / 16, n = n0 + e % 16;
    if (m < M && n < N) dst[(int64_t)m * N + n] = s;
  }
}

// A few src1 rows given as f32: every workgroup quantizes them into LDS itself
// (16 lanes per group of 128; no INIT launch, no workspace), then walks groups of
// 16 weight rows, blockIdx.x, blockIdx.x + gridDim.x, ...  The first rows'
// weights are requested before the quantization waits for src1, each next
// round's before the current one is computed; the barriers wait for LDS only,
// so that these loads stay under way.  Bound: latency (launch, src1, weights): 1 x
// 4096 x 4096 4.6 us, 7 x 1000 x 4128 6.3.
template <int ROUNDS>
__global__ __launch_bounds__(512) void k_mx4_fused(
    const float* __restrict__ x, const uint8_t* __restrict__ w, const uint8_t* __restrict__ wsc,
    float* __restrict__ dst, int M, int N, int K, int tiles) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int U = kUnit, W = 8;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int ng = (K + kGrp - 1) / kGrp, pitch = ng * (kGrp / 2) + 16;   // 16: rows in different banks
  // codes [M][pitch], scales [M][ng] dwords, the waves' partial tiles
  uint32_t* const sscale = reinterpret_cast<uint32_t*>(lds + M * pitch);
  float* const part = reinterpret_cast<float*>(lds + M * pitch + (M * ng * 4 + 15) / 16 * 16);

  // src1: M * ng <= 32 ROUNDS groups of 128, all requested at once
  const int total = M * ng;
  float4 p[ROUNDS], q[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int b = min((tid >> 4) + 32 * r, total - 1), m = b / ng;
    const int k = (b - m * ng) * kGrp + 8 * i16;
    p[r] = q[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < K) {
      const float4* s = reinterpret_cast<const float4*>(x + (int64_t)m * K + k);
      p[r] = s[0]; q[r] = s[1];
    }
  }
  const auto load = [&](Unit& r, int tile, int kb0) {
    const int64_t row = min(16 * tile + i16, N - 1);
    r = load_unit(w + row * (K / 2), wsc + row * 4 * ng, min(kb0 + wave * U, ng - 1), g, K, ng);
  };
  int tile = blockIdx.x, kb0 = 0;
  Unit cur;
  load(cur, tile, 0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int b = (tid >> 4) + 32 * r, bc = min(b, total - 1), m = bc / ng;
    const int k = (bc - m * ng) * kGrp + 8 * i16;
    uint32_t bytes;
    const uint32_t c = mx4_group(p[r], q[r], k < K, lane, bytes);
    if (b < total) {
      *reinterpret_cast<uint32_t*>(lds + m * pitch + k / 2) = c;
      if (i16 == 0) sscale[b] = bytes;
    }
  }
  lds_barrier();

  v4f acc = {0.f, 0.f, 0.f, 0.f};
  while (tile < tiles) {
    const bool last = kb0 + W * U >= ng;
    const int ntile = last ? tile + (int)gridDim.x : tile, nkb0 = last ? 0 : kb0 + W * U;
    Unit next;
    if (ntile < tiles) load(next, ntile, nkb0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + wave * U + u;
      if (kb >= ng) continue;                          // uniform
      uint4 c = make_uint4(0, 0, 0, 0);
      uint32_t s = 0x7f7f7f7fu;
      if (i16 < M) {
        c = *reinterpret_cast<const uint4*>(lds + i16 * pitch + kb * (kGrp / 2) + 16 * g);
        s = sscale[i16 * ng + kb];
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          operand(c), operand(cur.c[u]), acc, 4, 4, 0, (int)(s >> (8 * g)), 0, (int)(cur.s[u] >> (8 * g)));
    }
    if (last) {
      settle(acc);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * g + e < M) part[(wave * M + 4 * g + e) * 16 + i16] = acc[e];
      lds_barrier();
      for (int e = tid; e < 16 * M; e += 512) {
        float s = part[e];
#pragma unroll
        for (int v = 1; v < W; ++v) s += part[v * 16 * M + e];
        const int n = 16 * tile + e % 16;
        if (n < N) dst[(int64_t)(e / 16) * N + n] = s;
      }
      lds_barrier();                                   // the partial tiles are read
      acc = (v4f){0.f, 0.f, 0.f, 0.f};
    }
    cur = next;
    tile = ntile;
    kb0 = nkb0;
  }
}

// ---------------------------------------------------------------- product, many src1 rows

// Output tile of BM src1 rows x BN weight rows per workgroup; a stage is 256 k
// (128 bytes of codes and two dwords of scales per row), copied into LDS straight
// from memory, STAGES of them.  A stage is four steps of 64 k: lane half h holds
// blocks 4 h + q of the stage in step q, so that its scales are one dword, whose
// byte q the instruction picks.  Operands are read one step ahead of the products.
// The one barrier per stage stands before its last step's products: there every
// wave has read the whole stage, so the copy of the stage STAGES further can
// start, and the next stage has arrived.
//
// Bound: the weights' bytes for a few rows (32 x 14336 x 4096 8.2 us as traced, 4.0
// TB/s); for many neither the matrix cores (34% busy at 512 x 128256 x 4096: 173 us as
// traced, 3.1 PFLOP/s) nor the address units (61%) but the latency of copies: with 256 x
// 256 one stage and a part of the next are under way while one is computed, and a third
// stage of 256 k does not fit LDS.  (Four stages of 128 k would: not tried.)
//
// In LDS a row's eight 16-byte chunks are permuted by (row / 2) % 8, so that the
// rows of an operand read lie in different banks.  Scales are copied for two stages
// at a time (an epoch), 16 bytes of a row by four lanes, half of the rows with every
// stage.  A copy keeps the address units busy for about 2.2 cycles per line of 128
// bytes that it touches (1 KB of whole lines 18 cycles; measured on resident data),
// so 4 bytes per row and copy cost as much as all the codes.  (Four stages at a
// time: no faster on large grids and slower on small ones, whose first stage waits
// for more copies: 64 x 4096 x 4096 7.5 us against 6.8.)
//
// Where K ends inside the last stage, copies past a row's end take its first
// codes and its last scales instead; src1's codes there are replaced by zeros and
// all scales by 1 in registers (in a set's last stage, or last two of KW = 2, whose
// second set may end a stage further).
//
// KW = 2: two such sets of waves share the workgroup, each with half of the stages
// and LDS of its own; the second one's sums are added through LDS at the end (small
// grids, where a split over workgroups would need a second launch to join it).
constexpr int kStageK = 256;

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, int KW>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N * KW, 1) void k_mx4_wide(
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ wsc, const uint8_t* __restrict__ a,
    const uint8_t* __restrict__ asc, int M, int N, int K, float* __restrict__ dst, int tiles_m,
    int tiles, int split, int kchunk) {
  constexpr int NW = WAVES_M * WAVES_N;
  constexpr int WTM = BM / WAVES_M, WTN = BN / WAVES_N;
  constexpr int TM = WTM / 32, TN = WTN / 32;
  constexpr int kRow = kStageK / 2;                            // 128 bytes
  constexpr int kA = BN * kRow, STAGE = kA + BM * kRow;
  // scales: buffers of [weight rows, src1 rows][16 bytes] behind the stages
  constexpr int kScales = STAGES * STAGE, SBUF = (BM + BN) * 16, NB = STAGES;
  constexpr int WL = BN / 8 / NW, AL = BM / 8 / NW;            // pieces of 8 rows, 1 KB, per wave
  constexpr int SP = (BM + BN) / 32;                           // pieces of 16 rows' scales in a half,
  constexpr int SL = (SP + NW - 1) / NW;                       // per wave (some copied twice, alike)
  constexpr int kCopies = WL + AL + SL;
  // A stage's pieces (the scales are the last one).  The largest tiles' go in two
  // parts, kPart of them after the barrier that frees their buffer, the others in the
  // next stage's first step: the address units work through all of them for longer
  // than a step takes, and waves that wait to hand them over issue no products
  // (512 x 128256 x 4096, tile 256 x 256: 183 us against 193; 512 x 14336 x 4096, tile
  // 256 x 128: 25.9 against 29.8).  Smaller tiles copy less and lose 1 to 8 % by it.
  constexpr int kPieces = WL + AL + 1, kPart = STAGES == 2 ? kPieces - 2 * (kPieces / 4) : kPieces;
  constexpr int kPartCopies = kPart < kPieces ? kPart : kCopies;
  constexpr std::integral_constant<int, 0> first{};
  constexpr std::integral_constant<int, kPart> part{};
  constexpr std::integral_constant<int, kPieces> whole_stage{};
  static_assert(STAGES >= 2 && STAGES <= 4 && (STAGES - 1) * kCopies < 64, "wait counts");
  static_assert(BN % (8 * NW) == 0 && BM % (8 * NW) == 0 && BM % 32 == 0 && BN % 32 == 0,
                "whole pieces");
  extern __shared__ __attribute__((aligned(16))) uint8_t shared[];
  constexpr int kSet = kScales + NB * SBUF;                    // LDS of a set of waves
  static_assert(KW == 1 || (KW == 2 && BM * BN * 4 <= kSet), "the second set's sums lie in the first one's LDS");

  const int tid = threadIdx.x, lane = tid & 63, wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave_id / NW, wave = wave_id % NW;
  const int wm = wave % WAVES_M, wn = wave / WAVES_M;
  uint8_t* const lds = shared + kw * kSet;
  const int h = lane >> 5, l32 = lane & 31;
  const int ng = (K + kGrp - 1) / kGrp, nst = (K + kStageK - 1) / kStageK;
  const int t = xcd_remap(blockIdx.x, tiles * split);
  const int z = t / tiles, tt = t - z * tiles;
  const int tm = tt % tiles_m, tn = tt / tiles_m;    // m fastest: same weight tile adjacent
  const int m0 = tm * BM, n0 = tn * BN;
  // this set's first stage and stages (the second set's last one may lie past `end`)
  const int last = min(z * kchunk + kchunk, nst), end = min(last * kStageK, K);
  const int s1 = (last - z * kchunk + KW - 1) / KW, st0 = z * kchunk + kw * s1;

  // this lane's part of each piece
  const uint8_t* const wbase = w + (int64_t)n0 * (K / 2);
  const uint8_t* const abase = a + (int64_t)m0 * (K / 2);
  uint32_t woff[WL], aoff[AL];
  int chunk[WL > AL ? WL : AL];
#pragma unroll
  for (int i = 0; i < WL; ++i) woff[i] = (uint32_t)min((i * NW + wave) * 8 + (lane >> 3), N - 1 - n0) * (uint32_t)(K / 2);
#pragma unroll
  for (int i = 0; i < AL; ++i) aoff[i] = (uint32_t)min((i * NW + wave) * 8 + (lane >> 3), M - 1 - m0) * (uint32_t)(K / 2);
#pragma unroll
  for (int i = 0; i < (WL > AL ? WL : AL); ++i)      // (row / 2) % 8 of row 8 (i NW + wave) + lane / 8
    chunk[i] = (lane & 7) ^ ((4 * ((i * NW + wave) & 1) + (lane >> 4)) & 7);
  const uint8_t* const wscale = wsc + (int64_t)n0 * 4 * ng;
  const uint8_t* const ascale = asc + (int64_t)m0 * 4 * ng;
  const uint32_t lds0 = lds_offset(lds);
  // this lane's row in each half's pieces (the second one as the bits that differ: a
  // choice between two arrays would be kept in scratch memory)
  uint32_t soff[SL], sdiff[SL];
  const auto scale_row = [&](int i, int half) {
    const int r = 16 * ((i * NW + wave) % SP + half * SP);
    const bool isw = r < BN;                         // BN % 16 == 0
    return (uint32_t)min((isw ? r : r - BN) + (lane >> 2), isw ? N - 1 - n0 : M - 1 - m0) * (uint32_t)ng;
  };
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    soff[i] = scale_row(i, 0);
    sdiff[i] = soff[i] ^ scale_row(i, 1);
  }
  // Half u % 2 of the rows' scales of epoch u / 2.  With one of them ahead of all, and
  // u = s + 1 beside the codes of stage s, an epoch is whole when its first stage is.
  // Buffers: half 0 of epoch e is copied at stage 2 e - STAGES - 1, after its barrier;
  // epoch e - STAGES was last read in stage 2 (e - STAGES), which lies before.
  const auto copy_scales = [&](int u) {
    const int epoch = u >> 1, half = u & 1;
    const uint32_t dword = (uint32_t)min(2 * st0 + 4 * epoch + (lane & 3), ng - 1);
    const uint32_t base = lds0 + kScales + (uint32_t)(epoch % NB) * SBUF;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int r = 16 * ((i * NW + wave) % SP + half * SP);
      copy4(base + 16 * r, r < BN ? wscale : ascale, 4 * ((soff[i] ^ (sdiff[i] & -(uint32_t)half)) + dword));
    }
  };
  // pieces from .. to - 1 of a stage: weights, src1, then a set of scales
  const auto copy_pieces = [&](auto from, auto to, int s, int buf) {
    const uint32_t base = lds0 + buf * STAGE;
    const int kb = (st0 + s) * kRow;                 // bytes
#pragma unroll
    for (int i = 0; i < WL + AL; ++i) {
      if (i < from || i >= to) continue;
      const int c = i < WL ? i : i - WL, at = kb + 16 * chunk[c];
      const uint32_t in = at < K / 2 ? at : 0;
      if (i < WL) copy16(base + (c * NW + wave) * 1024, wbase, woff[i < WL ? i : 0] + in);
      else copy16(base + kA + (c * NW + wave) * 1024, abase, aoff[i < WL ? 0 : c] + in);
    }
    if (from < kPieces && to == kPieces) copy_scales(s + 1);   // and 0 ahead of all
  };

  v16f acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int wrow = (wn * WTN + l32) * kRow, arow = kA + (wm * WTM + l32) * kRow;
  const int x8 = (l32 >> 1) & 7;
  uint4 wr[2][TN], ar[2][TM];
  const auto read = [&](const uint8_t* base, int q) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      ar[q % 2][i] = *reinterpret_cast<const uint4*>(base + arow + 32 * i * kRow + 16 * ((4 * h + q) ^ x8));
#pragma unroll
    for (int j = 0; j < TN; ++j)
      wr[q % 2][j] = *reinterpret_cast<const uint4*>(base + wrow + 32 * j * kRow + 16 * ((4 * h + q) ^ x8));
  };
  uint32_t ws[TN], as[TM];
  const auto read_scales = [&](int s) {
    const uint8_t* const p = lds + kScales + (s >> 1) % NB * SBUF + 8 * (s & 1) + 4 * h;
#pragma unroll
    for (int i = 0; i < TM; ++i)
      as[i] = *reinterpret_cast<const uint32_t*>(p + 16 * (BN + wm * WTM + 32 * i + l32));
#pragma unroll
    for (int j = 0; j < TN; ++j)
      ws[j] = *reinterpret_cast<const uint32_t*>(p + 16 * (wn * WTN + 32 * j + l32));
  };

  copy_scales(0);
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < s1) copy_pieces(first, whole_stage, s, s);
  if (STAGES - 1 < s1) copy_pieces(first, part, STAGES - 1, STAGES - 1);
  if (s1 >= STAGES) wait_copies<(STAGES - 2) * kCopies + kPartCopies>();   // s1 >= 1
  else wait_copies<0>();
  __builtin_amdgcn_s_barrier();
  read(lds, 0);
  read_scales(0);

  // One stage.  kLeft: stages left with this one (STAGES + 1: more than are in
  // LDS, so the one STAGES further is copied).  No branches in here: the compiler
  // would move the products behind them, past the wait.
  int buf = 0;
  const auto stage = [&](auto left, int s) {
    constexpr int kLeft = decltype(left)::value;
    const uint8_t* const base = lds + buf * STAGE;
    const int next = buf + 1 == STAGES ? 0 : buf + 1;
    const int inside = end - (st0 + s) * kStageK - kGrp * h;   // this half's k before `end`
    if constexpr (kLeft <= KW) {                     // bytes of blocks past `end`: scale 1
      const uint32_t keep = inside >= kGrp ? ~0u : inside <= 0 ? 0u : (1u << (inside / 4)) - 1;
#pragma unroll
      for (int i = 0; i < TM; ++i) as[i] = (as[i] & keep) | (0x7f7f7f7fu & ~keep);
#pragma unroll
      for (int j = 0; j < TN; ++j) ws[j] = (ws[j] & keep) | (0x7f7f7f7fu & ~keep);
    }
    const auto step = [&](auto qc) {
      constexpr int q = decltype(qc)::value;
      uint32_t asq[TM], wsq[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i) asq[i] = as[i];
#pragma unroll
      for (int j = 0; j < TN; ++j) wsq[j] = ws[j];
      if constexpr (q < 3) {
        read(base, q + 1);
        if constexpr (q == 0 && kLeft >= STAGES)
          copy_pieces(part, whole_stage, s + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
      } else if constexpr (kLeft > 1) {
        // the next stage is here and this wave's reads of this one are done
        wait_copies<(kLeft > STAGES ? STAGES - 2 : kLeft - 2) * kCopies>();
        __builtin_amdgcn_s_barrier();
        if constexpr (kLeft > STAGES) copy_pieces(first, part, s + STAGES, buf);
        read(lds + next * STAGE, 0);
        read_scales(s + 1);
      }
      __builtin_amdgcn_sched_barrier(0);             // the reads stay ahead of the products
      if constexpr (kLeft <= KW) {                   // blocks past `end`: zeros
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          uint4& v = ar[q % 2][i];
          v = make_uint4(32 * q < inside ? v.x : 0, 32 * q < inside ? v.y : 0, 32 * q < inside ? v.z : 0,
                         32 * q < inside ? v.w : 0);
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              operand(ar[q % 2][i]), operand(wr[q % 2][j]), acc[i][j], 4, 4, q, (int)asq[i], q, (int)wsq[j]);
      __builtin_amdgcn_sched_barrier(0);
    };
    step(std::integral_constant<int, 0>());
    step(std::integral_constant<int, 1>());
    step(std::integral_constant<int, 2>());
    step(std::integral_constant<int, 3>());
    buf = next;
  };
  int s = 0;
  for (; s + STAGES < s1; ++s) stage(std::integral_constant<int, STAGES + 1>(), s);
  if constexpr (STAGES >= 4)
    if (s + 4 == s1) stage(std::integral_constant<int, 4>(), s++);
  if constexpr (STAGES >= 3)
    if (s + 3 == s1) stage(std::integral_constant<int, 3>(), s++);
  if (s + 2 == s1) stage(std::integral_constant<int, 2>(), s++);
  stage(std::integral_constant<int, 1>(), s);

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) settle(acc[i][j]);
  if constexpr (KW == 2) {
    // the second set's sums, 16 bytes per lane: [tile][r / 4][lane]
    __syncthreads();                                 // all reads of the stages are done
    float4* const sums = reinterpret_cast<float4*>(shared) + wave * (TM * TN * 4 * 64) + lane;
    if (kw == 1) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sums[((i * TN + j) * 4 + r) * 64] = make_float4(acc[i][j][4 * r], acc[i][j][4 * r + 1],
                                                            acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]);
    }
    __syncthreads();
    if (kw == 1) return;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 v = sums[((i * TN + j) * 4 + r) * 64];
          acc[i][j][4 * r] += v.x; acc[i][j][4 * r + 1] += v.y;
          acc[i][j][4 * r + 2] += v.z; acc[i][j][4 * r + 3] += v.w;
        }
  }

  // lane: weight row of column l32, src1 rows 8 (r / 4) + 4 h + r % 4
  const int mm = m0 + wm * WTM, nn = n0 + wn * WTN;
  float* const out = dst + (int64_t)z * M * N + (int64_t)mm * N + nn;
  const int64_t lane_off = (int64_t)(4 * h) * N + l32;
  const bool whole = mm + WTM <= M && nn + WTN <= N;             // uniform
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = 32 * i + 8 * (r / 4) + r % 4;
        if (whole || (mm + m + 4 * h < M && nn + 32 * j + l32 < N))
          (out + (int64_t)m * N + 32 * j)[lane_off] = acc[i][j][r];
      }
}

template <int NT>
hipError_t skinny(const Mx4Plan& p, const uint8_t* w, const uint8_t* wsc, const uint8_t* a,
                  const uint8_t* asc, float* dst, int M, int N, int K, hipStream_t s) {
  if (M > 16 * NT) return hipErrorInvalidValue;       // the plan gives it no more rows
  hipLaunchKernelGGL((k_mx4_skinny<NT>), dim3((unsigned)p.grid_n), dim3(64 * p.waves), p.lds, s, w,
                     wsc, a, asc, M, N, K, dst);
  return hipGetLastError();
}

template <int ROUNDS>
hipError_t fused(const Mx4Plan& p, const float* x, const uint8_t* w, const uint8_t* wsc, float* dst,
                 int M, int N, int K, hipStream_t s) {
  hipLaunchKernelGGL((k_mx4_fused<ROUNDS>), dim3((unsigned)p.grid_n), dim3(512), p.lds, s, x, w, wsc,
                     dst, M, N, K, (N + 15) / 16);
  return hipGetLastError();
}

template <int BM, int BN, int WAVES_M, int WAVES_N, int STAGES, int KW = 1>
hipError_t wide(const Mx4Plan& p, const uint8_t* w, const uint8_t* wsc, const uint8_t* a,
                const uint8_t* asc, float* dst, int M, int N, int K, void* ws, hipStream_t s) {
  constexpr int kLds = KW * STAGES * (BN + BM) * (kStageK / 2 + 16);
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
  auto* const kern = k_mx4_wide<BM, BN, WAVES_M, WAVES_N, STAGES, KW>;
  if (kLds > 65536) {
    static std::atomic<uint64_t> raised{0};          // devices whose limit is set already
    const hipError_t e = raise_lds(reinterpret_cast<const void*>(kern), kLds, raised);
    if (e != hipSuccess) return e;
  }
  float* const out = p.split > 1 ? reinterpret_cast<float*>((uint8_t*)ws + p.off_part) : dst;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles_m * p.tiles_n * p.split)),
                     dim3(64 * WAVES_M * WAVES_N * KW), kLds, s, w, wsc, a, asc, M, N, K, out,
                     (int)p.tiles_m, (int)(p.tiles_m * p.tiles_n), p.split, (int)p.kchunk);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.split > 1) e = launch_join_slices(out, dst, (int64_t)M * N, p.split, s);
  return e;
}

}  // namespace

hipError_t launch_mx4_quantize(const float* x, uint8_t* codes, uint8_t* scales, int64_t nrows,
                               int64_t k, hipStream_t s) {
  const int64_t ng = (k + kGrp - 1) / kGrp, groups = nrows * ng, grid = (groups + 15) / 16;
  hipLaunchKernelGGL(k_mx4_quantize, dim3((unsigned)(grid < kMaxGridX ? grid : kMaxGridX)), dim3(256),
                     0, s, x, codes, reinterpret_cast<uint32_t*>(scales), (int)k, (int)ng, groups);
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, float* y, int64_t nrows,
                                 int64_t k, hipStream_t s) {
  const int64_t ng = (k + kGrp - 1) / kGrp, pieces = nrows * (k / 8), grid = (pieces + 255) / 256;
  hipLaunchKernelGGL(k_mx4_dequantize, dim3((unsigned)(grid < kMaxGridX ? grid : kMaxGridX)), dim3(256),
                     0, s, codes, scales, y, (int)k, (int)ng, pieces);
  return hipGetLastError();
}

hipError_t launch_mx4_product(const Mx4Plan& p, const uint8_t* w, const uint8_t* wsc, const float* x,
                              const uint8_t* a, const uint8_t* asc, float* dst, int M, int N, int K,
                              void* ws, hipStream_t s) {
  if (p.kind == MX4_FUSED) {
    if (p.nt == 1) return fused<1>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 2) return fused<2>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 4) return fused<4>(p, x, w, wsc, dst, M, N, K, s);
    if (p.nt == 8) return fused<8>(p, x, w, wsc, dst, M, N, K, s);
    return hipErrorInvalidValue;
  }
  if (x) {                                            // INIT
    uint8_t* const codes = (uint8_t*)ws + p.off_a;
    uint8_t* const scales = (uint8_t*)ws + p.off_as;
    const hipError_t e = launch_mx4_quantize(x, codes, scales, M, K, s);
    if (e != hipSuccess) return e;
    a = codes;
    asc = scales;
  }
  if (p.kind == MX4_SKINNY) {
    if (p.nt == 1) return skinny<1>(p, w, wsc, a, asc, dst, M, N, K, s);
    if (p.nt == 2) return skinny<2>(p, w, wsc, a, asc, dst, M, N, K, s);
    return hipErrorInvalidValue;
  }
  if (p.bm == 32 && p.bn == 32) return wide<32, 32, 1, 1, 4, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 32 && p.bn == 64) return wide<32, 64, 1, 2, 4, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 64 && p.bn == 64) return wide<64, 64, 2, 2, 3>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 64 && p.bn == 128) return wide<64, 128, 2, 4, 3>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 128 && p.bn == 128) return wide<128, 128, 4, 2, 3>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 256 && p.bn == 128) return wide<256, 128, 4, 2, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  if (p.bm == 256 && p.bn == 256) return wide<256, 256, 2, 4, 2>(p, w, wsc, a, asc, dst, M, N, K, ws, s);
  return hipErrorInvalidValue;
}

}  // namespace qsg
