// A mixture-of-experts layer for a few tokens, for gfx950:
//
//   l[t][e] = x[t] . router[e];  p[t] = softmax(l[t]);  the top_k experts of
//   each token (ties: the lower index), w = p, or p / (sum of the chosen p);
//   h = silu(gate_e x[t]) * (up_e x[t]);  dst[t] = sum over the chosen of
//   w * down_e h.
//
// The choice of experts and their weights may be inputs instead (k_moe_take).
//
// Launches on one stream: the router's logits (and x in split form); the
// selection, unless it is small enough for every workgroup of the next
// launch to make it for itself; gate, up and h; down and the weighted sum
// (and the join of its slices where it is cut in several).  The layer is
// bound by the chosen experts' weights, each read once, so everything else
// is arranged around that stream:
//
// * Products run on v_mfma_f32_16x16x32_f16, weights decoded to binary16 in
//   registers (Q4_0 codes - 8, e4m3 and e2m1 codes and binary16 are all exact in it)
//   as operand B, tokens as the 16 rows of operand A.  One MFMA covers one
//   block of 32 k.
// * Activations stay fp32 in effect: each row's block of 32 values is scaled
//   by a power of two that puts its largest magnitude in [2^14, 2^15) and
//   split as hi + lo, two binary16 numbers: off by at most 2^-22 of the value
//   down to 2^-17 of the block's largest, by 2^-39 of the largest below that
//   (half of binary16's smallest step; far under the fp32 rounding of a sum
//   that the largest enters).  Two MFMAs per block; the matrix cores are idle
//   otherwise.
//   Rounding them to 8 bits, as the quantized products do, would save
//   nothing here: the activations' bytes are few.
// * A block's result C[m][n] enters the fp32 sum as (C * dw) * s, dw the
//   weights' scale and s the activations' block scale; the down product's w
//   multiplies the sum over a run of blocks.  In this order no factor falls
//   below fp32's normal range before the sum itself does: dw * s would (h of
//   1e-33 and e4m3 weights: s is 2^-126).  Nor does C * dw overflow for dw up to 2^99
//   (e4m3: |C| <= 32 * 448 * 2^15 < 2^28.9), 2^105 (e2m1: 32 * 6 * 2^15 < 2^22.6).
//   Token m of a pass of up to 16 sits in row 4 (m % 4) + m / 4, so
//   that a lane's four result registers are tokens g, 4 + g, 8 + g, 12 + g and
//   a pass of n tokens scales and adds ceil(n / 4) of them only: this vector
//   work per block, not the decode, grows with the rows in use.
// * x and h are kept in split form in the workspace, in operand order: per
//   row and block 128 bytes, [lane group g][hi 16 bytes | lo 16 bytes], and
//   one scale (a row's scales padded with zeros to a multiple of 4), so that
//   a lane's operand is two 16-byte loads and four blocks' scales are one.
// * Work moves in units of 4 blocks (128 k) per wave: while one unit is
//   computed from registers, the next one's weights are on their way to
//   registers and its activations (512 consecutive bytes per row; e4m3
//   weights too) to the wave's own piece of LDS, from which a lane takes its
//   operand.  (Weights two units ahead in gate / up, Q4_0R, measured no faster:
//   layer, 1 / 16 / 64 tokens, 8 experts of 4096 x 14336, 65 / 204 / 371 us against
//   61 / 200 / 364, and its wait had to count loads that the compiler issues; in
//   down nothing changed.)  Loading operands straight from memory costs one
//   16-byte access per lane, since neighbouring lanes belong to different rows:
//   the address units were 67% busy and the gate / up launch at 2.9 TB/s (32
//   tokens, 8 experts of 4096 x 14336).
#include <type_traits>

#include "device.h"
#include "kernels.h"
#include "../../include/mm.h"

namespace qsg {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v2ua __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- activations

// Where element c of a block lies among the 128 bytes of its split form (hi;
// lo is 16 bytes further).  Lane group g's eight elements: for Q4_0R the
// nibbles of code bytes 4g .. 4g+3 in the order its decode yields them
// (bytes 0, 2, 1, 3, low nibbles then high), else 8g .. 8g+7.
template <int TY>
__device__ __forceinline__ int split_pos(int c) {
  if constexpr (TY == MM_TYPE_Q4_0R) {
    const int b = c & 3;
    const int p = 4 * (c >> 4) + (b == 1 ? 2 : b == 2 ? 1 : b);
    return ((c & 15) >> 2) * 32 + 2 * p;
  } else {
    return (c >> 3) * 32 + 2 * (c & 7);
  }
}

// Writes one value of a block whose largest magnitude is amax; returns the
// block's scale.  An infinity or NaN gives NaN.
template <int TY>
__device__ __forceinline__ float split_store(uint8_t* blk, int c, float v, float amax) {
  int shift = 15 - __builtin_amdgcn_frexp_expf(amax);
  shift = shift > 126 ? 126 : shift;
  const float xs = __builtin_amdgcn_ldexpf(v, shift);
  const _Float16 hi = (_Float16)xs;
  const _Float16 lo = (_Float16)(xs - (float)hi);
  uint8_t* const p = blk + split_pos<TY>(c);
  *reinterpret_cast<_Float16*>(p) = hi;
  *reinterpret_cast<_Float16*>(p + 16) = lo;
  return __builtin_amdgcn_ldexpf(1.0f, -shift);
}

// Four values, 4 q .. 4 q + 3, of a block at once.
template <int TY>
__device__ __forceinline__ float split_store4(uint8_t* blk, int q, float4 v, float amax) {
  int shift = 15 - __builtin_amdgcn_frexp_expf(amax);
  shift = shift > 126 ? 126 : shift;
  const float x[4] = {v.x, TY == MM_TYPE_Q4_0R ? v.z : v.y, TY == MM_TYPE_Q4_0R ? v.y : v.z, v.w};
  union { _Float16 h[4]; uint2 u; } hi, lo;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float xs = __builtin_amdgcn_ldexpf(x[i], shift);
    hi.h[i] = (_Float16)xs;
    lo.h[i] = (_Float16)(xs - (float)hi.h[i]);
  }
  uint8_t* const p = blk + split_pos<TY>(4 * q);
  *reinterpret_cast<uint2*>(p) = hi.u;
  *reinterpret_cast<uint2*>(p + 16) = lo.u;
  return __builtin_amdgcn_ldexpf(1.0f, -shift);
}

// Maximum over each half wave (32 lanes), in every lane of it.
__device__ __forceinline__ float half_wave_max(float v) {
  v = fmaxf(v, dpp_f<0xB1>(v));
  v = fmaxf(v, dpp_f<0x4E>(v));
  v = fmaxf(v, dpp_f<0x141>(v));
  v = fmaxf(v, dpp_f<0x140>(v));
  return fmaxf(v, __shfl_xor(v, 16, 64));
}

// Splits 8 blocks of 32 values, 8 part .. 8 part + 7, of TT tokens from t0: a half
// wave (of 256 threads) each.
template <int TY, int TT>
__device__ __forceinline__ void split_rows(const float* __restrict__ x, uint8_t* __restrict__ xp,
                                           float* __restrict__ xs, int T, int D, int t0, int part) {
  const int tid = threadIdx.x;
  const int nb = D / 32, nbp = (nb + 3) & ~3, c = tid & 31;
  const int b = part * 8 + (tid >> 5);
  if (b >= nbp) return;
  float v[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j)
    v[j] = b < nb ? x[(int64_t)min(t0 + j, T - 1) * D + 32 * b + c] : 0.0f;
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = t0 + j;
    if (t >= T) break;
    float s = 0.0f;
    if (b < nb) s = split_store<TY>(xp + ((int64_t)t * nb + b) * 128, c, v[j], half_wave_max(fabsf(v[j])));
    if (c == 0) xs[(int64_t)t * nbp + b] = s;
  }
}

// A routing that is given: x in split form, and (one workgroup) the choice made
// fit for the launches behind it: what names no expert becomes -1, an expert that
// a token names several times is kept once, with the sum of its weights (so that
// no expert has more rows than there are tokens, and no two rows of one job add
// to the same sum).
//
// Slot i's expert, or -1, and its weight.
__device__ __forceinline__ int taken(const int* ids, const float* weights, int i, int k, int E, float& w) {
  const int first = i / k * k, id = ids[i];
  w = weights[i];
  if (id < 0 || id >= E) return -1;
  for (int j = first; j < i; ++j)
    if (ids[j] == id) return -1;
  for (int j = i + 1; j < first + k; ++j)
    if (ids[j] == id) w += weights[j];
  return id;
}

template <int TY, int TT>
__global__ __launch_bounds__(256) void k_moe_take(MoeArgs a, int splits) {
  if ((int)blockIdx.x < splits) {
    split_rows<TY, TT>(a.x, a.xp, a.xs, a.T, a.D, blockIdx.y * TT, blockIdx.x);
    return;
  }
  if (blockIdx.y) return;
  for (int i = threadIdx.x; i < a.T * a.top_k; i += 256) {
    float w;
    a.ids[i] = taken(a.given_ids, a.given_weights, i, a.top_k, a.E, w);
    a.weights[i] = w;
  }
}

// ---------------------------------------------------------------- router

// Logits in fp64 (the products of two fp32 values are exact there): the
// order of close logits decides which experts run, so it must not depend on
// the summation order.  One workgroup per expert and TT tokens; the
// workgroups past E split x, 8 blocks of 32 values of the TT tokens each.
template <int TY, int TT>
__global__ __launch_bounds__(256) void k_moe_router(const float* __restrict__ x,
                                                    const float* __restrict__ router,
                                                    double* __restrict__ logits,
                                                    uint8_t* __restrict__ xp,
                                                    float* __restrict__ xs, int T, int D, int E) {
  __shared__ double part[4][TT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t0 = blockIdx.y * TT;
  if ((int)blockIdx.x >= E) {
    split_rows<TY, TT>(x, xp, xs, T, D, t0, (int)blockIdx.x - E);
    return;
  }
  const int e = blockIdx.x;
  double acc[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) acc[i] = 0.0;
  const float* const r = router + (int64_t)e * D;
#pragma unroll 2
  for (int k = 4 * tid; k < D; k += 1024) {
    const float4 w = *reinterpret_cast<const float4*>(r + k);
    float4 v[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i)
      v[i] = *reinterpret_cast<const float4*>(x + (int64_t)min(t0 + i, T - 1) * D + k);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      acc[i] = fma((double)w.x, (double)v[i].x, acc[i]);
      acc[i] = fma((double)w.y, (double)v[i].y, acc[i]);
      acc[i] = fma((double)w.z, (double)v[i].z, acc[i]);
      acc[i] = fma((double)w.w, (double)v[i].w, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[i] += __shfl_xor(acc[i], o, 64);
    if (lane == 0) part[wave][i] = acc[i];
  }
  __syncthreads();
  if (tid < TT && t0 + tid < T)
    logits[(int64_t)(t0 + tid) * E + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// An expert's rank among a token's logits is the number of experts ahead of
// it (larger, or equal with a lower index; a NaN counts as the lowest), so
// every rank below top_k names its slot, with no passes over the top_k.
// Eight adjacent lanes share one expert's count.
__device__ __forceinline__ int rank_of(const double* l, int e, int E, int lane) {
  const double v = l[e];
  int rank = 0;
#pragma unroll 4
  for (int o = lane & 7; o < E; o += 8) {
    const double w = l[o];
    rank += (w > v || (w == v && o < e)) ? 1 : 0;
  }
  rank += dpp_i<0xB1>(rank);                         // quad_perm [1,0,3,2]
  rank += dpp_i<0x4E>(rank);                         // quad_perm [2,3,0,1]
  return rank + dpp_i<0x141>(rank);                  // row_half_mirror
}

// exp(l - best): the fp32 part of the fp64 difference, the rest to first order.
__device__ __forceinline__ float exp_diff(double l, double best) {
  const double d = l - best;
  const float hi = (float)d;
  const float p = expf(hi);
  return hi > -__builtin_inff() ? fmaf(p, (float)(d - (double)hi), p) : p;
}

// Probabilities of one token's chosen experts, by one thread.
__device__ __forceinline__ void token_weights(const double* l, const uint16_t* chosen, int E, int top_k,
                                              bool norm, bool nan_seen, float* out) {
  const double best = l[chosen[0]];
  float sum = 0.0f;
  if (norm) {
    for (int j = 0; j < top_k; ++j) sum += exp_diff(l[chosen[j]], best);
  } else {
    for (int e = 0; e < E; ++e) sum += exp_diff(l[e], best);
  }
  for (int j = 0; j < top_k; ++j) out[j] = nan_seen ? __builtin_nanf("") : exp_diff(l[chosen[j]], best) / sum;
}

// Selection as a launch of its own: one workgroup per token.
__global__ __launch_bounds__(512) void k_moe_select(const double* __restrict__ logits,
                                                    int* __restrict__ ids,
                                                    float* __restrict__ weights, int E, int top_k,
                                                    int norm) {
  __shared__ double l[kMoeMaxExperts];
  __shared__ uint16_t chosen[kMoeMaxTopK];
  __shared__ int nan_seen;
  const int t = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) nan_seen = 0;
  __syncthreads();
  if (tid < E) {
    const double v = logits[(int64_t)t * E + tid];
    if (v != v) nan_seen = 1;
    l[tid] = v == v ? v : -__builtin_inf();
  }
  __syncthreads();
  for (int i = tid; i < 8 * ((E + 63) & ~63); i += 512) {     // whole waves: E padded
    const int e = i >> 3, rank = rank_of(l, min(e, E - 1), E, tid);
    if ((i & 7) == 0 && e < E && rank < top_k) {
      chosen[rank] = (uint16_t)e;
      ids[t * top_k + rank] = e;
    }
  }
  __syncthreads();
  if (tid == 0) token_weights(l, chosen, E, top_k, norm, nan_seen, weights + t * top_k);
}

// ---------------------------------------------------------------- weights

// One 16-row tile of weights, a unit of 4 blocks of 32 k at a time.  bind():
// expert e's matrix of N rows of K; load(): issues a unit's loads; fetch():
// takes what load() sent through LDS (kLds bytes at lds), or tells the
// compiler that its loads have arrived; operand(j): block j as binary16, row
// lane % 16, in lane group order; scale(j): its dw.
template <int TY>
struct Tile;

template <>
struct Tile<MM_TYPE_Q4_0R> {
  static constexpr int kLds = 0;
  static constexpr int kPair = 1;
  const uint8_t* base;
  v4u c;                         // whole vectors, so that they stay in the registers that
  v2u d;                         // the loads fill
  __device__ __forceinline__ void bind(const uint8_t* w, const void*, int64_t e, int N, int K,
                                       int row0, int lane) {
    const int64_t phases = (K + 255) / 256;
    base = w + (e * (N / 16) + row0 / 16) * phases * kQ4RChunk + 16 * lane;
  }
  // a unit is half of a repacked chunk of 8 blocks
  __device__ __forceinline__ void fetch(const uint8_t*, int) {
    asm volatile("" : "+v"(c), "+v"(d));
  }
  __device__ __forceinline__ void load(int u, int, int lane, uint32_t, bool) {
    const uint8_t* p = base + (int64_t)(u >> 1) * kQ4RChunk;
    c = *reinterpret_cast<const v4u*>(p + 1024 * (u & 1));
    d = *reinterpret_cast<const v2u*>(p - 16 * lane + 2048 + 16 * (lane & 15) + 8 * (u & 1));
  }
  __device__ __forceinline__ v8h operand(int j) const {
    const uint32_t w = j == 0 ? c.x : j == 1 ? c.y : j == 2 ? c.z : c.w;
    const uint32_t w8 = w >> 8;
    // 0x6400 | q is the binary16 1024 + q, 0x6400 | 16 q is 1024 + 16 q
    const v2h m1032 = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    const v2h m72 = {(_Float16)-72.0f, (_Float16)-72.0f};
    const v2h r16 = {(_Float16)0.0625f, (_Float16)0.0625f};
    const v2h a = __builtin_bit_cast(v2h, (w & 0x000F000Fu) | 0x64006400u) + m1032;
    const v2h b = __builtin_bit_cast(v2h, (w8 & 0x000F000Fu) | 0x64006400u) + m1032;
    const v2h e = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (w & 0x00F000F0u) | 0x64006400u), r16, m72);
    const v2h f = __builtin_elementwise_fma(__builtin_bit_cast(v2h, (w8 & 0x00F000F0u) | 0x64006400u), r16, m72);
    return (v8h){a[0], a[1], b[0], b[1], e[0], e[1], f[0], f[1]};
  }
  __device__ __forceinline__ float scale(int j) const {
    const uint32_t w = j < 2 ? d.x : d.y;
    return f16_bits_to_f32((j & 1) ? w >> 16 : w);
  }
};

// e4m3 goes through LDS (16 rows of 128 codes, the 16-byte chunks of a row
// permuted by (row / 2) % 8): a lane's operand is 8 bytes of its row.
template <>
struct Tile<MM_TYPE_F8> {
  static constexpr int kLds = 2048;
  static constexpr int kPair = 1;
  const uint8_t* base;           // uniform
  const float* sc;
  uint32_t off[2];               // the rows this lane copies
  int chunk, K;
  uint2 c[4];
  float d, dnext;
  __device__ __forceinline__ void bind(const uint8_t* w, const void* s, int64_t e, int N, int k,
                                       int row0, int lane) {
    const int64_t nkb = (k + 127) / 128;
    K = k;
    base = w + (e * N + row0) * k;
    sc = (const float*)s + (e * ((N + 127) / 128) + row0 / 128) * nkb;
    // piece q: rows 8 q + lane / 8, position lane % 8; (row / 2) % 8
#pragma unroll
    for (int q = 0; q < 2; ++q) off[q] = (uint32_t)(8 * q + (lane >> 3)) * (uint32_t)k;
    chunk = lane & 7;
  }
  __device__ __forceinline__ void load(int u, int, int lane, uint32_t lds, bool) {
    dnext = sc[u];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = 128 * u + 16 * (chunk ^ ((4 * q + (lane >> 4)) & 7));
      copy16(lds + 1024 * q, base, off[q] + (uint32_t)min(k, K - 16));   // past K: meets s = 0
    }
  }
  __device__ __forceinline__ void fetch(const uint8_t* lds, int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = *reinterpret_cast<const uint2*>(lds + 128 * r + 16 * ((2 * j + (g >> 1)) ^ ((r >> 1) & 7)) + 8 * (g & 1));
    d = dnext;
  }
  __device__ __forceinline__ v8h operand(int j) const {
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j].x, 1.0f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j].x, 1.0f, true);
    const v2h e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j].y, 1.0f, false);
    const v2h f = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[j].y, 1.0f, true);
    return (v8h){a[0], a[1], b[0], b[1], e[0], e[1], f[0], f[1]};
  }
  __device__ __forceinline__ float scale(int) const { return d; }
};

// MXFP4 goes through LDS too, kPair units of neighbours at a time: with two, 16 rows
// of whole 128-byte lines (a copy of 64 bytes per row takes the address units as
// long): the even unit's load copies both, or the first one's where a wave begins
// with the odd one (fresh).  The 16-byte blocks of a row are permuted by its index,
// so that a column of blocks lies in all banks; a lane's operand is 4 bytes of its
// row's block.  A unit's four scale bytes are one dword of the row.  (Loads straight
// into registers, transposed there: 272 us against 261 with one unit and 237 with
// two, 32 tokens on 8 experts of 4096 x 14336.)
//
// One unit at a time for few tokens, whose workgroups then share a CU (gate / up of 4
// tokens, 16 experts of 2048 x 2048: 19 us against 22).
constexpr int kMxfp4Few = 100;
template <int kUnits>
struct MxTile {
  static constexpr int kLds = 1024 * kUnits;
  static constexpr int kPair = kUnits;
  const uint8_t* base;           // uniform
  const uint32_t* sc;
  uint32_t off[kUnits];          // the rows this lane copies
  int last, nb, unit;
  uint32_t c[4], dw[4];
  std::conditional_t<kUnits == 2, v2u, uint32_t> dnext;
  // where block b of row r lies among the row's 4 kUnits
  static __device__ __forceinline__ int place(int b, int r) {
    return kUnits == 2 ? b ^ ((r >> 1) & 7) : b ^ ((r >> 2) & 3);
  }
  __device__ __forceinline__ void bind(const uint8_t* w, const void* s, int64_t e, int N, int k,
                                       int row0, int lane) {
    nb = k / 32;
    last = k / 2 - 16;
    base = w + (e * N + row0) * (k / 2);
    sc = (const uint32_t*)s + (e * N + row0 + (lane & 15)) * ((k + 127) / 128);
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
      off[q] = (uint32_t)((16 * q + lane / 4) / kUnits) * (uint32_t)(k / 2);
  }
  __device__ __forceinline__ void load(int u, int, int lane, uint32_t lds, bool fresh) {
    unit = u;
    const int u0 = u & -kUnits;
    if (u != u0 && !fresh) return;                   // uniform
    if constexpr (kUnits == 2) {
      if (4 * (u0 + 1) < nb) dnext = *reinterpret_cast<const v2ua*>(sc + u0);
      else dnext.x = sc[u0];
    } else {
      dnext = sc[u0];
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      // blocks past K: the last one again
      const int at = 64 * u0 + 16 * place(lane & (4 * kUnits - 1), (16 * q + lane / 4) / kUnits);
      copy16(lds + 1024 * q, base, off[q] + (uint32_t)min(at, last));
    }
  }
  __device__ __forceinline__ void fetch(const uint8_t* lds, int lane) {
    const int r = lane & 15, g = lane >> 4, half = unit & (kUnits - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = *reinterpret_cast<const uint32_t*>(lds + 64 * kUnits * r + 16 * place(4 * half + j, r) + 4 * g);
    asm volatile("" : "+v"(dnext));
    // blocks past K: scale 1 (they meet activations of scale 0)
    const int left = nb - 4 * unit;
    const uint32_t keep = left >= 4 ? ~0u : (1u << (8 * left)) - 1;
    uint32_t d;
    if constexpr (kUnits == 2) d = half ? dnext.y : dnext.x;
    else d = dnext;
    d = (d & keep) | (0x7f7f7f7fu & ~keep);
    // 2^(byte - 127): the byte as an exponent, but for 0 (2^-127 is subnormal) and 255
    // (NaN), which take the fraction's top bit
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[j] = (j == 3 ? d >> 1 : d << (23 - 8 * j)) & 0x7f800000u;
    const uint32_t zero = (d - 0x01010101u) & ~d, ones = (~d - 0x01010101u) & d;
    if (__any(((zero | ones) & 0x80808080u) != 0)) { // rare
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!((dw[j] + 0x00800000u) & 0x7f000000u)) dw[j] |= 0x00400000u;
    }
  }
  __device__ __forceinline__ v8h operand(int j) const {
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[j], 1.0f, 0);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[j], 1.0f, 1);
    const v2h e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[j], 1.0f, 2);
    const v2h f = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c[j], 1.0f, 3);
    return (v8h){a[0], a[1], b[0], b[1], e[0], e[1], f[0], f[1]};
  }
  __device__ __forceinline__ float scale(int j) const { return __builtin_bit_cast(float, dw[j]); }
};
template <>
struct Tile<MM_TYPE_MXFP4> : MxTile<2> {};
template <>
struct Tile<kMxfp4Few> : MxTile<1> {};

template <>
struct Tile<MM_TYPE_F16> {
  static constexpr int kLds = 0;
  static constexpr int kPair = 1;
  const uint8_t* base;
  uint4 c[4];
  __device__ __forceinline__ void bind(const uint8_t* w, const void*, int64_t e, int N, int K,
                                       int row0, int lane) {
    base = w + 2 * ((e * N + row0 + (lane & 15)) * K + 8 * (lane >> 4));
  }
  __device__ __forceinline__ void fetch(const uint8_t*, int) {
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(c[j].x), "+v"(c[j].y), "+v"(c[j].z), "+v"(c[j].w));
  }
  __device__ __forceinline__ void load(int u, int nb, int, uint32_t, bool) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = *reinterpret_cast<const uint4*>(base + 64 * (int64_t)min(4 * u + j, nb - 1));
  }
  __device__ __forceinline__ v8h operand(int j) const { return __builtin_bit_cast(v8h, c[j]); }
  __device__ __forceinline__ float scale(int) const { return 1.0f; }
};

static_assert((uint64_t)kMoeMaxTokens * kMoeMaxTopK * 4 * kMoeMaxDim < 1ull << 32,
              "offsets into split h (4 bytes a value, a row per token and expert) fit 32 bits");

// The activations of a pass of up to 4 NR tokens, a unit at a time through
// the wave's LDS: [row][512 bytes], the 16-byte chunks of a row permuted by
// row % 16, then the rows' scales [row][4].  Rows past the pass repeat the
// last one, lanes of rows that are not copied read what is there: no result
// of theirs is kept.
template <int NR>
struct Acts {
  static constexpr int kLds = 4 * NR * 528;
  const uint8_t* base;           // uniform
  const float* sbase;
  uint32_t off[2 * NR], soff;    // the rows this lane copies
  int last;                      // last chunk of a row
  uint4 hi[4], lo[4];
  float4 s[NR];
  // row_of(m): the row of base that holds token m of the pass, m < n
  template <class F>
  __device__ __forceinline__ void bind(const uint8_t* split, const float* scales, int nb, int n,
                                       int lane, F row_of) {
    base = split;
    sbase = scales;
#pragma unroll
    for (int q = 0; q < 2 * NR; ++q)
      off[q] = (uint32_t)row_of(min(2 * q + (lane >> 5), n - 1)) * (uint32_t)(128 * nb);
    soff = (uint32_t)row_of(min(lane >> 2, n - 1)) * (uint32_t)((nb + 3) & ~3) + (lane & 3);
    last = 8 * nb - 1;
  }
  __device__ __forceinline__ void load(int u, int n, int lane, uint32_t lds) {
#pragma unroll
    for (int q = 0; q < 2 * NR; ++q) {
      if (2 * q < n) {                               // uniform
        const int chunk = (lane & 31) ^ ((2 * q + (lane >> 5)) & 15);
        copy16(lds + 1024 * q, base, off[q] + 16 * min(32 * u + chunk, last));
      }
    }
    if (lane < 16 * NR) copy4(lds + 2048 * NR, sbase, 4 * (soff + 4 * u));
  }
  __device__ __forceinline__ void fetch(const uint8_t* lds, int lane) {
    const int g = lane >> 4, row = 4 * (lane & 3) + ((lane & 15) >> 2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* const p = lds + 512 * (row & (4 * NR - 1));
      hi[j] = *reinterpret_cast<const uint4*>(p + 16 * ((8 * j + 2 * g) ^ (row & (4 * NR - 1))));
      lo[j] = *reinterpret_cast<const uint4*>(p + 16 * ((8 * j + 2 * g + 1) ^ (row & (4 * NR - 1))));
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = *reinterpret_cast<const float4*>(lds + 2048 * NR + 16 * (4 * r + g));
  }
  __device__ __forceinline__ float scale(int r, int j) const {
    return j == 0 ? s[r].x : j == 1 ? s[r].y : j == 2 ? s[r].z : s[r].w;
  }
};

// The same for a pass of up to 4 tokens whose workgroup holds all of split x in LDS:
// rows of held_pitch bytes (16 more than their blocks, so that four rows lie in
// different banks), then the rows' scales.
__host__ __device__ constexpr int held_pitch(int nbp) { return 128 * nbp + 16; }

struct ActsHeld {
  static constexpr int kLds = 0;
  const uint8_t *row, *srow;
  int unit;
  uint4 hi[4], lo[4];
  float4 s[1];
  template <class F>
  __device__ __forceinline__ void bind(const uint8_t* held, int T, int nbp, int n, int lane, F row_of) {
    const int g = lane >> 4;
    row = held + row_of(min((lane >> 2) & 3, n - 1)) * held_pitch(nbp) + 32 * g;
    srow = held + T * held_pitch(nbp) + row_of(min(g, n - 1)) * 4 * nbp;
  }
  __device__ __forceinline__ void load(int u, int, int, uint32_t) { unit = u; }
  __device__ __forceinline__ void fetch(const uint8_t*, int) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = *reinterpret_cast<const uint4*>(row + 512 * unit + 128 * j);
      lo[j] = *reinterpret_cast<const uint4*>(row + 512 * unit + 128 * j + 16);
    }
    s[0] = *reinterpret_cast<const float4*>(srow + 16 * unit);
  }
  __device__ __forceinline__ float scale(int, int j) const {
    return j == 0 ? s[0].x : j == 1 ? s[0].y : j == 2 ? s[0].z : s[0].w;
  }
};

// acc[i][r] += the unit's contribution of RT weight tiles to token 4 r + g.
template <int TY, int NR, int RT, class X>
__device__ __forceinline__ void unit_product(const X& x, const Tile<TY> (&w)[RT],
                                             float (&acc)[RT][NR]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const v8h hi = __builtin_bit_cast(v8h, x.hi[j]), lo = __builtin_bit_cast(v8h, x.lo[j]);
    float s[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = x.scale(r, j);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const v8h wv = w[i].operand(j);
      const float dw = w[i].scale(j);
      const v4f z = {0.f, 0.f, 0.f, 0.f};
      v4f c = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, wv, z, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, wv, c, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[i][r] = fmaf(c[r] * dw, s[r], acc[i][r]);
    }
    __builtin_amdgcn_sched_barrier(0);               // one block's operands in registers at a time
  }
}

// Units u, u + 1, ... < end of RT tiles for one pass: acc += ...  lds: the
// wave's staging (activations, then the tiles').  The wait at the top finds
// exactly the current unit's loads under way; its LDS is free again once the
// operands are in registers.
template <int TY, int NR, int RT>
__device__ __forceinline__ void run_units(Acts<NR>& x, Tile<TY> (&w0)[RT], int u, int end, int n,
                                          int nb, float (&acc)[RT][NR], uint8_t* lds, int lane) {
  const uint32_t at = lds_offset(lds), tat = at + Acts<NR>::kLds;
  const auto issue = [&](Tile<TY> (&w)[RT], int v, bool fresh) {
    x.load(v, n, lane, at);
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i].load(v, nb, lane, tat + i * Tile<TY>::kLds, fresh);
  };
  const auto take = [&](Tile<TY> (&w)[RT]) {
    wait_copies<0>();
    x.fetch(lds, lane);
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i].fetch(lds + Acts<NR>::kLds + i * Tile<TY>::kLds, lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  if (u >= end) return;
  issue(w0, u, true);
  if constexpr (Tile<TY>::kLds > 0) {
    for (; u < end; ++u) {
      take(w0);
      if (u + 1 < end) issue(w0, u + 1, false);
      unit_product<TY, NR, RT>(x, w0, acc);
    }
  } else {
    Tile<TY> w1[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) w1[i] = w0[i];
    for (; u < end; u += 2) {
      take(w0);
      if (u + 1 < end) issue(w1, u + 1, false);
      unit_product<TY, NR, RT>(x, w0, acc);
      if (u + 1 >= end) break;
      take(w1);
      if (u + 2 < end) issue(w0, u + 2, false);
      unit_product<TY, NR, RT>(x, w1, acc);
    }
  }
}

// ---------------------------------------------------------------- gate, up, h

constexpr int kUpWaves = 8;

// Partial sums kept apart in the join: one per wave, or one per pair of waves
// (w, w + 4) where e4m3's staging leaves no room for eight.
template <int TY, bool kFew>
constexpr int up_parts() { return Tile<TY>::kLds > 0 && !kFew ? kUpWaves / 2 : kUpWaves; }

// Dynamic LDS of the gate / up kernel: the waves' staging, then their partial
// sums (before both, the logits where it makes the selection).
template <int TY, bool kFew, bool kHeld>
constexpr int up_lds() {
  return kUpWaves * ((kHeld ? 0 : Acts<kFew ? 1 : 4>::kLds) + 4 * Tile<TY>::kLds) +
         up_parts<TY, kFew>() * 4 * (kFew ? 4 : 16) * 64;
}

// One pass of up to 4 NR tokens over all K for the row groups rg0, rg0 + step,
// ...: the waves take units in turn, across the groups, so that a group's
// first loads are under way while the one before is joined.  The join: partial
// sums to part[wave][tile][token][16] (kRows tokens), added in wave order,
// h = silu(g) u, split per block of 32 rows.
// held: split x in LDS, where kHeld.
template <int TY, int NR, int kRows, bool kHeld>
__device__ __forceinline__ void up_pass(const MoeArgs& a, int e, int rg0, int step, const int* list, int n,
                                        uint8_t* lds, float* part, const uint8_t* held, int lane, int wave) {
  constexpr int W = kUpWaves, P = up_parts<TY, kRows == 4>();
  asm volatile("" : "+v"(lane));                     // keep a pass's addresses inside the pass
  const int g = lane >> 4, i16 = lane & 15;
  const int nb = a.D / 32, units = (nb + 3) / 4;
  const int nfb = a.F / 32, nfp = (nfb + 3) & ~3;
  static_assert(!kHeld || NR == 1, "four tokens");
  using X = std::conditional_t<kHeld, ActsHeld, Acts<NR>>;
  X x;
  const auto token = [&](int m) { return list[m] / a.top_k; };
  if constexpr (kHeld) x.bind(held, a.T, (nb + 3) & ~3, n, lane, token);
  else x.bind(a.xp, a.xs, nb, n, lane, token);
  float acc[4][NR];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = 0.0f;
  const uint32_t at = lds_offset(lds), tat = at + X::kLds;
  const auto issue_w = [&](Tile<TY> (&w)[4], int rg, int u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i].bind(i < 2 ? a.gate : a.up, i < 2 ? a.gate_scale : a.up_scale, e, a.F, a.D,
                32 * rg + 16 * (i & 1), lane);
      w[i].load(u, nb, lane, tat + i * Tile<TY>::kLds, false);   // begins with an even unit
    }
  };
  const auto fetch = [&](Tile<TY> (&w)[4]) {
    x.fetch(lds, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i].fetch(lds + X::kLds + i * Tile<TY>::kLds, lane);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  const auto join = [&](int rg) {
    const auto put = [&](bool add) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float* const q = part + ((wave % P * 4 + i) * kRows + 4 * r + g) * 16 + i16;
          *q = add ? *q + acc[i][r] : acc[i][r];
          acc[i][r] = 0.0f;
        }
    };
    if (wave < P) put(false);
    lds_barrier();
    if constexpr (P < W) {
      if (wave >= P) put(true);
      lds_barrier();
    }
    const int tid = 64 * wave + lane, m = tid >> 5, c = tid & 31;    // 16 tokens x 32 rows
    if (m < n) {
      const float* const p = part + ((c >> 4) * kRows + m) * 16 + (c & 15);
      float gs = p[0], us = p[32 * kRows];
#pragma unroll
      for (int v = 1; v < P; ++v) {
        gs += p[v * 64 * kRows];
        us += p[v * 64 * kRows + 32 * kRows];
      }
      const float h = gs / (1.0f + expf(-gs)) * us;
      const float amax = half_wave_max(fabsf(h));
      const int64_t to = list[m];
      const float s = split_store<TY>(a.hp + (to * nfb + rg) * 128, c, h, amax);
      if (c == 0) a.hs[to * nfp + rg] = s;
      // the last block's workgroup also writes the row's padding scales
      if (rg == nfb - 1 && c > 0 && rg + c < nfp) a.hs[to * nfp + rg + c] = 0.0f;
    }
    lds_barrier();                                   // the partial sums are read
  };
  // a wave's units: kPair neighbours, then W of those further
  constexpr int P2 = Tile<TY>::kPair;
  if (P2 * wave >= units) {                          // no units: only the joins
    for (int rg = rg0; rg < nfb; rg += step) join(rg);
    return;
  }
  // one unit of row group rg; the next one's loads; the join after the last
  int rg = rg0, u = P2 * wave;
  const auto issue = [&](Tile<TY> (&w)[4], int r, int v) {
    x.load(v, n, lane, at);
    issue_w(w, r, v);
  };
  const auto body = [&](Tile<TY> (&w)[4], Tile<TY> (&next)[4]) {
    wait_copies<0>();
    fetch(w);
    const int further = P2 == 2 && !(u & 1) ? u + 1 : u + P2 * (W - 1) + 1;
    const bool last = further >= units;
    const int nrg = last ? rg + step : rg, nu = last ? P2 * wave : further;
    if (nrg < nfb) issue(next, nrg, nu);
    unit_product<TY, NR, 4>(x, w, acc);
    if (last) join(rg);
    rg = nrg;
    u = nu;
  };
  Tile<TY> w0[4];
  issue(w0, rg, u);
  if constexpr (Tile<TY>::kLds > 0) {
    while (rg < nfb) body(w0, w0);
  } else {
    Tile<TY> w1[4];
    while (rg < nfb) {
      body(w0, w1);
      if (rg >= nfb) break;
      body(w1, w0);
    }
  }
}

// One workgroup: groups of 32 rows of gate and the same rows of up (four 16-row
// tiles that share the activations), every a.up_groups-th group of the
// blockIdx.y-th expert in use, over its tokens in passes of 16.  a.fold: every
// workgroup ranks the logits itself (a launch less), and one writes ids and
// weights for the next launch.  kHeld: the choice is given, and every workgroup
// makes it fit and splits x itself (a launch less, and no copies of x beside the
// weights').
template <int TY, bool kFew, bool kHeld>
__global__ __launch_bounds__(64 * kUpWaves, TY == kMxfp4Few ? 4 : 2) void k_moe_up(MoeArgs a) {
  static_assert(kFew || !kHeld, "few tokens");
  constexpr int W = kUpWaves, kRows = kFew ? 4 : 16;
  constexpr int kStage = (kHeld ? 0 : Acts<kFew ? 1 : 4>::kLds) + 4 * Tile<TY>::kLds;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint16_t sids[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ uint32_t bits[kMoeMaxExperts / 32];
  __shared__ uint32_t nans[kMoeMaxTokens / 32];
  __shared__ int list[kMoeMaxTokens];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k = a.top_k, E = a.E, assigned = a.T * k;
  uint8_t* const held = lds + up_lds<TY, kFew, kHeld>();
  if constexpr (kHeld) {
    const bool outputs = blockIdx.x == gridDim.x - 1;   // one more column of workgroups
    if (outputs && blockIdx.y) return;
    // four values per thread, eight threads per block of 32
    const int nb = a.D / 32, nbp = (nb + 3) & ~3, row = 8 * nbp;
    float* const hs = reinterpret_cast<float*>(held + a.T * held_pitch(nbp));
    int id = -1;
    if (wave == 0 && lane < assigned) id = a.given_ids[lane];        // assigned <= 64
    for (int i0 = tid; i0 < a.T * row && !outputs; i0 += 4 * 64 * W) {
      float4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + 64 * W * q, t = held_token(i, row, a.T), at = i - t * row;
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < a.T && at < 8 * nb) v[q] = *reinterpret_cast<const float4*>(a.x + t * a.D + 4 * at);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = i0 + 64 * W * q, t = held_token(i, row, a.T), at = i - t * row;
        if (64 * W * q + (i0 - tid) >= a.T * row) break;             // uniform
        float amax = fmaxf(fmaxf(fabsf(v[q].x), fabsf(v[q].y)), fmaxf(fabsf(v[q].z), fabsf(v[q].w)));
        amax = fmaxf(amax, dpp_f<0xB1>(amax));
        amax = fmaxf(amax, dpp_f<0x4E>(amax));
        amax = fmaxf(amax, dpp_f<0x141>(amax));      // eight lanes
        if (t >= a.T) continue;                      // eight lanes alike: row % 8 == 0
        const float s = split_store4<TY>(held + t * held_pitch(nbp) + 128 * (at >> 3), at & 7, v[q], amax);
        if ((at & 7) == 0) hs[t * nbp + (at >> 3)] = at < 8 * nb ? s : 0.0f;
      }
    }
    if (wave == 0) {
      if (id >= E) id = -1;
      const float w = outputs && lane < assigned ? a.given_weights[lane] : 0.0f;
      const int slot = lane % k;
      float sum = w;
      bool again = false;
      for (int j = 1; j < k; ++j) {                  // the slots before and behind of the same token
        const int before = __shfl_up(id, j, 64);
        again |= j <= slot && before == id;
        if (!outputs) continue;                      // uniform
        const int behind = __shfl_down(id, j, 64);
        const float more = __shfl_down(w, j, 64);
        if (slot + j < k && behind == id) sum += more;
      }
      if (lane < assigned) {
        const int kept = again ? -1 : max(id, -1);
        sids[lane] = (uint16_t)kept;                 // -1: no expert's
        if (outputs) {
          a.ids[lane] = kept;
          a.weights[lane] = sum;
        }
      }
    }
    if (outputs) return;
    __syncthreads();
  } else if (a.fold) {
    double* const l = reinterpret_cast<double*>(lds);
    if (tid < kMoeMaxTokens / 32) nans[tid] = 0;
    __syncthreads();
    for (int i = tid; i < a.T * E; i += 64 * W) {
      const double v = a.logits[i];
      if (v != v) atomicOr(&nans[i / E >> 5], 1u << (i / E & 31));
      l[i] = v == v ? v : -__builtin_inf();
    }
    __syncthreads();
    for (int i = tid; i < (8 * a.T * E + 63) / 64 * 64; i += 64 * W) {   // whole waves
      const int j = min(i >> 3, a.T * E - 1), t = j / E;
      const int rank = rank_of(l + t * E, j - t * E, E, lane);
      if ((i & 7) == 0 && i >> 3 == j && rank < k) sids[t * k + rank] = (uint16_t)(j - t * E);
    }
    __syncthreads();
    if (blockIdx.x == gridDim.x - 1) {               // one more column of workgroups: the outputs
      if (blockIdx.y) return;
      for (int i = tid; i < assigned; i += 64 * W) a.ids[i] = sids[i];
      if (tid < a.T)
        token_weights(l + tid * E, sids + tid * k, E, k, a.norm, nans[tid >> 5] >> (tid & 31) & 1,
                      a.weights + tid * k);
      return;
    }
  } else {
    for (int i = tid; i < assigned; i += 64 * W) sids[i] = (uint16_t)a.ids[i];
    __syncthreads();
  }
  int e, n = 1;
  if (a.T == 1) {
    e = sids[blockIdx.y];
    if (e >= E) return;                              // a slot without an expert
    if (tid == 0) list[0] = blockIdx.y;
    __syncthreads();
  } else {
    if (tid < kMoeMaxExperts / 32) bits[tid] = 0;
    __syncthreads();
    for (int i = tid; i < assigned; i += 64 * W)
      if (sids[i] < E) atomicOr(&bits[sids[i] >> 5], 1u << (sids[i] & 31));
    __syncthreads();
    int left = blockIdx.y, word = 0;
    while (word < kMoeMaxExperts / 32 && left >= __popc(bits[word])) left -= __popc(bits[word++]);
    if (word == kMoeMaxExperts / 32) return;         // fewer experts in use than slots
    uint32_t v = bits[word];
    for (; left > 0; --left) v &= v - 1;
    e = 32 * word + __ffs((int)v) - 1;
    if (wave == 0) {
      int c = 0;
      for (int b = 0; b < assigned; b += 64) {
        const bool mine = b + lane < assigned && sids[b + lane] == e;
        const uint64_t vote = __ballot(mine);
        if (mine) list[c + __popcll(vote & ((1ull << lane) - 1))] = b + lane;
        c += __popcll(vote);
      }
      if (lane == 0) count = c;
    }
    __syncthreads();
    n = count;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  n = __builtin_amdgcn_readfirstlane(n);
  uint8_t* const stage = lds + wave * kStage;
  float* const part = reinterpret_cast<float*>(lds + W * kStage);
  __syncthreads();                                   // the logits, where they were here, are read
  for (int m0 = 0; m0 < n; m0 += 16) {
    const int rows = min(n - m0, 16), rg = blockIdx.x, step = a.up_groups;
    if constexpr (kFew) {
      up_pass<TY, 1, kRows, kHeld>(a, e, rg, step, list + m0, rows, stage, part, held, lane, wave);
    } else {
      if (rows <= 4) up_pass<TY, 1, kRows, kHeld>(a, e, rg, step, list + m0, rows, stage, part, held, lane, wave);
      else if (rows <= 8) up_pass<TY, 2, kRows, false>(a, e, rg, step, list + m0, rows, stage, part, held, lane, wave);
      else up_pass<TY, 4, kRows, false>(a, e, rg, step, list + m0, rows, stage, part, held, lane, wave);
    }
  }
}

// ---------------------------------------------------------------- down

// A job is one expert with up to 16 of the tokens that use it.
struct Jobs {
  uint16_t e[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];
  uint16_t first[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];   // in order[]
  uint16_t rows[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];
  uint16_t order[kMoeMaxTokens * kMoeMaxTopK];       // assignments, grouped by expert
  int cnt[kMoeMaxExperts], at[kMoeMaxExperts];
  uint16_t job0[kMoeMaxExperts];
  int count;
};

// Groups the assignments by expert (an id of -1: none), in ascending order within
// one (the order decides which job a token of a much used expert falls into, and with it how
// the waves cut its sum).
__device__ __forceinline__ void make_jobs(Jobs& js, const int* ids, int T, int assigned, int E,
                                          int lane, int wave) {
  const int tid = threadIdx.x, nt = blockDim.x;
  if (T == 1) {                                      // every assignment is a job
    if (wave == 0) {
      const int id = lane < assigned ? ids[lane] : -1;
      const uint64_t vote = __ballot(id >= 0);
      const int j = __popcll(vote & ((1ull << lane) - 1));
      if (id >= 0) {
        js.e[j] = (uint16_t)id;
        js.first[j] = (uint16_t)j;
        js.order[j] = (uint16_t)lane;
        js.rows[j] = 1;
      }
      if (lane == 0) js.count = __popcll(vote);
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < E; e += nt) js.cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < assigned; i += nt) {
    const int id = ids[i];
    if (id >= 0) atomicAdd(&js.cnt[id], 1);
  }
  __syncthreads();
  if (wave == 0) {
    int base = 0, jobs = 0;
    for (int b = 0; b < E; b += 64) {
      const int c = b + lane < E ? js.cnt[b + lane] : 0, j = (c + 15) >> 4;
      int sc = c, sj = j;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int vc = __shfl_up(sc, o, 64), vj = __shfl_up(sj, o, 64);
        if (lane >= o) { sc += vc; sj += vj; }
      }
      if (b + lane < E) {
        js.at[b + lane] = base + sc - c;
        js.job0[b + lane] = (uint16_t)(jobs + sj - j);
      }
      base += __shfl(sc, 63, 64);
      jobs += __shfl(sj, 63, 64);
    }
    if (lane == 0) js.count = jobs;
  }
  __syncthreads();
  for (int e = tid; e < E; e += nt) {
    const int c = js.cnt[e], first = js.at[e];
    for (int j = 0; 16 * j < c; ++j) {
      js.e[js.job0[e] + j] = (uint16_t)e;
      js.first[js.job0[e] + j] = (uint16_t)(first + 16 * j);
      js.rows[js.job0[e] + j] = (uint16_t)min(c - 16 * j, 16);
    }
  }
  __syncthreads();
  if (wave == 0) {
    // 64 at a time: the lanes of the same expert by one vote per bit of its index
    for (int b = 0; b < assigned; b += 64) {
      const int id = b + lane < assigned ? ids[b + lane] : -1;
      const bool in = id >= 0;
      const int e = in ? id : 0;
      uint64_t same = __ballot(in);
#pragma unroll
      for (int bit = 1; bit < kMoeMaxExperts; bit <<= 1) {
        const uint64_t v = __ballot((e & bit) != 0);
        same &= (e & bit) ? v : ~v;
      }
      if (in) {
        const int ahead = __popcll(same & ((1ull << lane) - 1)), at = js.at[e];
        js.order[at + ahead] = (uint16_t)(b + lane);
        if (ahead == 0) js.at[e] = at + __popcll(same);
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
}

// Units u0 <= u < u1 of one job: acc of RT tiles over the job's tokens, times
// their weights, added to the wave's sums[token][16 RT].
template <int TY, int NR, int RT>
__device__ __forceinline__ void down_job(const MoeArgs& a, int e, int row0, const uint16_t* order,
                                         int n, int u0, int u1, float* sums, uint8_t* lds, int lane) {
  asm volatile("" : "+v"(lane));                     // keep a job's addresses inside the job
  const int g = lane >> 4, i16 = lane & 15;
  const int nb = a.F / 32;
  Acts<NR> x;
  x.bind(a.hp, a.hs, nb, n, lane, [&](int m) { return (int)order[m]; });
  float acc[RT][NR], p[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) p[r] = a.weights[order[min(4 * r + g, n - 1)]];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = 0.0f;
  Tile<TY> w[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) w[i].bind(a.down, a.down_scale, e, a.D, a.F, row0 + 16 * i, lane);
  run_units<TY, NR, RT>(x, w, u0, u1, n, nb, acc, lds, lane);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (4 * r + g < n) {
      float* const s = sums + (order[4 * r + g] / a.top_k) * 16 * RT + i16;
#pragma unroll
      for (int i = 0; i < RT; ++i) s[16 * i] = fmaf(acc[i][r], p[r], s[16 * i]);
    }
  }
}

// One workgroup: 16 RT rows of dst for all tokens, summed over slice
// blockIdx.y of the (job, unit) sequence; each wave takes one run of it and
// adds up per token in LDS, and the waves' sums are added in wave order.
template <int TY, int RT, int W, bool kFew>
__global__ __launch_bounds__(64 * W) void k_moe_down(MoeArgs a, float* __restrict__ out) {
  __shared__ Jobs js;
  constexpr int kStage = Acts<kFew ? 1 : 4>::kLds + RT * Tile<TY>::kLds;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // the waves' staging, then
  float* const sums = reinterpret_cast<float*>(lds + W * kStage); // [W][T][16 RT]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int per = a.T * 16 * RT;
  for (int i = tid; i < W * per; i += 64 * W) sums[i] = 0.0f;
  make_jobs(js, a.ids, a.T, a.T * a.top_k, a.E, lane, wave);
  const int row0 = blockIdx.x * 16 * RT;
  const int units = (a.F / 32 + 3) / 4;
  const int total = js.count * units, parts = W * gridDim.y, part = blockIdx.y * W + wave;
  int at = (int)((int64_t)total * part / parts);
  const int end = (int)((int64_t)total * (part + 1) / parts);
  while (at < end) {
    const int j = at / units, u0 = at - j * units, u1 = min(units, u0 + end - at);
    const int e = __builtin_amdgcn_readfirstlane(js.e[j]);
    const int n = __builtin_amdgcn_readfirstlane((int)js.rows[j]);
    const uint16_t* const order = js.order + js.first[j];
    float* const s = sums + wave * per;
    if constexpr (kFew) down_job<TY, 1, RT>(a, e, row0, order, n, u0, u1, s, lds + wave * kStage, lane);
    else if (n <= 4) down_job<TY, 1, RT>(a, e, row0, order, n, u0, u1, s, lds + wave * kStage, lane);
    else if (n <= 8) down_job<TY, 2, RT>(a, e, row0, order, n, u0, u1, s, lds + wave * kStage, lane);
    else down_job<TY, 4, RT>(a, e, row0, order, n, u0, u1, s, lds + wave * kStage, lane);
    at += u1 - u0;
  }
  __syncthreads();
  out += (int64_t)blockIdx.y * a.T * a.D;
  for (int i = tid; i < per; i += 64 * W) {
    float s = sums[i];
#pragma unroll
    for (int v = 1; v < W; ++v) s += sums[v * per + i];
    out[(int64_t)(i / (16 * RT)) * a.D + row0 + i % (16 * RT)] = s;
  }
}

template <int TY, int RT, int W, bool kFew>
hipError_t down(const MoePlan& p, const MoeArgs& a, float* out, hipStream_t s) {
  const int lds = W * (Acts<kFew ? 1 : 4>::kLds + RT * Tile<TY>::kLds + a.T * 16 * RT * 4);
  if (lds > kMoeMaxLds) return hipErrorInvalidValue;  // the plan keeps T RT small enough
  auto* const kern = k_moe_down<TY, RT, W, kFew>;
  static std::atomic<uint64_t> raised{0};            // devices whose limit is set already
  const hipError_t e = raise_lds(reinterpret_cast<const void*>(kern), kMoeMaxLds, raised);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(a.D / (16 * RT), p.slices), dim3(64 * W), lds, s, a, out);
  return hipGetLastError();
}

template <int TY, bool kFew, bool kHeld>
hipError_t up(dim3 grid, const MoeArgs& a, hipStream_t s) {
  const int nbp = (a.D / 32 + 3) & ~3;
  if (kHeld && a.T * nbp > kMoeHeldBlocks) return hipErrorInvalidValue;   // the plan's rule
  const int lds = up_lds<TY, kFew, kHeld>() + (kHeld ? a.T * (held_pitch(nbp) + 4 * nbp) : 0);
  constexpr int most = up_lds<TY, kFew, kHeld>() +
                       (kHeld ? kMoeHeldBlocks * 132 + kMoeFewTokens * held_pitch(0) : 0);
  static_assert(most <= kMoeMaxLds, "LDS");
  auto* const kern = k_moe_up<TY, kFew, kHeld>;
  if (most > 65536) {
    static std::atomic<uint64_t> raised{0};
    const hipError_t e = raise_lds(reinterpret_cast<const void*>(kern), most, raised);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, grid, dim3(64 * kUpWaves), lds, s, a);
  return hipGetLastError();
}

template <int TY>
hipError_t run(const MoePlan& p, const MoeArgs& a, float* part, hipStream_t s) {
  const int splits = (((a.D / 32 + 3) & ~3) + 7) / 8;
  if (p.held) {
    // no launch: see k_moe_up
  } else if (a.given_ids) {
    if (a.T == 1) hipLaunchKernelGGL((k_moe_take<TY, 1>), dim3(splits + 1, 1), dim3(256), 0, s, a, splits);
    else hipLaunchKernelGGL((k_moe_take<TY, 4>), dim3(splits + 1, (a.T + 3) / 4), dim3(256), 0, s, a, splits);
  } else if (a.T == 1)
    hipLaunchKernelGGL((k_moe_router<TY, 1>), dim3(a.E + splits, 1), dim3(256), 0, s, a.x, a.router, a.logits, a.xp, a.xs, a.T, a.D, a.E);
  else
    hipLaunchKernelGGL((k_moe_router<TY, 4>), dim3(a.E + splits, (a.T + 3) / 4), dim3(256), 0, s, a.x, a.router, a.logits, a.xp, a.xs, a.T, a.D, a.E);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!a.fold && !a.given_ids) {
    hipLaunchKernelGGL(k_moe_select, dim3(a.T), dim3(512), 0, s, a.logits, a.ids, a.weights, a.E, a.top_k, a.norm);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int assigned = a.T * a.top_k;
  const dim3 grid(a.up_groups + (a.fold || p.held ? 1 : 0), assigned < a.E ? assigned : a.E);
  const bool few = a.T <= kMoeFewTokens;
  constexpr int kFewType = TY == MM_TYPE_MXFP4 ? kMxfp4Few : TY;
  e = p.held ? up<kFewType, true, true>(grid, a, s)
      : few  ? up<kFewType, true, false>(grid, a, s)
             : up<TY, false, false>(grid, a, s);
  if (e != hipSuccess) return e;
  float* const out = p.slices > 1 ? part : a.dst;
  if (few) e = down<kFewType, 1, 16, true>(p, a, out, s);
  else if (Tile<TY>::kLds == 0 && p.rt == 4) e = down<TY, Tile<TY>::kLds ? 1 : 4, 8, false>(p, a, out, s);
  else if (p.rt == 2 && TY == MM_TYPE_MXFP4 && a.T > kMoeMxPairTokens) e = down<kFewType, 2, 8, false>(p, a, out, s);
  else if (p.rt == 2) e = down<TY, 2, 8, false>(p, a, out, s);
  else e = down<TY, 1, 8, false>(p, a, out, s);
  if (e == hipSuccess && p.slices > 1) e = launch_join_slices(part, a.dst, (int64_t)a.T * a.D, p.slices, s);
  return e;
}

}  // namespace

hipError_t launch_moe(int type, const MoePlan& p, const MoeArgs& a, float* part, hipStream_t s) {
  switch (type) {
    case MM_TYPE_Q4_0R: return run<MM_TYPE_Q4_0R>(p, a, part, s);
    case MM_TYPE_F8: return run<MM_TYPE_F8>(p, a, part, s);
    case MM_TYPE_F16: return run<MM_TYPE_F16>(p, a, part, s);
    case MM_TYPE_MXFP4: return run<MM_TYPE_MXFP4>(p, a, part, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qsg
