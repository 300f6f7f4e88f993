// A mixture-of-experts layer for a few tokens, for gfx950:
//
//   l[t][e] = x[t] . router[e];  p[t] = softmax(l[t]);  the top_k experts of
//   each token (ties: the lower index), w = p, or p / (sum of the chosen p);
//   h = silu(gate_e x[t]) * (up_e x[t]);  dst[t] = sum over the chosen of
//   w * down_e h.
//
// Launches on one stream: the router's logits (and x in split form); the
// selection, unless it is small enough for every workgroup of the next
// launch to make it for itself; gate, up and h; down and the weighted sum
// (and the join of its slices where it is cut in several).  The layer is
// bound by the chosen experts' weights, each read once, so everything else
// is arranged around that stream:
//
// * Products run on v_mfma_f32_16x16x32_f16, weights decoded to binary16 in
//   registers (Q4_0 codes - 8, e4m3 codes and binary16 are all exact in it)
//   as operand B, tokens as the 16 rows of operand A.  One MFMA covers one
//   block of 32 k.
// * Activations stay fp32 in effect: each row's block of 32 values is scaled
//   by a power of two that puts its largest magnitude in [2^14, 2^15) and
//   split as hi + lo, two binary16 numbers (22 significant bits; below 2^-28
//   of the block's largest value bits are lost, far under fp32 rounding of
//   the sums).  Two MFMAs per block; the matrix cores are idle otherwise.
//   Rounding them to 8 bits, as the quantized products do, would save
//   nothing here: the activations' bytes are few.
// * A block's result C[m][n] enters the fp32 sum as C * (dw * s), dw the
//   weights' scale and s the activations' block scale (times w in the down
//   product).  Token m of a pass of up to 16 sits in row 4 (m % 4) + m / 4, so
//   that a lane's four result registers are tokens g, 4 + g, 8 + g, 12 + g and
//   a pass of n tokens scales and adds ceil(n / 4) of them only: this vector
//   work per block, not the decode, grows with the rows in use.
// * x and h are kept in split form in the workspace, in operand order: per
//   row and block 128 bytes, [lane group g][hi 16 bytes | lo 16 bytes], and
//   one scale (a row's scales padded with zeros to a multiple of 4), so that
//   a lane's operand is two 16-byte loads and four blocks' scales are one.
// * Work moves in units of 4 blocks (128 k); a wave holds one unit while the
//   next one's loads are in flight.
#include "device.h"
#include "kernels.h"
#include "../../include/mm.h"

namespace qsg {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

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

// Maximum over each half wave (32 lanes), in every lane of it.
__device__ __forceinline__ float half_wave_max(float v) {
  v = fmaxf(v, dpp_f<0xB1>(v));
  v = fmaxf(v, dpp_f<0x4E>(v));
  v = fmaxf(v, dpp_f<0x141>(v));
  v = fmaxf(v, dpp_f<0x140>(v));
  return fmaxf(v, __shfl_xor(v, 16, 64));
}

// ---------------------------------------------------------------- router

// Logits in fp64 (the products of two fp32 values are exact there): the
// order of close logits decides which experts run, so it must not depend on
// the summation order.  One workgroup per expert and TT tokens; the
// workgroups past E split x, 32 blocks of 32 values of the TT tokens each.
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
    const int nb = D / 32, nbp = (nb + 3) & ~3, c = tid & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = ((int)blockIdx.x - E) * 32 + (tid >> 5) + 8 * i;   // per half wave
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int t = t0 + j;
        if (t >= T || b >= nbp) continue;
        float s = 0.0f;
        if (b < nb) {
          const float v = x[(int64_t)t * D + 32 * b + c];
          s = split_store<TY>(xp + ((int64_t)t * nb + b) * 128, c, v, half_wave_max(fabsf(v)));
        }
        if (c == 0) xs[(int64_t)t * nbp + b] = s;
      }
    }
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
// expert e's matrix of N rows of K; load(): issues a unit's loads;
// operand(j): block j as binary16, row lane % 16, in lane group order;
// scale(j): its dw.
template <int TY>
struct Tile;

template <>
struct Tile<MM_TYPE_Q4_0R> {
  const uint8_t* base;
  uint4 c;
  uint2 d;
  __device__ __forceinline__ void bind(const uint8_t* w, const float*, int64_t e, int N, int K,
                                       int row0, int lane) {
    const int64_t phases = (K + 255) / 256;
    base = w + (e * (N / 16) + row0 / 16) * phases * kQ4RChunk + 16 * lane;
  }
  // a unit is half of a repacked chunk of 8 blocks
  __device__ __forceinline__ void load(int u, int, int lane) {
    const uint8_t* p = base + (int64_t)(u >> 1) * kQ4RChunk;
    c = *reinterpret_cast<const uint4*>(p + 1024 * (u & 1));
    d = *reinterpret_cast<const uint2*>(p - 16 * lane + 2048 + 16 * (lane & 15) + 8 * (u & 1));
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

template <>
struct Tile<MM_TYPE_F8> {
  const uint8_t* base;
  const float* sc;
  uint2 c[4];
  float d;
  __device__ __forceinline__ void bind(const uint8_t* w, const float* s, int64_t e, int N, int K,
                                       int row0, int lane) {
    const int64_t nkb = (K + 127) / 128;
    base = w + (e * N + row0 + (lane & 15)) * K + 8 * (lane >> 4);
    sc = s + (e * ((N + 127) / 128) + row0 / 128) * nkb;
  }
  __device__ __forceinline__ void load(int u, int nb, int) {
    d = sc[u];
#pragma unroll
    for (int j = 0; j < 4; ++j)                      // past K: the last block, with s = 0
      c[j] = *reinterpret_cast<const uint2*>(base + 32 * (int64_t)min(4 * u + j, nb - 1));
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

template <>
struct Tile<MM_TYPE_F16> {
  const uint8_t* base;
  uint4 c[4];
  __device__ __forceinline__ void bind(const uint8_t* w, const float*, int64_t e, int N, int K,
                                       int row0, int lane) {
    base = w + 2 * ((e * N + row0 + (lane & 15)) * K + 8 * (lane >> 4));
  }
  __device__ __forceinline__ void load(int u, int nb, int) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = *reinterpret_cast<const uint4*>(base + 64 * (int64_t)min(4 * u + j, nb - 1));
  }
  __device__ __forceinline__ v8h operand(int j) const { return __builtin_bit_cast(v8h, c[j]); }
  __device__ __forceinline__ float scale(int) const { return 1.0f; }
};

// A unit's activations: this lane's operand pieces of its row (the token
// 4 (i16 % 4) + i16 / 4 of the pass; zeros where there is none) and the
// scales of the NR tokens 4 r + g whose results it holds.
template <int NR>
struct Acts {
  uint4 hi[4], lo[4];
  float4 s[NR];
  __device__ __forceinline__ void load(const uint8_t* row, bool live, const float* const (&sc)[NR],
                                       int u, int nb) {
#pragma unroll
    for (int j = 0; j < 4; ++j) hi[j] = lo[j] = make_uint4(0, 0, 0, 0);
    if (live) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* const p = row + 128 * (int64_t)min(4 * u + j, nb - 1);
        hi[j] = *reinterpret_cast<const uint4*>(p);
        lo[j] = *reinterpret_cast<const uint4*>(p + 16);
      }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = *reinterpret_cast<const float4*>(sc[r] + 4 * u);
  }
  __device__ __forceinline__ float scale(int r, int j) const {
    return j == 0 ? s[r].x : j == 1 ? s[r].y : j == 2 ? s[r].z : s[r].w;
  }
};

// acc[i][r] += the unit's contribution of RT weight tiles to token 4 r + g;
// p: a factor per token.
template <int TY, int NR, int RT>
__device__ __forceinline__ void unit_product(const Acts<NR>& x, const Tile<TY> (&w)[RT],
                                             const float (&p)[NR], float (&acc)[RT][NR]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const v8h hi = __builtin_bit_cast(v8h, x.hi[j]), lo = __builtin_bit_cast(v8h, x.lo[j]);
    float s[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) s[r] = x.scale(r, j) * p[r];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const v8h wv = w[i].operand(j);
      const float dw = w[i].scale(j);
      const v4f z = {0.f, 0.f, 0.f, 0.f};
      v4f c = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, wv, z, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, wv, c, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < NR; ++r) acc[i][r] = fmaf(c[r], dw * s[r], acc[i][r]);
    }
  }
}

// ---------------------------------------------------------------- gate, up, h

constexpr int kUpWaves = 8;

// kTwo: the next unit's loads are issued before the current one's product
// (two units in registers); the other form leaves that to the other waves of
// the SIMD.  K units wave, wave + W, ... of four tiles (32 rows of gate, the same of up)
// for one pass of up to 4 NR tokens; the partial sums go to
// part[wave][tile][token][16].
template <int TY, int NR, bool kTwo>
__device__ __forceinline__ void up_pass(const MoeArgs& a, int e, int row0, const int* list, int n,
                                        float* part, int lane, int wave) {
  const int g = lane >> 4, i16 = lane & 15;
  const int nb = a.D / 32, nbp = (nb + 3) & ~3, units = nbp / 4;
  const int mine = 4 * (i16 & 3) + (i16 >> 2);
  const bool live = mine < n;
  const uint8_t* const row = a.xp + (int64_t)(live ? list[mine] / a.top_k : 0) * nb * 128 + 32 * g;
  const float* sc[NR];
  float one[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    sc[r] = a.xs + (int64_t)(list[min(4 * r + g, n - 1)] / a.top_k) * nbp;
    one[r] = 1.0f;
  }
  float acc[4][NR];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = 0.0f;
  Tile<TY> w0[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w0[i].bind(i < 2 ? a.gate : a.up, i < 2 ? a.gate_scale : a.up_scale, e, a.F, a.D,
               row0 + 16 * (i & 1), lane);
  const auto load = [&](Tile<TY> (&w)[4], Acts<NR>& x, int u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i].load(u, nb, lane);
    x.load(row, live, sc, u, nb);
  };
  int u = wave;
  Acts<NR> x0;
  if constexpr (!kTwo) {
    for (; u < units; u += kUpWaves) {
      load(w0, x0, u);
      unit_product<TY, NR, 4>(x0, w0, one, acc);
    }
  } else {
    Tile<TY> w1[4];
    Acts<NR> x1;
#pragma unroll
    for (int i = 0; i < 4; ++i) w1[i] = w0[i];
    if (u < units) load(w0, x0, u);
    for (; u < units; u += 2 * kUpWaves) {
      const bool more = u + kUpWaves < units;
      if (more) load(w1, x1, u + kUpWaves);
      unit_product<TY, NR, 4>(x0, w0, one, acc);
      if (!more) break;
      if (u + 2 * kUpWaves < units) load(w0, x0, u + 2 * kUpWaves);
      unit_product<TY, NR, 4>(x1, w1, one, acc);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) part[((wave * 4 + i) * 16 + 4 * r + g) * 16 + i16] = acc[i][r];
}

// One workgroup: 32 rows of gate and the same rows of up of the blockIdx.y-th
// expert in use, over its tokens in passes of 16.  Eight waves split K; their
// partial tiles are added in LDS in wave order, then h = silu(g) u, split per
// block of 32 rows.  a.fold: every workgroup ranks the logits itself (a launch less), and one
// writes ids and weights for the next launch.
template <int TY, bool kFew>
__global__ __launch_bounds__(64 * kUpWaves, kFew || TY != MM_TYPE_Q4_0R ? 2 : 4) void k_moe_up(MoeArgs a) {
  constexpr int W = kUpWaves;
  __shared__ __attribute__((aligned(16))) float part[W * 4 * 256];
  __shared__ uint16_t sids[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ uint32_t bits[kMoeMaxExperts / 32];
  __shared__ uint32_t nans[kMoeMaxTokens / 32];
  __shared__ int list[kMoeMaxTokens];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int k = a.top_k, E = a.E, assigned = a.T * k;
  if (a.fold) {
    double* const l = reinterpret_cast<double*>(part);
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
    if (tid == 0) list[0] = blockIdx.y;
    __syncthreads();
  } else {
    if (tid < kMoeMaxExperts / 32) bits[tid] = 0;
    __syncthreads();
    for (int i = tid; i < assigned; i += 64 * W) atomicOr(&bits[sids[i] >> 5], 1u << (sids[i] & 31));
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
  const int nfb = a.F / 32, nfp = (nfb + 3) & ~3;

  const int rg = blockIdx.x;
  for (int m0 = 0; m0 < n; m0 += 16) {
    const int rows = min(n - m0, 16);
    if constexpr (kFew) {
      up_pass<TY, 1, TY != MM_TYPE_F16>(a, e, 32 * rg, list + m0, rows, part, lane, wave);
    } else {
      if (rows <= 4) up_pass<TY, 1, false>(a, e, 32 * rg, list + m0, rows, part, lane, wave);
      else if (rows <= 8) up_pass<TY, 2, false>(a, e, 32 * rg, list + m0, rows, part, lane, wave);
      else up_pass<TY, 4, false>(a, e, 32 * rg, list + m0, rows, part, lane, wave);
    }
    __syncthreads();
    const int m = tid >> 5, c = tid & 31;          // 16 tokens x 32 rows
    if (m < rows) {
      const float* const p = part + (c >> 4) * 256 + m * 16 + (c & 15);
      float gs = p[0], us = p[512];
#pragma unroll
      for (int v = 1; v < W; ++v) {
        gs += p[v * 1024];
        us += p[v * 1024 + 512];
      }
      const float h = gs / (1.0f + expf(-gs)) * us;
      const float amax = half_wave_max(fabsf(h));
      const int64_t at = list[m0 + m];
      const float s = split_store<TY>(a.hp + (at * nfb + rg) * 128, c, h, amax);
      if (c == 0) a.hs[at * nfp + rg] = s;
      // the last block's workgroup also writes the row's padding scales
      if (rg == nfb - 1 && c > 0 && rg + c < nfp) a.hs[at * nfp + rg + c] = 0.0f;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- down

// A job is one expert with up to 16 of the tokens that use it.
struct Jobs {
  int e[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];
  uint16_t first[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];   // in order[]
  uint16_t rows[kMoeMaxExperts + kMoeMaxTokens * kMoeMaxTopK / 16];
  uint16_t order[kMoeMaxTokens * kMoeMaxTopK];       // assignments, grouped by expert
  int cnt[kMoeMaxExperts], at[kMoeMaxExperts], job0[kMoeMaxExperts];
  int count;
};

// Groups the assignments by expert.  Within an expert the order is that of
// the atomics, which no result depends on: a token's contributions are added
// expert by expert, wherever in a job's rows it sits.
__device__ __forceinline__ void make_jobs(Jobs& js, const int* ids, int T, int assigned, int E,
                                          int lane, int wave) {
  const int tid = threadIdx.x, nt = blockDim.x;
  if (T == 1) {                                      // every assignment is a job
    if (tid < assigned) {
      js.e[tid] = ids[tid];
      js.first[tid] = js.order[tid] = (uint16_t)tid;
      js.rows[tid] = 1;
    }
    if (tid == 0) js.count = assigned;
    __syncthreads();
    return;
  }
  for (int e = tid; e < E; e += nt) js.cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < assigned; i += nt) atomicAdd(&js.cnt[ids[i]], 1);
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
        js.job0[b + lane] = jobs + sj - j;
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
      js.e[js.job0[e] + j] = e;
      js.first[js.job0[e] + j] = (uint16_t)(first + 16 * j);
      js.rows[js.job0[e] + j] = (uint16_t)min(c - 16 * j, 16);
    }
  }
  __syncthreads();
  for (int i = tid; i < assigned; i += nt) js.order[atomicAdd(&js.at[ids[i]], 1)] = (uint16_t)i;
  __syncthreads();
}

// Units u0 <= u < u1 of one job: acc of RT tiles over the job's tokens, added
// to the wave's sums[token][16 RT].
template <int TY, int NR, int RT>
__device__ __forceinline__ void down_job(const MoeArgs& a, int e, int row0, const uint16_t* order,
                                         int n, int u0, int u1, float* sums, int lane) {
  const int g = lane >> 4, i16 = lane & 15;
  const int nb = a.F / 32, nbp = (nb + 3) & ~3;
  const int mine = 4 * (i16 & 3) + (i16 >> 2);
  const bool live = mine < n;
  const uint8_t* const row = a.hp + (int64_t)(live ? order[mine] : 0) * nb * 128 + 32 * g;
  const float* sc[NR];
  float p[NR];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int at = order[min(4 * r + g, n - 1)];
    sc[r] = a.hs + (int64_t)at * nbp;
    p[r] = a.weights[at];
  }
  float acc[RT][NR];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int r = 0; r < NR; ++r) acc[i][r] = 0.0f;
  Tile<TY> w0[RT], w1[RT];
  Acts<NR> x0, x1;
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    w0[i].bind(a.down, a.down_scale, e, a.D, a.F, row0 + 16 * i, lane);
    w1[i] = w0[i];
  }
  const auto load = [&](Tile<TY> (&w)[RT], Acts<NR>& x, int u) {
#pragma unroll
    for (int i = 0; i < RT; ++i) w[i].load(u, nb, lane);
    x.load(row, live, sc, u, nb);
  };
  load(w0, x0, u0);
  for (int u = u0; u < u1; u += 2) {
    const bool more = u + 1 < u1;
    if (more) load(w1, x1, u + 1);
    unit_product<TY, NR, RT>(x0, w0, p, acc);
    if (!more) break;
    if (u + 2 < u1) load(w0, x0, u + 2);
    unit_product<TY, NR, RT>(x1, w1, p, acc);
  }
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (4 * r + g < n) {
      float* const s = sums + (order[4 * r + g] / a.top_k) * 16 * RT + i16;
#pragma unroll
      for (int i = 0; i < RT; ++i) s[16 * i] += acc[i][r];
    }
  }
}

// One workgroup: 16 RT rows of dst for all tokens, summed over slice
// blockIdx.y of the (job, unit) sequence; each wave takes one run of it and
// adds up per token in LDS, and the waves' sums are added in wave order.
template <int TY, int RT, int W, bool kFew>
__global__ __launch_bounds__(64 * W) void k_moe_down(MoeArgs a, float* __restrict__ out) {
  __shared__ Jobs js;
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [W][T][16 RT]
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
    if (kFew || n <= 4) down_job<TY, 1, RT>(a, e, row0, order, n, u0, u1, s, lane);
    else if (n <= 8) down_job<TY, 2, RT>(a, e, row0, order, n, u0, u1, s, lane);
    else down_job<TY, 4, RT>(a, e, row0, order, n, u0, u1, s, lane);
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
  const int lds = W * a.T * 16 * RT * 4;
  auto* const kern = k_moe_down<TY, RT, W, kFew>;
  static std::atomic<uint64_t> raised{0};            // devices whose limit is set already
  const hipError_t e = raise_lds(reinterpret_cast<const void*>(kern), kMoeMaxSums, raised);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(a.D / (16 * RT), p.slices), dim3(64 * W), lds, s, a, out);
  return hipGetLastError();
}

template <int TY>
hipError_t run(const MoePlan& p, const MoeArgs& a, float* part, hipStream_t s) {
  const int splits = (a.D / 32 + 31) / 32;
  if (a.T == 1)
    hipLaunchKernelGGL((k_moe_router<TY, 1>), dim3(a.E + splits, 1), dim3(256), 0, s, a.x, a.router, a.logits, a.xp, a.xs, a.T, a.D, a.E);
  else
    hipLaunchKernelGGL((k_moe_router<TY, 4>), dim3(a.E + splits, (a.T + 3) / 4), dim3(256), 0, s, a.x, a.router, a.logits, a.xp, a.xs, a.T, a.D, a.E);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!a.fold) {
    hipLaunchKernelGGL(k_moe_select, dim3(a.T), dim3(512), 0, s, a.logits, a.ids, a.weights, a.E, a.top_k, a.norm);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int assigned = a.T * a.top_k;
  const dim3 grid(a.F / 32 + (a.fold ? 1 : 0), assigned < a.E ? assigned : a.E);
  const bool few = a.T <= kMoeFewTokens;
  if (few) hipLaunchKernelGGL((k_moe_up<TY, true>), grid, dim3(64 * kUpWaves), 0, s, a);
  else hipLaunchKernelGGL((k_moe_up<TY, false>), grid, dim3(64 * kUpWaves), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* const out = p.slices > 1 ? part : a.dst;
  if (few) e = down<TY, 1, 16, true>(p, a, out, s);
  else if (p.rt == 4) e = down<TY, 4, 8, false>(p, a, out, s);
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
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qsg
