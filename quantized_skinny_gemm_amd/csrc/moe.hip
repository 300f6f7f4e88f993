// A mixture-of-experts layer for a few tokens, for gfx950:
//
//   l[t][e] = x[t] . router[e];  p[t] = softmax(l[t]);  the top_k experts of
//   each token (ties: the lower index), w = p, or p / (sum of the chosen p);
//   h = silu(gate_e x[t]) * (up_e x[t]);  dst[t] = sum over the chosen of
//   w * down_e h.
//
// Four launches on one stream: logits; selection; gate, up and h; down and
// the weighted sum.  The layer is bound by the chosen experts' weights, each
// read once, so everything else is arranged around that stream:
//
// * Products run on v_mfma_f32_16x16x32_f16, weights decoded to binary16 in
//   registers (Q4_0 codes - 8, e4m3 codes and binary16 are all exact in it),
//   tokens as the 16 rows of operand A.  One MFMA covers one block of 32 k.
// * Activations stay fp32 in effect: each row's block of 32 values is scaled
//   by a power of two that puts its largest magnitude in [2^14, 2^15) and
//   split as hi + lo, two binary16 numbers (22 significant bits; below 2^-28
//   of the block's largest value bits are lost, far under fp32 rounding of
//   the sums).  Two MFMAs per block; the matrix cores are idle otherwise.
//   Rounding them to 8 bits, as the quantized products do, would save
//   nothing here: the activations' bytes are few.
// * A block's result C[m][n] enters the fp32 sum as C * (dw * s), dw the
//   weights' scale and s the activations' block scale (times w in the down
//   product).
// * x and h are kept in that form in the workspace, in operand order: per
//   row and block 128 bytes, [lane group g][hi 16 bytes | lo 16 bytes], and
//   one scale, so that a lane's operand is two 16-byte loads.
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
// the summation order.  One wave per expert and TT tokens.
template <int TT>
__global__ __launch_bounds__(256) void k_moe_logits(const float* __restrict__ x,
                                                    const float* __restrict__ router,
                                                    double* __restrict__ logits, int T, int D,
                                                    int E) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (e >= E) return;
  const int t0 = blockIdx.y * TT;
  double acc[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) acc[i] = 0.0;
  const float* const r = router + (int64_t)e * D;
  for (int k = 4 * lane; k < D; k += 256) {
    const float4 w = *reinterpret_cast<const float4*>(r + k);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int t = t0 + i < T ? t0 + i : T - 1;
      const float4 v = *reinterpret_cast<const float4*>(x + (int64_t)t * D + k);
      acc[i] = fma((double)w.x, (double)v.x, acc[i]);
      acc[i] = fma((double)w.y, (double)v.y, acc[i]);
      acc[i] = fma((double)w.z, (double)v.z, acc[i]);
      acc[i] = fma((double)w.w, (double)v.w, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) acc[i] += __shfl_xor(acc[i], o, 64);
    if (lane == 0 && t0 + i < T) logits[(int64_t)(t0 + i) * E + e] = acc[i];
  }
}

// One workgroup per token: an expert's rank among the token's logits is the
// number of experts ahead of it (larger, or equal with a lower index), so
// every rank below top_k names its slot.  Also splits the token's x.
template <int TY>
__global__ __launch_bounds__(512) void k_moe_select(const float* __restrict__ x,
                                                    const double* __restrict__ logits,
                                                    int* __restrict__ ids,
                                                    float* __restrict__ weights,
                                                    uint8_t* __restrict__ xp,
                                                    float* __restrict__ xs, int D, int E,
                                                    int top_k, int norm) {
  __shared__ double sl[512];
  __shared__ float chosen[kMoeMaxTopK];
  __shared__ float part[8];
  __shared__ int nan_seen;
  const int t = blockIdx.x, tid = threadIdx.x;
  if (tid == 0) nan_seen = 0;
  __syncthreads();
  double l = -__builtin_inf();
  if (tid < E) {
    l = logits[(int64_t)t * E + tid];
    if (l != l) {
      l = -__builtin_inf();
      nan_seen = 1;
    }
  }
  sl[tid] = l;
  // x of this token while the logits arrive
  const int nb = D / 32, half = tid >> 5, c = tid & 31;
  for (int b = half; b < nb; b += 16) {
    const float v = x[(int64_t)t * D + 32 * b + c];
    const float amax = half_wave_max(fabsf(v));
    const float s = split_store<TY>(xp + ((int64_t)t * nb + b) * 128, c, v, amax);
    if (c == 0) xs[(int64_t)t * nb + b] = s;
  }
  __syncthreads();
  int rank = 0;
  double best = -__builtin_inf();
  for (int e = 0; e < E; ++e) {
    const double o = sl[e];
    rank += (o > l || (o == l && e < tid)) ? 1 : 0;
    best = o > best ? o : best;
  }
  // exp of the fp64 difference: its fp32 part and the rest to first order
  float p = 0.0f;
  if (tid < E) {
    const double dl = l - best;
    const float hi = (float)dl;
    const float lo = (float)(dl - (double)hi);
    p = expf(hi);
    p = hi > -__builtin_inff() ? fmaf(p, lo, p) : p;
  }
  if (tid < E && rank < top_k) {
    ids[t * top_k + rank] = tid;
    chosen[rank] = p;
  }
  float sum = wave_sum(p);
  if ((tid & 63) == 0) part[tid >> 6] = sum;
  __syncthreads();
  if (tid < top_k) {
    sum = 0.0f;
    if (norm) {
      for (int j = 0; j < top_k; ++j) sum += chosen[j];
    } else {
      for (int j = 0; j < 8; ++j) sum += part[j];
    }
    const float w = chosen[tid] / sum;
    weights[t * top_k + tid] = nan_seen ? __builtin_nanf("") : w;
  }
}

// ---------------------------------------------------------------- weights

// One 16-row tile of weights, a "unit" of kBlocks blocks of 32 k at a time.
// load(): issues the loads of a unit; operand(j): block j as binary16, row
// lane % 16, in lane group order; scale(j): its dw, one per row.
template <int TY>
struct Tile;

template <>
struct Tile<MM_TYPE_Q4_0R> {
  static constexpr int kBlocks = 8;
  const uint8_t* base;
  uint4 c0, c1, d;
  __device__ __forceinline__ void bind(const uint8_t* w, const float*, int64_t e, int N, int K,
                                       int row0, int lane) {
    const int64_t phases = (K + 255) / 256;
    base = w + (e * (N / 16) + row0 / 16) * phases * kQ4RChunk + 16 * lane;
  }
  __device__ __forceinline__ void load(int u, int, int lane) {
    const uint8_t* p = base + (int64_t)u * kQ4RChunk;
    c0 = *reinterpret_cast<const uint4*>(p);
    c1 = *reinterpret_cast<const uint4*>(p + 1024);
    d = *reinterpret_cast<const uint4*>(p - 16 * lane + 2048 + 16 * (lane & 15));
  }
  __device__ __forceinline__ v8h operand(int j) const {
    const uint4& c = j < 4 ? c0 : c1;
    const uint32_t w = (j & 3) == 0 ? c.x : (j & 3) == 1 ? c.y : (j & 3) == 2 ? c.z : c.w;
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
    const uint32_t w = j < 2 ? d.x : j < 4 ? d.y : j < 6 ? d.z : d.w;
    return f16_bits_to_f32((j & 1) ? w >> 16 : w);
  }
};

template <>
struct Tile<MM_TYPE_F8> {
  static constexpr int kBlocks = 4;
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
    for (int j = 0; j < 4; ++j) {
      const int b = 4 * u + j < nb ? 4 * u + j : nb - 1;       // past K: not used
      c[j] = *reinterpret_cast<const uint2*>(base + 32 * (int64_t)b);
    }
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
  static constexpr int kBlocks = 4;
  const uint8_t* base;
  uint4 c[4];
  __device__ __forceinline__ void bind(const uint8_t* w, const float*, int64_t e, int N, int K,
                                       int row0, int lane) {
    base = w + 2 * ((e * N + row0 + (lane & 15)) * K + 8 * (lane >> 4));
  }
  __device__ __forceinline__ void load(int u, int nb, int) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = 4 * u + j < nb ? 4 * u + j : nb - 1;
      c[j] = *reinterpret_cast<const uint4*>(base + 64 * (int64_t)b);
    }
  }
  __device__ __forceinline__ v8h operand(int j) const { return __builtin_bit_cast(v8h, c[j]); }
  __device__ __forceinline__ float scale(int) const { return 1.0f; }
};

// C[m][n] of one block from the split activations: lo first, then hi.
__device__ __forceinline__ v4f block_product(const uint4& hi, const uint4& lo, const v8h& w) {
  const v4f z = {0.f, 0.f, 0.f, 0.f};
  const v4f c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, lo), w, z, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, hi), w, c, 0, 0, 0);
}

// The row scales a lane's four output registers need (rows 4 g + r), each
// row's value held by the lanes of that row index.
__device__ __forceinline__ v4f row_scales(float s, int lane) {
  v4f v;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    v[r] = __builtin_bit_cast(float, __builtin_amdgcn_ds_bpermute(4 * (4 * (lane >> 4) + r), __builtin_bit_cast(int, s)));
  return v;
}

// ---------------------------------------------------------------- gate, up, h

// The experts that any of n assignments names, as a bit set in LDS.
__device__ __forceinline__ void mark_experts(const int* ids, int n, uint32_t* bits) {
  if (threadIdx.x < 16) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int a = threadIdx.x; a < n; a += blockDim.x) atomicOr(&bits[ids[a] >> 5], 1u << (ids[a] & 31));
  __syncthreads();
}

// One workgroup: 32 rows of gate and the same rows of up (four 16-row tiles
// that share each activation load) of the blockIdx.y-th expert in use, over
// its tokens in passes of 16.  Eight waves split K; their partial tiles are
// added in LDS in wave order, then h = silu(g) u, split per block of 32 rows.
template <int TY>
__global__ __launch_bounds__(512) void k_moe_up(MoeArgs a) {
  constexpr int W = 8;
  __shared__ __attribute__((aligned(16))) float part[W * 4 * 256];
  __shared__ uint32_t bits[16];
  __shared__ int list[kMoeMaxTokens];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int assigned = a.T * a.top_k;
  int e = 0, n = 1;
  if (a.T == 1) {
    e = a.ids[blockIdx.y];
    if (tid == 0) list[0] = blockIdx.y;
    __syncthreads();
  } else {
    mark_experts(a.ids, assigned, bits);
    int left = blockIdx.y, word = 0;
    while (word < 16 && left >= __popc(bits[word])) left -= __popc(bits[word++]);
    if (word == 16) return;                          // fewer experts in use than slots
    uint32_t v = bits[word];
    for (; left > 0; --left) v &= v - 1;
    e = 32 * word + __ffs((int)v) - 1;
    if (wave == 0) {
      int c = 0;
      for (int b = 0; b < assigned; b += 64) {
        const bool mine = b + lane < assigned && a.ids[b + lane] == e;
        const uint64_t vote = __ballot(mine);
        if (mine) list[c + __popcll(vote & ((1ull << lane) - 1))] = b + lane;
        c += __popcll(vote);
      }
      if (lane == 0) count = c;
    }
    __syncthreads();
    n = count;
  }
  const int row0 = blockIdx.x * 32;
  const int nb = a.D / 32, units = (nb + Tile<TY>::kBlocks - 1) / Tile<TY>::kBlocks;
  Tile<TY> w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i].bind(i < 2 ? a.gate : a.up, i < 2 ? a.gate_scale : a.up_scale, e, a.F, a.D,
              row0 + 16 * (i & 1), lane);

  for (int m0 = 0; m0 < n; m0 += 16) {
    const bool live = m0 + i16 < n;
    const int tok = live ? list[m0 + i16] / a.top_k : 0;
    const uint8_t* const xrow = a.xp + (int64_t)tok * nb * 128 + 32 * g;
    const float* const xsc = a.xs + (int64_t)tok * nb;
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = (v4f){0.f, 0.f, 0.f, 0.f};
    for (int u = wave; u < units; u += W) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i].load(u, nb, lane);
#pragma unroll
      for (int j = 0; j < Tile<TY>::kBlocks; ++j) {
        const int b = u * Tile<TY>::kBlocks + j;
        if (b >= nb) break;
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        float s = 0.0f;
        if (live) {
          hi = *reinterpret_cast<const uint4*>(xrow + 128 * (int64_t)b);
          lo = *reinterpret_cast<const uint4*>(xrow + 128 * (int64_t)b + 16);
          s = xsc[b];
        }
        const v4f sr = row_scales(s, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const v4f c = block_product(hi, lo, w[i].operand(j));
          const float dw = w[i].scale(j);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(c[r], dw * sr[r], acc[i][r]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[(wave * 4 + i) * 256 + (4 * g + r) * 16 + i16] = acc[i][r];
    __syncthreads();
    {
      const int m = tid >> 5, c = tid & 31;          // 16 tokens x 32 rows
      const float* const p = part + (c >> 4) * 256 + m * 16 + (c & 15);
      float gs = p[0], us = p[512];
#pragma unroll
      for (int v = 1; v < W; ++v) {
        gs += p[v * 1024];
        us += p[v * 1024 + 512];
      }
      const float h = gs / (1.0f + expf(-gs)) * us;
      const float amax = half_wave_max(fabsf(h));
      if (m0 + m < n) {
        const int64_t blk = (int64_t)list[m0 + m] * (a.F / 32) + blockIdx.x;
        const float s = split_store<TY>(a.hp + blk * 128, c, h, amax);
        if (c == 0) a.hs[blk] = s;
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- down

// One workgroup: 16 rows of dst for NT tiles of 16 tokens, summed over the
// experts those tokens use.  Row m of operand A is token m, zero where the
// token does not use the expert, so the experts' contributions add up in the
// accumulators; the waves take (expert, unit) pairs in turn and are joined
// in LDS in wave order.
template <int TY, int NT>
__global__ __launch_bounds__(512) void k_moe_down(MoeArgs a) {
  constexpr int W = 8;
  __shared__ __attribute__((aligned(16))) float part[W * NT * 256];
  __shared__ int sids[16 * NT * kMoeMaxTopK];
  __shared__ uint32_t bits[16];
  __shared__ int used[512];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, i16 = lane & 15;
  const int t0 = blockIdx.y * 16 * NT, k = a.top_k;
  const int tokens = min(16 * NT, a.T - t0);
  for (int i = tid; i < 16 * NT * k; i += blockDim.x) sids[i] = i < tokens * k ? a.ids[t0 * k + i] : -1;
  mark_experts(a.ids + t0 * k, tokens * k, bits);
  if (wave == 0) {
    int c = 0;
    for (int b = 0; b < a.E; b += 64) {
      const int e = b + lane;
      const bool in = e < a.E && (bits[e >> 5] >> (e & 31) & 1);
      const uint64_t vote = __ballot(in);
      if (in) used[c + __popcll(vote & ((1ull << lane) - 1))] = e;
      c += __popcll(vote);
    }
    if (lane == 0) count = c;
  }
  __syncthreads();
  const int row0 = blockIdx.x * 16;
  const int nb = a.F / 32, units = (nb + Tile<TY>::kBlocks - 1) / Tile<TY>::kBlocks;
  const int total = count * units;

  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = (v4f){0.f, 0.f, 0.f, 0.f};
  for (int idx = wave; idx < total; idx += W) {
    const int slot = idx / units, u = idx - slot * units;
    const int e = __builtin_amdgcn_readfirstlane(used[slot]);
    Tile<TY> w;
    w.bind(a.down, a.down_scale, e, a.D, a.F, row0, lane);
    w.load(u, nb, lane);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int at = -1;
      for (int j = 0; j < k; ++j)
        if (sids[(16 * t + i16) * k + j] == e) at = (t0 + 16 * t + i16) * k + j;
      if (__ballot(at >= 0) == 0) continue;
      const uint8_t* const hrow = a.hp + (int64_t)max(at, 0) * nb * 128 + 32 * g;
      const float* const hsc = a.hs + (int64_t)max(at, 0) * nb;
      const float p = at >= 0 ? a.weights[at] : 0.0f;
#pragma unroll
      for (int j = 0; j < Tile<TY>::kBlocks; ++j) {
        const int b = u * Tile<TY>::kBlocks + j;
        if (b >= nb) break;
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        float s = 0.0f;
        if (at >= 0) {
          hi = *reinterpret_cast<const uint4*>(hrow + 128 * (int64_t)b);
          lo = *reinterpret_cast<const uint4*>(hrow + 128 * (int64_t)b + 16);
          s = hsc[b] * p;
        }
        const v4f sr = row_scales(s, lane);
        const v4f c = block_product(hi, lo, w.operand(j));
        const float dw = w.scale(j);
        // s = 0: a token without this expert, which a NaN weight must not reach
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = sr[r] != 0.0f ? fmaf(c[r], dw * sr[r], acc[t][r]) : acc[t][r];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[(wave * NT + t) * 256 + (4 * g + r) * 16 + i16] = acc[t][r];
  __syncthreads();
  for (int i = tid; i < 256 * NT; i += blockDim.x) {
    float s = part[i];
#pragma unroll
    for (int v = 1; v < W; ++v) s += part[v * NT * 256 + i];
    const int t = t0 + (i >> 4);
    if (t < a.T) a.dst[(int64_t)t * a.D + row0 + (i & 15)] = s;
  }
}

template <int TY>
hipError_t run(const MoeArgs& a, hipStream_t s) {
  if (a.T == 1)
    hipLaunchKernelGGL((k_moe_logits<1>), dim3((a.E + 3) / 4, 1), dim3(256), 0, s, a.x, a.router, a.logits, a.T, a.D, a.E);
  else
    hipLaunchKernelGGL((k_moe_logits<4>), dim3((a.E + 3) / 4, (a.T + 3) / 4), dim3(256), 0, s, a.x, a.router, a.logits, a.T, a.D, a.E);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_moe_select<TY>), dim3(a.T), dim3(512), 0, s, a.x, a.logits, a.ids, a.weights,
                     a.xp, a.xs, a.D, a.E, a.top_k, a.norm);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int assigned = a.T * a.top_k;
  hipLaunchKernelGGL((k_moe_up<TY>), dim3(a.F / 32, assigned < a.E ? assigned : a.E), dim3(512), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.T <= 16)
    hipLaunchKernelGGL((k_moe_down<TY, 1>), dim3(a.D / 16, 1), dim3(512), 0, s, a);
  else if (a.T <= 32)
    hipLaunchKernelGGL((k_moe_down<TY, 2>), dim3(a.D / 16, 1), dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((k_moe_down<TY, 4>), dim3(a.D / 16, (a.T + 63) / 64), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe(int type, const MoeArgs& a, hipStream_t s) {
  switch (type) {
    case MM_TYPE_Q4_0R: return run<MM_TYPE_Q4_0R>(a, s);
    case MM_TYPE_F8: return run<MM_TYPE_F8>(a, s);
    case MM_TYPE_F16: return run<MM_TYPE_F16>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qsg
