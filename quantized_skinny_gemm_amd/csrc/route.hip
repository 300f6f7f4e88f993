// Routing to experts, for gfx950: scores of a token's logits, the choice by score
// plus bias within the best groups, the chosen scores as weights.
//
// One wave per token; lane l holds experts l, l + 64, ... (R of them).  Scores are
// fp64: which experts run must not hang on a rounding.  A choice is compared as
// an integer that orders as the number does (0: not to be had, 1: NaN), the upper
// half first: a maximum over the wave by DPP, then the lanes that hold it; only
// where several do (equal upper halves) the lower halves and the indices decide.
// Bound: dependent latencies.  One token, 256 experts in 8 groups, sigmoid, 8 chosen:
// 5.3 us as traced, of which 1.7 are what one choice among 64 experts takes (launch, read,
// a score, write), 0.8 four experts per lane and their bias, 1.5 the groups, 1.4 the seven
// further experts chosen (0.2 each); the wave waits for 72% of its time.  4095
// tokens, 64 experts, 6 chosen: softmax 5.6 us, sigmoid 5.1; with one chosen 4.4 and
// 3.7.  There vector instructions take about 2.5 us of a SIMD's time (one in seven is
// fp64: the exponentials do not bound it), and a wave waits for 58% of its.
#include "device.h"
#include "kernels.h"
#include "../../include/mm.h"

namespace qsg {

namespace {

constexpr double kInf = __builtin_inf();

template <int kCtrl, int kRowMask>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRowMask, 0xf, false));
}
// Maximum over the wave, in every lane.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = dpp_umax<0xB1, 0xf>(v);
  v = dpp_umax<0x4E, 0xf>(v);
  v = dpp_umax<0x141, 0xf>(v);
  v = dpp_umax<0x140, 0xf>(v);
  v = dpp_umax<0x142, 0xa>(v);      // row_bcast15 into rows 1 and 3
  v = dpp_umax<0x143, 0xc>(v);      // row_bcast31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ double readlane_d(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// An integer that orders as c does; a score plus bias is never -0.
__device__ __forceinline__ uint64_t order_of(double c) {
  if (c != c) return 1;
  const uint64_t b = __builtin_bit_cast(uint64_t, c);
  return b >> 63 ? ~b : b | 1ull << 63;
}

constexpr int kTokens = 4;           // waves, and tokens, per workgroup

template <int R>
__global__ __launch_bounds__(64 * kTokens) void k_route(RouteArgs a) {
  __shared__ double choice[kTokens][64 * R];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kTokens + wave;
  if (t >= a.T) return;                              // whole waves; no barriers below
  const float* const row = a.logits + t * a.E;

  float l[R], b[R];
  float top = -__builtin_inff();
  bool odd = false;                                  // NaN, or infinite under a softmax
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < a.E ? row[e] : -__builtin_inff();
    b[i] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    odd |= l[i] != l[i] || (a.softmax && l[i] == __builtin_inff());
    top = fmaxf(top, l[i]);
  }
  const bool poisoned = __any(odd);
  double p[R];
  if (a.softmax) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      p[i] = l[i] > -__builtin_inff() ? exp((double)l[i] - (double)top) : 0.0;
      if (l[i] != l[i]) p[i] = __builtin_nan("");
      s += p[i];
    }
    s = wave_sum_d(s);
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] = s > 0.0 ? p[i] / s : p[i];
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }

  uint64_t key[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const double c = p[i] + (double)b[i];
    const bool masked = l[i] == -__builtin_inff() || b[i] == -__builtin_inff();
    key[i] = masked ? 0 : order_of(c);
    if (a.groups > 1) choice[wave][lane + 64 * i] = masked || c != c ? -kInf : c;
  }
  if (a.groups > 1) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    // `lpg` lanes per group, a power of two: each its best two, then theirs joined
    const int lpg = a.lanes_per_group, g = lane / lpg, per = a.E / a.groups;
    double first = -kInf, second = -kInf;
    if (g < a.groups)
      for (int j = lane % lpg; j < per; j += lpg) {
        const double v = choice[wave][g * per + j];
        second = fmax(second, fmin(first, v));
        first = fmax(first, v);
      }
    for (int o = 1; o < lpg; o <<= 1) {
      const double f = __shfl_xor(first, o, 64), s = __shfl_xor(second, o, 64);
      second = fmax(fmax(second, s), fmin(first, f));
      first = fmax(first, f);
    }
    const double v = a.group_top == 2 && second > -kInf ? first + second : first;
    int ahead = 0;
    for (int o = 0; o < a.groups; ++o) {
      const double w = readlane_d(v, o * lpg);
      ahead += w > v || (w == v && o < g) ? 1 : 0;
    }
    const uint64_t kept = __ballot(g < a.groups && ahead < a.group_k);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int e = lane + 64 * i;
      if (e < a.E && !(kept >> (e / per * lpg) & 1)) key[i] = 0;
    }
  }

  int id = -1;                                       // lane j: slot j
  double w = 0.0, total = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t k = key[0];
    double s = p[0];
    int e = lane;
#pragma unroll
    for (int i = 1; i < R; ++i)
      if (key[i] > k) { k = key[i]; s = p[i]; e = lane + 64 * i; }
    const uint32_t hi = wave_umax((uint32_t)(k >> 32));
    uint64_t who = __ballot((uint32_t)(k >> 32) == hi);
    if (__popcll(who) > 1) {                         // uniform
      const bool in = (uint32_t)(k >> 32) == hi;
      const uint32_t lo = wave_umax(in ? (uint32_t)k : 0u);
      const bool tie = in && (uint32_t)k == lo;
      const uint32_t least = wave_umax(tie ? ~(uint32_t)e : 0u);
      who = __ballot(tie && ~(uint32_t)e == least);
    }
    const int from = __ffsll((unsigned long long)who) - 1;
    const uint64_t best = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), from) << 32 |
                          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, from);
    if (best == 0) break;                            // uniform: nothing is left
    const double sw = readlane_d(s, from);
    const int se = __builtin_amdgcn_readlane(e, from);
    if (lane == j) { id = se; w = sw; }
    total += sw;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (lane + 64 * i == se) key[i] = 0;
  }
  if (lane < a.top_k) {
    if (a.norm) w = total > 0.0 ? w / total : 0.0;
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = poisoned ? __builtin_nanf("") : (float)(w * (double)a.scale);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const dim3 g((unsigned)((a.T + kTokens - 1) / kTokens)), b(64 * kTokens);
  if (a.E <= 64) hipLaunchKernelGGL((k_route<1>), g, b, 0, s, a);
  else if (a.E <= 128) hipLaunchKernelGGL((k_route<2>), g, b, 0, s, a);
  else if (a.E <= 256) hipLaunchKernelGGL((k_route<4>), g, b, 0, s, a);
  else if (a.E <= 512) hipLaunchKernelGGL((k_route<8>), g, b, 0, s, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace qsg
