// Root-mean-square norm with the residual's addition, for gfx950:
//
//   v = x + residual;  rstd = 1 / sqrt(mean(v^2) + eps);  y = (v * rstd) * weight
//
// v is written too (the residual stream); y as f32, as e4m3 codes with a scale
// per 128 values, or as MXFP4: what the products of those types take, without
// y's way through memory and a quantizer's launch.
//
// A row belongs to 1 to 16 waves of one workgroup; a lane holds up to R pieces
// of 8 consecutive values from the one read to the one write, 16 neighbouring
// lanes a block of 128.  The sum of squares is held in fp64 (the kernel waits for
// memory, so this costs nothing): it does not overflow, and how a row is cut among
// lanes, which follows the number of rows, moves it by about 1e-16 only: rstd, rounded
// to fp32, can differ in its last bit between batches for about one row in 10^8.
// Bound: HBM (8 bytes per value read, 4 written for v, 0.53 to 4 for y).  2047 x 8192
// into MXFP4, 210 MB: 45 us, 4.7 TB/s; 1 x 4096 into e4m3: 3.0 us, launch and the
// latencies of one read, a join over LDS and one write.
#include "f8.h"
#include "kernels.h"
#include "mx4.h"
#include "../../include/mm.h"

namespace qsg {

namespace {

// loads and stores of four floats that need no more than a float's alignment
typedef float v4fu __attribute__((ext_vector_type(4), aligned(4)));

struct Piece {
  float4 a, b;
};

// Values k .. k + 7 of a row of D, zeros past its end.
__device__ __forceinline__ Piece load_piece(const float* row, int k, int D) {
  Piece p;
  if (k + 8 <= D) {
    const v4fu u = *reinterpret_cast<const v4fu*>(row + k), v = *reinterpret_cast<const v4fu*>(row + k + 4);
    p.a = make_float4(u[0], u[1], u[2], u[3]);
    p.b = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    const auto at = [&](int j) { return k + j < D ? row[k + j] : 0.0f; };
    p.a = make_float4(at(0), at(1), at(2), at(3));
    p.b = make_float4(at(4), at(5), at(6), at(7));
  }
  return p;
}

__device__ __forceinline__ void store_piece(float* row, int k, int D, const Piece& p) {
  if (k + 8 <= D) {
    *reinterpret_cast<v4fu*>(row + k) = (v4fu){p.a.x, p.a.y, p.a.z, p.a.w};
    *reinterpret_cast<v4fu*>(row + k + 4) = (v4fu){p.b.x, p.b.y, p.b.z, p.b.w};
  } else {
    const float v[8] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k + j < D) row[k + j] = v[j];
  }
}

__device__ __forceinline__ float4 add4(const float4& a, const float4& b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 scale4(const float4& v, float s, const float4& w) {
  return make_float4(v.x * s * w.x, v.y * s * w.y, v.z * s * w.z, v.w * s * w.w);
}
__device__ __forceinline__ double square4(const float4& v, double s) {
  s = fma((double)v.x, (double)v.x, s);
  s = fma((double)v.y, (double)v.y, s);
  s = fma((double)v.z, (double)v.z, s);
  return fma((double)v.w, (double)v.w, s);
}

// y's piece at k of row t in the output type; 16 neighbouring lanes together
// (a lane past the row's end holds zeros).
template <int TY>
__device__ __forceinline__ void write_y(const NormArgs& a, int64_t t, int k, int lane, const Piece& y) {
  if constexpr (TY == MM_TYPE_F32) {
    if (k < a.D) store_piece((float*)a.y + t * a.D, k, a.D, y);
  } else if constexpr (TY == MM_TYPE_F8) {
    float d;
    const uint2 c = f8_row_block(y.a, y.b, d);
    if (k < a.D) {
      *reinterpret_cast<uint2*>((uint8_t*)a.y + t * a.D + k) = c;
      if ((lane & 15) == 0) ((float*)a.scales)[t * ((a.D + 127) / 128) + k / 128] = d;
    }
  } else {
    uint32_t bytes;
    const uint32_t c = mx4_group(y.a, y.b, k < a.D, lane, bytes);
    if (k < a.D) {
      *reinterpret_cast<uint32_t*>((uint8_t*)a.y + (t * a.D + k) / 2) = c;
      if ((lane & 15) == 0) ((uint32_t*)a.scales)[t * ((a.D + 127) / 128) + k / 128] = bytes;
    }
  }
}

// Workgroups of `rows` rows with `waves` waves each.  R > 0: a row is at most
// 512 waves R values, held in registers; R = 0: rows of any length, read a
// second time (v from `sum` where it is written, which may be x or residual
// itself, so nothing here is declared free of aliases).
template <int TY, int R>
__global__ __launch_bounds__(1024) void k_rms_norm(NormArgs a, int waves, int rows) {
  __shared__ double part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = wave / waves, wr = wave - r * waves;   // row of the workgroup, wave of the row
  const int64_t t = (int64_t)blockIdx.x * rows + r;
  const bool live = t < a.T;
  const int64_t at = (live ? t : 0) * a.D;
  const float* const x = a.x + at;
  const float* const res = a.residual ? a.residual + at : nullptr;
  float* const sum = a.sum ? a.sum + at : nullptr;
  const int k0 = 8 * (wr * 64 + lane), step = 512 * waves;

  const auto value = [&](int k) {
    Piece v = load_piece(x, k, a.D);
    if (res) {
      const Piece q = load_piece(res, k, a.D);
      v.a = add4(v.a, q.a);
      v.b = add4(v.b, q.b);
    }
    return v;
  };
  Piece v[R > 0 ? R : 1], w[R > 0 ? R : 1];
  double s = 0.0;
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] = value(k0 + i * step);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (a.weight) w[i] = load_piece(a.weight, k0 + i * step, a.D);
#pragma unroll
    for (int i = 0; i < R; ++i) s = square4(v[i].b, square4(v[i].a, s));
    if (live && sum) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (k0 + i * step < a.D) store_piece(sum, k0 + i * step, a.D, v[i]);
    }
  } else {
    if (live)
      for (int k = k0; k < a.D; k += step) {
        const Piece p = value(k);
        s = square4(p.b, square4(p.a, s));
        if (sum) store_piece(sum, k, a.D, p);
      }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if (waves > 1) {
    if (lane == 0) part[wave] = s;
    __syncthreads();
    s = 0.0;
    for (int i = 0; i < waves; ++i) s += part[r * waves + i];
  }
  if (!live) return;                                   // whole waves
  const float rstd = (float)(1.0 / sqrt(s / (double)a.D + (double)a.eps));
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  if constexpr (R > 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int k = k0 + i * step;
      Piece y;
      y.a = scale4(v[i].a, rstd, a.weight ? w[i].a : one);
      y.b = scale4(v[i].b, rstd, a.weight ? w[i].b : one);
      if (k >= a.D) y.a = y.b = make_float4(0.f, 0.f, 0.f, 0.f);   // not 0 * an infinite rstd
      write_y<TY>(a, t, k, lane, y);
    }
  } else {
    // whole groups of 16 lanes: a block of 128 ends with the row
    for (int k = k0; k - 8 * (lane & 15) < a.D; k += step) {
      Piece p = sum ? load_piece(sum, k, a.D) : value(k), y;
      const Piece q = a.weight ? load_piece(a.weight, k, a.D) : Piece{one, one};
      y.a = scale4(p.a, rstd, q.a);
      y.b = scale4(p.b, rstd, q.b);
      if (k >= a.D) y.a = y.b = make_float4(0.f, 0.f, 0.f, 0.f);
      write_y<TY>(a, t, k, lane, y);
    }
  }
}

template <int TY>
hipError_t run(const NormArgs& a, hipStream_t s) {
  int waves, rows;
  norm_shape(a.T, a.D, &waves, &rows);
  const int64_t pieces = ((int64_t)a.D + 7) / 8;
  const int64_t held = (pieces + 64 * waves - 1) / (64 * waves), grid = (a.T + rows - 1) / rows;
  const dim3 g((unsigned)grid), b((unsigned)(64 * waves * rows));
  if (held <= 1) hipLaunchKernelGGL((k_rms_norm<TY, 1>), g, b, 0, s, a, waves, rows);
  else if (held <= 2) hipLaunchKernelGGL((k_rms_norm<TY, 2>), g, b, 0, s, a, waves, rows);
  else if (held <= 4) hipLaunchKernelGGL((k_rms_norm<TY, 4>), g, b, 0, s, a, waves, rows);
  else hipLaunchKernelGGL((k_rms_norm<TY, 0>), g, b, 0, s, a, waves, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(int type, const NormArgs& a, hipStream_t s) {
  switch (type) {
    case MM_TYPE_F32: return run<MM_TYPE_F32>(a, s);
    case MM_TYPE_F8: return run<MM_TYPE_F8>(a, s);
    case MM_TYPE_MXFP4: return run<MM_TYPE_MXFP4>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qsg
