// Device helpers of the microscaled 4-bit type (MXFP4), shared by its quantizer
// and products (mx4.hip) and the norm that writes it (norm.hip).
//
// Codec: 32 values along K share a scale 2^(byte - 127),
//   byte = max(floor(log2(amax)) - 2 + 127, 0), code = e2m1(x / 2^(byte - 127)),
// round to nearest, ties to the even code; magnitudes past 6 (at most 8) become
// 6.  The quotient is exact (or below 2^-100, where the code is 0).  A block with
// an infinity or NaN gets byte 255 (NaN) and codes 0.
#pragma once

#include "device.h"

namespace qsg {

// The scale byte of a block from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t mx4_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}

// Codes of eight values of a block, first value in the lowest four bits.
__device__ __forceinline__ uint32_t mx4_pack8(const float4& a, const float4& b, uint32_t byte) {
  // 2^(127 - byte): a normal number, since byte <= 252 where it is used
  const float inv = __builtin_bit_cast(float, byte == 255 ? 0u : (254u - byte) << 23);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a.x * inv, a.y * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a.z * inv, a.w * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, b.x * inv, b.y * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, b.z * inv, b.w * inv, 1.0f, 3);
  return byte == 255 ? 0 : w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}
__device__ __forceinline__ uint32_t amax8_bits(const float4& a, const float4& b) {
  return max(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w))),
             max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
}

// A group of 128 values by 16 lanes of a DPP row, 8 values each (zeros past the
// row's end): this lane's codes, and the group's four scale bytes in every lane.
// `live`: the lane's block lies inside the row (its byte is 127 otherwise).
__device__ __forceinline__ uint32_t mx4_group(const float4& a, const float4& b, bool live, int lane,
                                              uint32_t& bytes) {
  uint32_t m = amax8_bits(a, b);
  m = max(m, (uint32_t)dpp_i<0xB1>((int)m));         // quad_perm [1,0,3,2]
  m = max(m, (uint32_t)dpp_i<0x4E>((int)m));         // quad_perm [2,3,0,1]: the block of 32
  const uint32_t byte = mx4_byte(m);
  uint32_t s = (live ? byte : 127u) << (8 * ((lane >> 2) & 3));
  // lanes 0..15 hold quads 0 0 0 0 1 1 1 1 2 2 2 2 3 3 3 3: or over half rows, then rows
  s |= (uint32_t)dpp_i<0x141>((int)s);               // row_half_mirror: quads 0|1, 2|3
  s |= (uint32_t)dpp_i<0x140>((int)s);               // row_mirror: all four
  bytes = s;
  return mx4_pack8(a, b, byte);
}

}  // namespace qsg
