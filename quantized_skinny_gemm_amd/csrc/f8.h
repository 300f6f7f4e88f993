// Device helpers of the e4m3 type with one fp32 scale per block of 128, shared by
// its quantizer and products (f8.hip) and the norm that writes it (norm.hip).  The
// codec is described in f8.hip.
#pragma once

#include "device.h"

namespace qsg {

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

}  // namespace qsg
