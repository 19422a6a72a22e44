// Coding of microscaled blocks (mx.hip, add_norm.hip): 32 entries of a row
// share one power of two, and are kept as e4m3 or e2m1 values over it.
//
// The scale is the least power of two 2^e, e >= -127, under which the block's
// largest magnitude is at most the format's largest value (448 or 6), kept as
// the byte e + 127: nothing is cut off, as it is where the scale is taken from the
// magnitude's power of two alone.  x / 2^e is exact in fp32, so the only rounding is the one
// to the format, to nearest even: every run and every implementation gets the
// same bits.  Rows are padded to whole blocks with zero codes.
//   e4m3: off by at most 2^-4 of the value (2^-10 * 2^e below 2^-6 * 2^e).  An
//         infinity or NaN becomes a NaN and leaves its neighbours as they are.
//   e2m1: off by at most 1/4 of the value (2^-2 * 2^e below 2^e).  The format
//         has no NaN, so a block with an infinity or NaN gets the byte 255,
//         under which every entry is a NaN.
#pragma once

#include "row_ops.h"

namespace mdlm {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxNan = 255u;

// The byte of a block of e2m1 codes from the bits of its largest magnitude:
// 6 = 1.5 * 2^2 (e4m3's is ckpt_exp_byte: 448 = 1.75 * 2^8).
__device__ __forceinline__ uint32_t mx4_exp_byte(uint32_t top) {
  const int b = (int)(top >> 23) - 2 + ((top & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return (uint32_t)(b > 0 ? b : 0);
}

// 2^(b - 127), NaN for the byte 255.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __uint_as_float(b == kMxNan ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
}

// Largest magnitude over each four lanes.
__device__ __forceinline__ uint32_t lanes4_max(uint32_t x) {
  return dpp_max<kXor2>(dpp_max<kXor1>(x));
}

// Bits of the largest magnitude of eight values (kNonFinite or more if one is
// not finite).
__device__ __forceinline__ uint32_t top_of8(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = m > a ? m : a;
  }
  return m;
}

// Eight of a block's entries, four lanes of a quad holding the block (all of
// them take part): this lane's codes, and the block's byte.
__device__ __forceinline__ uint2 mx8_encode(const float v[8], uint32_t& byte) {
  const uint32_t top = lanes4_max(top_of8(v));
  if (__ballot(top >= kNonFinite) == 0) {
    byte = ckpt_exp_byte(top);
    return ckpt_encode8<false>(v, ckpt_inv_scale(byte));
  }
  byte = ckpt_exp_byte(lanes4_max(finite_top8(v)));
  return ckpt_encode8<true>(v, ckpt_inv_scale(byte));
}

__device__ __forceinline__ uint32_t mx4_encode(const float v[8], uint32_t& byte) {
  const uint32_t top = lanes4_max(top_of8(v));
  const bool fine = top < kNonFinite;
  byte = fine ? mx4_exp_byte(top) : kMxNan;
  const float inv = ckpt_inv_scale(fine ? byte : 0u);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * inv, v[1] * inv, 1.f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * inv, v[3] * inv, 1.f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * inv, v[5] * inv, 1.f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * inv, v[7] * inv, 1.f, 3);
  return fine ? c : 0u;
}

// Values of eight e2m1 codes, given 2^e (exact in fp32).
__device__ __forceinline__ void mx4_decode(uint32_t c, float scale, float v[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 1);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 2);
  const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.f, 3);
  v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
  v[4] = d.x * scale, v[5] = d.y * scale, v[6] = e.x * scale, v[7] = e.y * scale;
}

}  // namespace mdlm
