// Device helpers of the kernels that work on rows of H entries (embed.hip,
// norm.hip, ckpt8.hip): eight entries at a time as fp32, sums over lanes, and
// the 8-bit checkpoint's coding of a block of 128 entries.
#pragma once

#include "mdlm_internal.h"

namespace mdlm {

typedef __bf16 bf16_t;

// Global memory takes 16-byte accesses at any address that is a multiple of
// the entry's size, so rows of odd length need no path of their own: only
// the entries past the last whole eight are read and written one at a time.
// These types carry that alignment, and the compiler still emits one wide
// instruction for each.
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Eight consecutive entries as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  uint32_t w[4];
};
template <>
struct Raw8<float> {
  float w[8];
};

// Entries [c, c + 8) of a row of H; entries past the row's end read as zero.
// FULL: H is a multiple of 8.  Rows shorter than c read nothing.
template <bool FULL>
__device__ __forceinline__ Raw8<bf16_t> load8(const bf16_t* __restrict__ row, int c, int H) {
  Raw8<bf16_t> r;
  if (c + 8 <= H) {
    const u32x4_a2 v = *reinterpret_cast<const u32x4_a2*>(row + c);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else {
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0;
    if (!FULL) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (c + i < H) r.w[i / 2] |= (uint32_t)p[c + i] << (16 * (i & 1));
    }
  }
  return r;
}

template <bool FULL>
__device__ __forceinline__ Raw8<float> load8(const float* __restrict__ row, int c, int H) {
  Raw8<float> r;
  if (c + 8 <= H) {
    const f32x4_a4 a = *reinterpret_cast<const f32x4_a4*>(row + c);
    const f32x4_a4 b = *reinterpret_cast<const f32x4_a4*>(row + c + 4);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
    r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = 0.f;
    if (!FULL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (c + i < H) r.w[i] = row[c + i];
    }
  }
  return r;
}

__device__ __forceinline__ void widen(const Raw8<bf16_t>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.w[i];
}

// fp32 -> entries, rounded to nearest even (one instruction for two).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef bf16_t bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <bool FULL>
__device__ __forceinline__ void store8(bf16_t* __restrict__ row, int c, int H,
                                       const float v[8]) {
  if (c + 8 <= H) {
    u32x4_a2 o;
    o.x = pack_bf16(v[0], v[1]), o.y = pack_bf16(v[2], v[3]);
    o.z = pack_bf16(v[4], v[5]), o.w = pack_bf16(v[6], v[7]);
    *reinterpret_cast<u32x4_a2*>(row + c) = o;
  } else if (!FULL) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) row[c + i] = (bf16_t)v[i];
  }
}

template <bool FULL>
__device__ __forceinline__ void store8(float* __restrict__ row, int c, int H, const float v[8]) {
  if (c + 8 <= H) {
    f32x4_a4 a, b;
    a.x = v[0], a.y = v[1], a.z = v[2], a.w = v[3];
    b.x = v[4], b.y = v[5], b.z = v[6], b.w = v[7];
    *reinterpret_cast<f32x4_a4*>(row + c) = a;
    *reinterpret_cast<f32x4_a4*>(row + c + 4) = b;
  } else if (!FULL) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) row[c + i] = v[i];
  }
}

// The same for a caller that knows (FULL) that [c, c + 8) lies in the row: no
// condition remains.
template <bool FULL, typename T>
__device__ __forceinline__ Raw8<T> load8_in(const T* row, int c, int H) {
  return FULL ? load8<true>(row, c, c + 8) : load8<false>(row, c, H);
}
template <bool FULL, typename T>
__device__ __forceinline__ void store8_in(T* row, int c, int H, const float v[8]) {
  FULL ? store8<true>(row, c, c + 8, v) : store8<false>(row, c, H, v);
}

// ---- reductions over lanes -----------------------------------------------
// Data-parallel-primitive controls: lane ^ 1 and lane ^ 2 within a quad, and
// the mirrors within 8 and within 16 lanes.  After the first two every quad
// holds one value, so a mirror pairs each lane with the other quad (other
// half) as an exchange would.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

// Sum over each 16 lanes, the same on all of them.
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp<kXor1>(x);
  x += dpp<kXor2>(x);
  x += dpp<kMirror8>(x);
  x += dpp<kMirror16>(x);
  return x;
}
// Largest value over each 16 (LANES = 8: each 8) lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
  return x > y ? x : y;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
  x = dpp_max<kXor1>(x);
  x = dpp_max<kXor2>(x);
  x = dpp_max<kMirror8>(x);
  return LANES == 8 ? x : dpp_max<kMirror16>(x);
}
// Sum over the wave (every lane must be active), the same on all lanes.
__device__ __forceinline__ float wave_sum(float x) {
  const int r = __builtin_bit_cast(int, row16_sum(x));
  const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 0));
  const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 16));
  const float c = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 32));
  const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(r, 48));
  return (a + b) + (c + d);
}

// The value that lane `from` (the same on all lanes) holds.
__device__ __forceinline__ float lane_value(float x, int from) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), from));
}

// A use of x that computes nothing: a load into it has come by then.
template <typename X>
__device__ __forceinline__ void arrived(X& x) {
  asm volatile("" : "+v"(x));
}

__device__ __forceinline__ void arrived(Raw8<bf16_t>& r) { arrived(r.w[0]); }
__device__ __forceinline__ void arrived(Raw8<float>& r) { arrived(r.w[0]), arrived(r.w[4]); }

// ---- 8-bit checkpoint ------------------------------------------------------
// A block of 128 entries x is kept as e4m3 values q and one byte b for the
// block: x ~ q * 2^e, e = b - 127, where 2^e is the least power of two (not
// below 2^-127) that brings the block's largest finite magnitude to 448 (the
// largest e4m3 value) or less.  The scale being a power of two, x / 2^e is
// exact in fp32 and the only rounding is the one to e4m3, off by at most
// 2^-4 of the value (2^-10 * 2^e below the least normal one): every run and
// every implementation gets the same bits.  An infinity or NaN becomes a NaN
// and leaves its neighbours as they are.
constexpr int kCkptBlock = 128;

// The block's byte from the bits of its largest finite magnitude:
// 448 = 1.75 * 2^8, so e = (exponent of top) - 8, one more when top's
// significand passes 1.75.
__device__ __forceinline__ uint32_t ckpt_exp_byte(uint32_t top) {
  const int b = (int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(b > 0 ? b : 0);
}
__device__ __forceinline__ float ckpt_inv_scale(uint32_t b) {  // 2^-e, b <= 247
  return __uint_as_float((254u - b) << 23);
}
__device__ __forceinline__ float ckpt_scale(uint32_t b) {  // 2^e; 2^-127 is subnormal
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

// Largest magnitude of eight entries, as fp32 bits; an infinity or NaN gives
// kNonFinite or more.
constexpr uint32_t kNonFinite = 0x7F800000u;
__device__ __forceinline__ uint32_t top8(const Raw8<bf16_t>& r) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, r.w[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.w[i] & 0x7FFF7FFFu));
  return (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
}
__device__ __forceinline__ uint32_t top8(const Raw8<float>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(r.w[i]) & 0x7FFFFFFFu;
    m = m > a ? m : a;
  }
  return m;
}
// The same over the finite ones alone.
__device__ __forceinline__ uint32_t finite_top8(const float v[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = a < kNonFinite && a > m ? a : m;
  }
  return m;
}

// Codes of eight entries, given 2^-e.  CHECK: some may not be finite.
template <bool CHECK>
__device__ __forceinline__ uint2 ckpt_encode8(const float v[8], float inv) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    s[i] = !CHECK || __builtin_isfinite(v[i]) ? v[i] * inv : __builtin_nanf("");
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// Values of eight codes, given 2^e (exact in fp32).
__device__ __forceinline__ void ckpt_decode8(uint2 q, float scale, float v[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false);
  const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
  v[0] = a.x * scale, v[1] = a.y * scale, v[2] = b.x * scale, v[3] = b.y * scale;
  v[4] = c.x * scale, v[5] = c.y * scale, v[6] = d.x * scale, v[7] = d.y * scale;
}

template <bool FULL>
__device__ __forceinline__ uint2 load8_codes(const uint8_t* __restrict__ row, int c, int H) {
  if (c + 8 <= H) {
    const u32x2_a1 v = *reinterpret_cast<const u32x2_a1*>(row + c);
    return make_uint2(v.x, v.y);
  }
  uint2 r = make_uint2(0u, 0u);
  if (!FULL) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) {
        const uint32_t b = (uint32_t)row[c + i] << (8 * (i & 3));
        if (i < 4)
          r.x |= b;
        else
          r.y |= b;
      }
  }
  return r;
}

template <bool FULL>
__device__ __forceinline__ uint2 load8_codes_in(const uint8_t* row, int c, int H) {
  return FULL ? load8_codes<true>(row, c, c + 8) : load8_codes<false>(row, c, H);
}

template <bool FULL>
__device__ __forceinline__ void store8_codes(uint8_t* __restrict__ row, int c, int H, uint2 q) {
  if (c + 8 <= H) {
    u32x2_a1 v;
    v.x = q.x, v.y = q.y;
    *reinterpret_cast<u32x2_a1*>(row + c) = v;
  } else if (!FULL) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < H) row[c + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}

template <bool FULL>
__device__ __forceinline__ void store8_codes_in(uint8_t* row, int c, int H, uint2 q) {
  FULL ? store8_codes<true>(row, c, c + 8, q) : store8_codes<false>(row, c, H, q);
}

// Sixteen codes at once where the row has them all (a 16-byte access).
template <bool FULL>
__device__ __forceinline__ void store16_codes(uint8_t* __restrict__ row, int c, int H, uint2 q0,
                                              uint2 q1) {
  if (FULL || c + 16 <= H) {
    u32x4_a1 v;
    v.x = q0.x, v.y = q0.y, v.z = q1.x, v.w = q1.y;
    *reinterpret_cast<u32x4_a1*>(row + c) = v;
  } else {
    store8_codes<false>(row, c, H, q0);
    store8_codes<false>(row, c + 8, H, q1);
  }
}

}  // namespace mdlm
