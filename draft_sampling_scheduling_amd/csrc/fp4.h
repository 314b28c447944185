// fp4.h -- elements held in 4 bits: E2M1 codes (sign, two bits of exponent, one of mantissa: 0, .5,
// 1, 1.5, 2, 3, 4, 6), 32 of them with a power of two, 2^(byte - 127), as gfx950's conversions take
// them.
//
// Quantising a group: the power 2^e is the smallest with max|x| <= 7 * 2^e.  Then no value is off
// by more than half a step of the codes around it, for 7 is as far from 6 as the middle of two
// codes 2 apart is from either; of a value in the middle the even code is taken, as the hardware
// does.  e stays in [-120, 125], where every value is a normal float and bf16; a group that holds
// an infinity or NaN gets byte 255, and all of it reads as NaN.
#pragma once

#include "dev.h"

namespace dspark {

constexpr int kGroup4 = 32;            // elements that share a power of two
constexpr uint32_t kScaleNaN = 255;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// byte's power of two, for the conversions below (they take the exponent's bits alone: 0 is 2^-127
// and 255 NaN, as the byte says; measured over every code and byte)
__device__ __forceinline__ float fp4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// two codes of a byte (0 .. 3) of eight
template <int BYTE>
__device__ __forceinline__ uint32_t fp4_bf16(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, BYTE));
}
// eight codes as bf16: exact but for powers past 2^125
__device__ __forceinline__ uint4 fp4_bf16x8(uint32_t codes, float scale) {
  return make_uint4(fp4_bf16<0>(codes, scale), fp4_bf16<1>(codes, scale), fp4_bf16<2>(codes, scale),
                    fp4_bf16<3>(codes, scale));
}
__device__ __forceinline__ void fp4_f32x8(uint32_t codes, float scale, float (&x)[8]) {
  const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
  const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
  const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
  const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y; x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}

// What quantising looks at: a float's bits.  A double on its way to a code is first a float that
// lies between the same two floats of 23 bits, its last bit set if the double is not that float
// itself: codes, and the middles between them, have 2 bits, so each comes out as from the double.
__device__ __forceinline__ uint32_t fp4_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t fp4_bits(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x);
  const uint32_t hi = (uint32_t)(u >> 32), lo = (uint32_t)u, size = hi & 0x7FFFFFFFu;
  uint32_t f;
  if (size >= 0x7FF00000u)
    f = 0x7FC00000u;  // infinite or NaN
  else if (size >= 0x47F00000u)
    f = 0x7F7FFFFFu;  // 2^128 and more: past the largest code of the largest power
  else if (size < 0x38100000u)
    f = 0;  // below 2^-126: 0 at any power
  else
    f = ((size - 0x38000000u) << 3 | lo >> 29) | ((lo & 0x1FFFFFFFu) != 0);
  return f | (hi & 0x80000000u);
}

// the byte of a group whose largest |x| has these bits
__device__ __forceinline__ uint32_t fp4_byte(uint32_t top) {
  const uint32_t expo = top >> 23;  // 127 + floor(log2)
  if (expo == 255) return kScaleNaN;
  const int byte = (int)expo - 2 + ((top & 0x7FFFFFu) > 0x600000u);  // 7 is 1.75 * 2^2
  return (uint32_t)min(max(byte, 127 - 120), 127 + 125);
}

// codes of eight values (their bits) of a group with this byte
__device__ __forceinline__ uint32_t fp4_codes(const uint32_t (&x)[8], uint32_t byte) {
  if (byte == kScaleNaN) return 0;
  const float scale = fp4_scale(byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(x[0]), __uint_as_float(x[1]), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(x[2]), __uint_as_float(x[3]), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(x[4]), __uint_as_float(x[5]), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(x[6]), __uint_as_float(x[7]), scale, 3);
}

}  // namespace dspark
