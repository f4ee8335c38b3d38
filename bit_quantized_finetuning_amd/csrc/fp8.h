// 8-bit floating point on gfx950: conversions, the row quantizer's power-of-two
// scale, and the 16 x 16 x 128 matrix instruction.
//
// e4m3 (4 exponent bits, 3 of mantissa, largest value 448, no infinity) and
// e5m2 (5 and 2, largest finite value 57344), both as torch's float8_e4m3fn and
// float8_e5m2 define them. v_cvt_pk_{fp8,bf8}_f32 round to nearest even; an
// e4m3 conversion of anything from 464 up (and of NaN) gives NaN, so callers
// scale first.
#pragma once

#include <cmath>

#include "common.h"

namespace qlora {

typedef int i32x2v __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp8Group = 128;        // values of a row, rows / columns of a weight block, per scale
constexpr float kE4m3Max = 448.f;
constexpr float kFp8Tiny = 0x1p-100f;  // the least magnitude a scale is made for (an all-zero group's)

// Four floats to four bytes, element order.
template <bool E5M2>
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  int v;
  if constexpr (E5M2) {
    v = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, v, true);
  } else {
    v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  }
  return (uint32_t)v;
}

// The row quantizer's scale: the least power of two s with amax <= MAX * s. The
// largest value of either format is 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2), so
// s = 2^(e - 8) for amax = f * 2^e with f <= 1.75 and 2^(e - 7) above; adding
// 0x1fffff to the bits carries into the exponent exactly when f > 1.75. Being a
// power of two it divides without rounding, so the codes carry the only one,
// and the group's relative precision is that of any other scale (the format is
// a floating one); the range lost is below one binade.
struct RowScale {
  float s, inv;
};
template <bool E5M2>
__device__ __forceinline__ RowScale row_scale(float amax) {
  const uint32_t bits = __float_as_uint(fmaxf(amax, kFp8Tiny));
  const uint32_t e = ((bits + 0x1fffffu) >> 23) - (E5M2 ? 15u : 8u);
  return RowScale{__uint_as_float(e << 23), __uint_as_float((254u - e) << 23)};
}

// max over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float max16(float v) {
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0xB1, 0xf, 0xf, true)));   // quad xor 1
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x4E, 0xf, 0xf, true)));   // quad xor 2
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x141, 0xf, 0xf, true)));  // half mirror
  v = fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x140, 0xf, 0xf, true)));  // mirror
  return v;
}

// D = A B + C over 128 values of K: lane l holds row (column) l & 15 and 32 bytes
// of K; which K the bytes of lane group l >> 4 stand for is the caller's choice
// as long as both operands agree. D: lane l holds column (l & 15) of the second
// operand, rows 4 (l >> 4) + i of the first. A is e4m3; B is e4m3 or e5m2.
template <bool B_E5M2>
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, B_E5M2 ? 1 : 0, 0, 0, 0, 0);
}

// Two float32 values as two bf16 terms each: the upper 8 bits of the significand
// (cut, so that nothing rounds up to an infinity) and the rest, rounded: at most
// 2^-15 of the value is lost. An infinity leaves no rest.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo) {
  auto rest = [](float x) {
    return fabsf(x) == INFINITY ? 0.f : x - __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  };
  hi = perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  lo = pack_bf16x2(rest(a), rest(b));
}

__device__ __forceinline__ i32x8 join8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

}  // namespace qlora
