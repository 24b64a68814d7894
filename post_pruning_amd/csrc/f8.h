// Numbers in 8-bit floating point with one scale, a power of two, for every
// block of 128.
//
// A block with the largest magnitude a is held as codes x 2^-e in e4m3 or e5m2
// with the least e >= -127 for which a 2^-e is at most the format's largest
// value, 1.75 * 2^TOP.  x 2^-e is exact in fp32 (or so far below the smallest code that it
// rounds to zero), so the hardware's conversion, to nearest and ties to even,
// decides as exact arithmetic does.  e + 127 is the scale byte that the matrix
// instructions take as it is.
#pragma once

#include "sg_internal.h"

namespace sg {

constexpr int kF8Block = SG_F8_BLOCK;
constexpr uint32_t kF8NaN = 0x7fu;  // a NaN in both formats

// The scale byte of a block whose largest magnitude has these fp32 bits
// (finite).  A block of zeros takes 2^0.
template <bool E5>
__device__ __forceinline__ uint32_t f8_scale_of(uint32_t peak) {
  constexpr int TOP = E5 ? 15 : 8;
  const int byte = (int)(peak >> 23) - TOP + ((peak & 0x7fffffu) > 0x600000u ? 1 : 0);
  return peak == 0u ? 127u : (uint32_t)max(byte, 0);
}

// 2^-e and 2^e of a scale byte e + 127 (bytes up to 248).
__device__ __forceinline__ float f8_down(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float f8_up(uint32_t byte) {
  return __uint_as_float(byte != 0u ? byte << 23 : 1u << 22);
}

// Codes of four scaled values.
template <bool E5>
__device__ __forceinline__ uint32_t f8_codes(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (E5) {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
  return (uint32_t)w;
}

// The values of four codes.
template <bool E5>
__device__ __forceinline__ floatx4 f8_values(uint32_t w) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  f2 lo, hi;
  if constexpr (E5) {
    lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  }
  return floatx4{lo[0], lo[1], hi[0], hi[1]};
}

}  // namespace sg
