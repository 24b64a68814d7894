// Products of two matrices whose rows both run along the contraction:
//   out[b][a] = epilogue( sum_k A[a][k] B[b][k] )
// in signed bytes (int32 sums) or bf16 (fp32 sums).  Both element types are
// moved as 64-byte row pieces: one MFMA step takes 16 bytes of a row a lane
// (v_mfma_i32_16x16x64_i8: 64 elements, v_mfma_f32_16x16x32_bf16: 32).
// A's rows are the MFMA's rows, so a lane ends up with four neighbouring
// outputs of one row of `out`.
#pragma once

#include "sg_internal.h"

namespace sg {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

// What happens to a sum.
enum {
  EP_LINEAR = 0,  // (int + a_off[a] * b_sum[b]) * a_scale[a] * b_scale[b]
  EP_PLAIN = 1,   // the fp32 sum
  EP_MASKED = 2   // the fp32 sum where mask[b][a] == 0, else 0; optionally added to `out`
};

struct NtArgs {
  const unsigned char* A;
  const unsigned char* B;
  int64_t lda, ldb;     // bytes between rows
  int64_t na, nb;       // rows
  int64_t kbytes;       // contraction, a multiple of 64 bytes, zero-padded in one operand at least
  void* out;
  int out_dtype;
  int64_t ldo;
  const int32_t* a_off;
  const float* a_scale;
  const float* b_scale;
  const int32_t* b_sum;
  const uint8_t* mask;  // [nb x na], contiguous
  int accumulate;
};

__device__ __forceinline__ uint32_t bf16_of(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

template <bool I8>
struct NtAcc;
template <>
struct NtAcc<true> {
  typedef intx4 type;
  static __device__ __forceinline__ type zero() { return intx4{0, 0, 0, 0}; }
  static __device__ __forceinline__ type mma(u32x4 a, u32x4 b, type c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, a), __builtin_bit_cast(intx4, b), c, 0, 0,
                                                 0);
  }
};
template <>
struct NtAcc<false> {
  typedef floatx4 type;
  static __device__ __forceinline__ type zero() { return floatx4{0.f, 0.f, 0.f, 0.f}; }
  static __device__ __forceinline__ type mma(u32x4 a, u32x4 b, type c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
};

// Four neighbouring outputs of row b from column a on (those inside the
// matrix), from four sums.
template <int EP, typename V4>
__device__ __forceinline__ void nt_store4(const NtArgs& g, int64_t a, int64_t b, V4 v, bool vec) {
  if (b >= g.nb || a >= g.na) return;
  const int cnt = (int)(g.na - a < 4 ? g.na - a : 4);
  float f[4];
  if constexpr (EP == EP_LINEAR) {
    const float sb = g.b_scale[b];
    const int32_t qb = g.b_sum[b];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ai = a + (i < cnt ? i : 0);
      // wraps like the sums of two's complement; the total fits (n <= 65536)
      const uint32_t tot = (uint32_t)v[i] + (uint32_t)g.a_off[ai] * (uint32_t)qb;
      // the channel's scale first: a sum times the scale of a huge token could
      // leave the range that the output stays in
      f[i] = (float)(int32_t)tot * g.a_scale[ai] * sb;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
  if constexpr (EP == EP_MASKED) {
    if (g.mask) {
      const uint8_t* mk = g.mask + b * g.na + a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt && mk[i]) f[i] = 0.0f;
    }
  }
  if (g.out_dtype == SG_F32) {
    float* o = static_cast<float*>(g.out) + b * g.ldo + a;
    if (vec && cnt == 4) {
      floatx4 w = floatx4{f[0], f[1], f[2], f[3]};
      if (EP == EP_MASKED && g.accumulate) w += *reinterpret_cast<const floatx4*>(o);
      *reinterpret_cast<floatx4*>(o) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) o[i] = f[i] + ((EP == EP_MASKED && g.accumulate) ? o[i] : 0.0f);
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
    if (EP == EP_MASKED && g.accumulate) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) f[i] += bf16_to_f32(o[i]);
    }
    if (vec && cnt == 4) {
      const uint2 w = make_uint2(bf16_of(f[0]) | (bf16_of(f[1]) << 16), bf16_of(f[2]) | (bf16_of(f[3]) << 16));
      *reinterpret_cast<uint2*>(o) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) o[i] = (uint16_t)bf16_of(f[i]);
    }
  }
}

// Whether four neighbouring outputs can be stored at once.
inline bool nt_vec_out(const NtArgs& g) {
  const int64_t e = g.out_dtype == SG_F32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(g.out) % (4 * e) == 0 && g.ldo % 4 == 0;
}

}  // namespace sg
