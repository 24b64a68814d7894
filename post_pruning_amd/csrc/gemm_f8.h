// Products of two matrices in 8-bit floating point whose rows both run along
// the contraction, with a scale for every 128 of it:
//   out[b][a] = epilogue( sum_k A[a][k] 2^ea[k/128][a] B[b][k] 2^eb[k/128][b] )
// A is e4m3, B e4m3 or e5m2.  A's rows are the MFMA's rows, so a lane ends up
// with neighbouring outputs of one row of `out`.
#pragma once

#include "dropout.h"
#include "gemm_nt.h"

namespace sg {

struct F8Args {
  // A, B, na, nb, lda, ldb, out, out_dtype, ldo, mask, accumulate; kbytes a
  // multiple of 128, zero-padded in both operands
  NtArgs g;
  const uint8_t *a_scale, *b_scale;  // bytes e + 127, [kbytes / 128] rows of a_lds and b_lds bytes
  int64_t a_lds, b_lds;
  int has_drop;  // dropout of the outputs, of which the first row is row0 of the whole
  int64_t row0;
  DropArgs drop;
};

typedef int f8_frag __attribute__((ext_vector_type(8)));  // 32 codes of a row: 16-byte pieces p and p + 4 of 128 bytes

// The products of 128 codes a row as exact products with fp32 sums: the codes are widened
// to bf16, which holds them exactly.  (The matrix instruction for 8-bit floating
// point aligns every eight products to the largest of them and cuts what lies
// 2^-13 below it: measured, relative errors of 1.5e-5 to 7e-5.)
struct F8Wide {
  bf16x8 v[4];
};
template <bool E5>
__device__ __forceinline__ F8Wide f8_widen(const f8_frag& f) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  F8Wide w;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    bf16x2 lo, hi;
    if constexpr (E5) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f[q], 1.0f, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f[q], 1.0f, true);
    } else {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[q], 1.0f, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[q], 1.0f, true);
    }
    const int at = 4 * (q & 1);
    w.v[q >> 1][at] = lo[0];
    w.v[q >> 1][at + 1] = lo[1];
    w.v[q >> 1][at + 2] = hi[0];
    w.v[q >> 1][at + 3] = hi[1];
  }
  return w;
}
__device__ __forceinline__ floatx4 f8_dot_wide(const F8Wide& a, const F8Wide& b) {
  floatx4 c = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[q], b.v[q], c, 0, 0, 0);
  return c;
}
// acc += part * 2^(e - 254), e the sum of two scale bytes: one rounding (ldexp
// is exact down to the subnormal numbers), and no intermediate leaves the range.
__device__ __forceinline__ float f8_add_scaled(float acc, float part, int e) {
  return acc + __builtin_amdgcn_ldexpf(part, e - 254);
}

// Dropout of N neighbouring outputs of row b from column a on (a a multiple of 4).
template <int N, typename V4>
__device__ __forceinline__ void f8_drop(const F8Args& f, const DropKey& key, int64_t a, int64_t b, V4 (&v)[N / 4]) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const u32x4 w = drop_words(key, (uint32_t)(f.row0 + b), (uint32_t)(a >> 2) + q);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[q][e] = w[e] >= f.drop.threshold ? v[q][e] * f.drop.grow : 0.0f;
  }
}

}  // namespace sg
