// y = residual + (kept ? x / (1 - p) : 0), the mask made from a counter and
// never stored.  The gradient with respect to x is the same call on dy.
#include "dropout.h"

#include <algorithm>

namespace sg {
namespace {

template <typename XT>
struct Row8;  // eight neighbours of a row
template <>
struct Row8<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_any*>(p); }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&f)[8]) {
    u32x4 w;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[2 * k]) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[2 * k + 1]) << 16);
    *reinterpret_cast<u32x4_any*>(p) = w;
  }
};
template <>
struct Row8<float> {
  u32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const u32x4_any*>(p);
    v[1] = *reinterpret_cast<const u32x4_any*>(p + 4);
  }
  __device__ __forceinline__ float get(int e) const { return __uint_as_float(v[e >> 2][e & 3]); }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<u32x4_any*>(p + 4 * k) =
          __builtin_bit_cast(u32x4, floatx4{f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]});
  }
};

__device__ __forceinline__ float as_f32(uint16_t h) { return bf16_to_f32(h); }
__device__ __forceinline__ float as_f32(float f) { return f; }
__device__ __forceinline__ void put(uint16_t* p, float f) { *p = __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ void put(float* p, float f) { *p = f; }

// A thread takes eight neighbours of a row: two counters.  x times the factor
// is rounded to fp32, the sum with the residual again, then to the type.
//
// Bound by HBM, with the generator's 40 wide multiplies for eight elements close behind:
// 8192 x 8192 in bf16 55 us (4.9 TB/s), with a residual 73 (5.5); 8192 x 4096 in fp32 41
// (6.6).  Rows of any alignment are read and written 16 bytes at a time: 8191 x 4095 in
// bf16 30 us, element by element 70.
template <typename XT, bool RES>
__global__ __launch_bounds__(256) void dropout_kernel(XT* Y, int64_t ldy, const XT* X, int64_t ldx, const XT* R,
                                                      int64_t ldr, int64_t T, int64_t n, const DropArgs d) {
  const DropKey key = drop_key(d);
  const int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
  if (c0 >= n) return;
  for (int64_t t = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; t < T; t += (int64_t)gridDim.y * blockDim.y) {
    const XT* x = X + t * ldx + c0;
    const XT* r = RES ? R + t * ldr + c0 : nullptr;
    XT* y = Y + t * ldy + c0;
    const u32x4 w[2] = {drop_words(key, (uint32_t)t, (uint32_t)(c0 >> 2)),
                        drop_words(key, (uint32_t)t, (uint32_t)(c0 >> 2) + 1)};
    auto one = [&](int e, float xv, float rv) {
      const float kept = w[e >> 2][e & 3] >= d.threshold ? __fmul_rn(xv, d.grow) : 0.0f;
      return RES ? __fadd_rn(kept, rv) : kept;
    };
    if (c0 + 8 <= n) {
      Row8<XT> xv, rv;
      xv.load(x);
      if constexpr (RES) rv.load(r);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = one(e, xv.get(e), RES ? rv.get(e) : 0.0f);
      Row8<XT>::store(y, f);
    } else {
      const int last = (int)(n - 1 - c0);  // (elements past the last re-read it, without a branch for each)
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = one(e, as_f32(x[min(e, last)]), RES ? as_f32(r[min(e, last)]) : 0.0f);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e <= last) put(y + e, f[e]);
    }
  }
}

template <typename XT>
void launch_dropout_t(void* Y, int64_t ldy, const void* X, int64_t ldx, const void* R, int64_t ldr, int64_t T,
                      int64_t n, const DropArgs& d, hipStream_t st) {
  XT* const y = static_cast<XT*>(Y);
  const XT *const x = static_cast<const XT*>(X), *const r = static_cast<const XT*>(R);
  const int64_t cpr = ceil_div(n, 8);
  int bx = 4;
  while (bx < 256 && bx < cpr) bx *= 2;
  const dim3 block((unsigned)bx, (unsigned)(256 / bx));
  const int64_t gx = ceil_div(cpr, bx);  // (a launch holds less than 2^32 threads)
  const dim3 grid((unsigned)gx, (unsigned)std::min({ceil_div(T, 256 / bx), (int64_t)65535, ((int64_t)1 << 23) / gx}));
  if (R)
    dropout_kernel<XT, true><<<grid, block, 0, st>>>(y, ldy, x, ldx, r, ldr, T, n, d);
  else
    dropout_kernel<XT, false><<<grid, block, 0, st>>>(y, ldy, x, ldx, r, ldr, T, n, d);
}

}  // namespace

sg_status launch_dropout(void* Y, int64_t ldy, const void* X, int dtype, int64_t ldx, const void* R, int64_t ldr,
                         int64_t T, int64_t n, const DropArgs& d, hipStream_t st) {
  if (dtype == SG_BF16)
    launch_dropout_t<uint16_t>(Y, ldy, X, ldx, R, ldr, T, n, d, st);
  else
    launch_dropout_t<float>(Y, ldy, X, ldx, R, ldr, T, n, d, st);
  return check_launch("sg_dropout");
}

}  // namespace sg
