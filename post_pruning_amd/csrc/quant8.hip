// The 8-bit forms of a layer's activations and weights.
//
//   quantize    s_t = max_c |x_tc| / 127,  q_tc = nearest code of 127 x_tc / max_c |x_tc|
//   read back   x_tc ~ q_tc s_t
//   pack        a layer's uint8 codes as signed bytes in padded rows
//
// All three are bound by HBM: a bf16 activation is 2 bytes in and 1 byte out.
#include "sg_internal.h"

#include <algorithm>

namespace sg {
namespace {

constexpr int QCH = 8;  // elements one thread handles at a time

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}

__device__ __forceinline__ int wave_sum_i32(int v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Eight elements of a row from column c0 on, as the bits of fp32 values;
// columns from n on read as 0 and are not touched in memory.
template <typename XT, bool VEC>
__device__ __forceinline__ void load_chunk(const XT* row, int64_t c0, int64_t n, uint32_t (&u)[QCH]) {
  if (VEC && c0 + QCH <= n) {
    if constexpr (sizeof(XT) == 2) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(row + c0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[2 * k] = v[k] << 16;
        u[2 * k + 1] = v[k] & 0xffff0000u;
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4*>(row + c0);
      const u32x4 b = *reinterpret_cast<const u32x4*>(row + c0 + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = a[k];
        u[4 + k] = b[k];
      }
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < QCH; ++k) {
    u[k] = 0u;
    if (c0 + k < n) {
      if constexpr (sizeof(XT) == 2)
        u[k] = (uint32_t)row[c0 + k] << 16;
      else
        u[k] = __float_as_uint(row[c0 + k]);
    }
  }
}

// What a row's codes are formed with.  Rows with a peak below 2^-100 are
// lifted by 2^100 first (exact), so that 127 / peak stays finite.
struct RowScale {
  float peak;  // max |x| (lifted)
  float lift;  // 1 or 2^100
  float inv;   // 127 / peak, 0 for a row of zeros or one with a NaN or an infinity
};

__device__ __forceinline__ RowScale row_scale(uint32_t umax) {
  RowScale r;
  r.lift = umax < 0x0d800000u ? 0x1p100f : 1.0f;
  r.peak = __uint_as_float(umax) * r.lift;
  r.inv = (umax == 0u || umax >= 0x7f800000u) ? 0.0f : 127.0f / r.peak;
  return r;
}

// The code of x: 127 x / peak to the nearest integer, halves to even, as in
// exact arithmetic.  x * inv is off by less than 2^-16 (two roundings of at
// most 2^-24 relative, codes up to 127), so only values that close to a half
// can fall on the wrong side; those compare 254 |x| with (2k + 1) peak, both
// exact in 64 bits (24-bit significands times integers below 2^8).
__device__ __forceinline__ int code_of(uint32_t ubits, const RowScale& rs) {
  const float x = __uint_as_float(ubits) * rs.lift;
  const float r = x * rs.inv;
  float k = rintf(r);
  const float away = fabsf(r - k);
  if (away > 0.5f - 0x1p-14f && rs.inv != 0.0f) {
    const float lo = floorf(fabsf(r));
    const double d = 254.0 * fabs((double)x) - (2.0 * (double)lo + 1.0) * (double)rs.peak;
    const bool odd = ((int)lo & 1) != 0;
    const float kk = (d > 0.0 || (d == 0.0 && odd)) ? lo + 1.0f : lo;
    k = copysignf(kk, x);
  }
  return rs.inv != 0.0f ? (int)k : 0;
}

// One row per TPR threads.  A row of up to KEEP * 8 * TPR elements is read
// once and kept in registers between the peak and the codes; longer rows are
// read a second time (from L2).  Bound by HBM: 32768 x 4096 bf16 take 84-93 us,
// 4.3-4.8 TB/s of bytes read and written (a plain copy reaches 5.2), fp32 118
// us, 5.7 TB/s.  Rows that are not 16-byte aligned are read element by element:
// 182 and 234 us.  A few short rows are bound by latency instead, hence many
// threads a row.
template <typename XT, int TPR, int KEEP, bool VEC>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void quantize_kernel(
    int8_t* __restrict__ Q, int64_t ldq, float* __restrict__ scale, int32_t* __restrict__ sum,
    const XT* __restrict__ X, int64_t T, int64_t n, int64_t ldx) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR;
  constexpr int WPR = TPR / 64;  // waves per row
  __shared__ uint32_t s_max[THREADS / 64];
  __shared__ int s_sum[THREADS / 64];
  const int tid = threadIdx.x;
  const int lt = tid % TPR;
  const int64_t t = (int64_t)blockIdx.x * (THREADS / TPR) + tid / TPR;
  if (TPR == 64 && t >= T) return;  // whole waves; they meet no barrier
  const XT* row = X + t * ldx;
  const int nch = (int)(round_up(n, 64) / QCH);

  uint32_t keep[KEEP > 0 ? KEEP : 1][QCH];
  uint32_t umax = 0u;
  if constexpr (KEEP > 0) {
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (lt + k * TPR < nch) load_chunk<XT, VEC>(row, (int64_t)(lt + k * TPR) * QCH, n, keep[k]);
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (lt + k * TPR < nch) {
#pragma unroll
        for (int e = 0; e < QCH; ++e) umax = max(umax, keep[k][e] & 0x7fffffffu);
      }
  } else {
    for (int c = lt; c < nch; c += TPR) {
      load_chunk<XT, VEC>(row, (int64_t)c * QCH, n, keep[0]);
#pragma unroll
      for (int e = 0; e < QCH; ++e) umax = max(umax, keep[0][e] & 0x7fffffffu);
    }
  }
  // as unsigned integers, magnitudes order like their values and NaN and
  // infinity lie above every finite one
  umax = wave_max_u32(umax);
  if constexpr (WPR > 1) {
    if ((tid & 63) == 0) s_max[tid >> 6] = umax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) umax = max(umax, s_max[w]);
  }
  const RowScale rs = row_scale(umax);

  int total = 0;
  int8_t* qrow = Q + t * ldq;
  auto emit = [&](int c, const uint32_t (&u)[QCH]) {
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < QCH; ++e) {
      const int q = code_of(u[e], rs);
      total += q;
      w[e >> 2] |= ((uint32_t)q & 0xffu) << (8 * (e & 3));
    }
    *reinterpret_cast<uint2*>(qrow + (int64_t)c * QCH) = make_uint2(w[0], w[1]);
  };
  if constexpr (KEEP > 0) {
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      if (lt + k * TPR < nch) emit(lt + k * TPR, keep[k]);
  } else {
    for (int c = lt; c < nch; c += TPR) {
      load_chunk<XT, VEC>(row, (int64_t)c * QCH, n, keep[0]);
      emit(c, keep[0]);
    }
  }
  total = wave_sum_i32(total);
  if constexpr (WPR > 1) {
    if ((tid & 63) == 0) s_sum[tid >> 6] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < WPR; ++w) total += s_sum[w];
  }
  if (lt == 0) {
    scale[t] = umax == 0u ? 1.0f
                          : (umax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(umax) / 127.0f);
    sum[t] = total;
  }
}

// fp32 -> bf16 bits, round to nearest, ties to even; NaN stays a quiet NaN.
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x);
}

// Sixteen codes a thread.  blockDim = (bx, by): bx threads along a row.  Bound
// by HBM: 32768 x 4096 to bf16 take 66-74 us, 5.5-6.1 TB/s of bytes read and
// written, to fp32 169 us, 4.0 TB/s.  Rows that are not 16-byte aligned are
// written element by element: 327 and 624 us.
template <typename XT, bool VEC>
__global__ __launch_bounds__(256) void dequantize_kernel(XT* __restrict__ X, int64_t ldx,
                                                         const int8_t* __restrict__ Q, int64_t ldq,
                                                         const float* __restrict__ scale, int64_t T, int64_t n) {
  const int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 16;
  if (c0 >= n) return;
  for (int64_t t = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; t < T; t += (int64_t)gridDim.y * blockDim.y) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(Q + t * ldq + c0);
    const float s = scale[t];
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = (float)((int32_t)(v[e >> 2] << (24 - 8 * (e & 3))) >> 24) * s;
    XT* o = X + t * ldx + c0;
    if (VEC && c0 + 16 <= n) {
      if constexpr (sizeof(XT) == 2) {
        u32x4 w[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k >> 2][k & 3] = bf16_bits(f[2 * k]) | (bf16_bits(f[2 * k + 1]) << 16);
        *reinterpret_cast<u32x4*>(o) = w[0];
        *reinterpret_cast<u32x4*>(o + 8) = w[1];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<floatx4*>(o + 4 * k) = floatx4{f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]};
      }
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (c0 + e < n) {
          if constexpr (sizeof(XT) == 2)
            o[e] = (XT)bf16_bits(f[e]);
          else
            o[e] = f[e];
        }
    }
  }
}

// A layer's codes as signed bytes (code - 128) in rows padded with zeros to a
// multiple of 64 bytes, and what turns an integer sum into the layer's output:
// sum (code - z) q = sum (code - 128) q + (128 - z) sum q.  Once a layer:
// 11008 x 4096 take 21-24 us, 17 at the rate of a large copy; a thread moves
// only four bytes at a time.
__global__ __launch_bounds__(256) void pack_w8_kernel(int8_t* __restrict__ Wq, int64_t ldw,
                                                      int32_t* __restrict__ offset, float* __restrict__ w_scale,
                                                      const uint8_t* __restrict__ codes,
                                                      const float* __restrict__ scale,
                                                      const float* __restrict__ zero, int64_t m, int64_t n) {
  const int nq = (int)(round_up(n, 64) / 4);
  for (int64_t r = blockIdx.x; r < m; r += gridDim.x) {
    const uint8_t* src = codes + r * n;
    uint32_t* dst = reinterpret_cast<uint32_t*>(Wq + r * ldw);
    const bool vec = (reinterpret_cast<uintptr_t>(src) & 3u) == 0;
    for (int c = threadIdx.x; c < nq; c += blockDim.x) {
      const int64_t c0 = 4 * (int64_t)c;
      uint32_t w = 0u;
      if (vec && c0 + 4 <= n) {
        w = *reinterpret_cast<const uint32_t*>(src + c0) ^ 0x80808080u;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c0 + e < n) w |= (uint32_t)(src[c0 + e] ^ 0x80u) << (8 * e);
      }
      dst[c] = w;
    }
    if (threadIdx.x == 0) {
      const float z = zero[r];
      const bool ok = z >= 0.0f && z <= 255.0f && z == rintf(z);
      offset[r] = ok ? 128 - (int)z : 0;
      w_scale[r] = ok ? scale[r] : __uint_as_float(0x7fc00000u);
    }
  }
}

template <typename XT, bool VEC>
void launch_quantize_rows(int8_t* Q, int64_t ldq, float* scale, int32_t* sum, const XT* X, int64_t T, int64_t n,
                       int64_t ldx, hipStream_t st) {
  // Threads a row.  Many rows (32768, bf16): n = 1024 takes 24 us with 64 and
  // 44 with 256, n = 2048 58 and 53, n = 4096 106 and 86; n = 8192 (8192 rows)
  // 44 with 256 and 91 with 1024.  Few rows are bound by latency: 64 rows of
  // 4096 take 4.9 us with 256 and 4.1 with 1024, one row of 8192 5.2 and 4.1;
  // one row of 1024 4.0 with 64 and 3.6 with 256 or 1024.
  const bool few = T <= 128;
  if (n <= 1024 && !few)
    quantize_kernel<XT, 64, 2, VEC><<<dim3((unsigned)ceil_div(T, 4)), 256, 0, st>>>(Q, ldq, scale, sum, X, T, n, ldx);
  else if (n <= (few ? 2048 : 8192))
    quantize_kernel<XT, 256, 4, VEC><<<dim3((unsigned)T), 256, 0, st>>>(Q, ldq, scale, sum, X, T, n, ldx);
  else if (n <= 32768)
    quantize_kernel<XT, 1024, 4, VEC><<<dim3((unsigned)T), 1024, 0, st>>>(Q, ldq, scale, sum, X, T, n, ldx);
  else
    quantize_kernel<XT, 1024, 0, VEC><<<dim3((unsigned)T), 1024, 0, st>>>(Q, ldq, scale, sum, X, T, n, ldx);
}

// A launch holds less than 2^32 threads, up to 1024 of them a row.
template <typename XT, bool VEC>
void launch_quantize_t(int8_t* Q, int64_t ldq, float* scale, int32_t* sum, const XT* X, int64_t T, int64_t n,
                       int64_t ldx, hipStream_t st) {
  constexpr int64_t most = (int64_t)1 << 21;
  for (int64_t t = 0; t < T; t += most)
    launch_quantize_rows<XT, VEC>(Q + t * ldq, ldq, scale + t, sum + t, X + t * ldx, std::min(most, T - t), n, ldx, st);
}

bool rows_aligned16(const void* p, int64_t ld, int64_t elt) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * elt) % 16 == 0;
}

}  // namespace

sg_status launch_quantize_tokens(int8_t* Q, int64_t ldq, float* scale, int32_t* sum, const void* X, int x_dtype,
                                 int64_t T, int64_t n, int64_t ldx, hipStream_t st) {
  if (x_dtype == SG_BF16) {
    const uint16_t* x = static_cast<const uint16_t*>(X);
    if (rows_aligned16(X, ldx, 2))
      launch_quantize_t<uint16_t, true>(Q, ldq, scale, sum, x, T, n, ldx, st);
    else
      launch_quantize_t<uint16_t, false>(Q, ldq, scale, sum, x, T, n, ldx, st);
  } else {
    const float* x = static_cast<const float*>(X);
    if (rows_aligned16(X, ldx, 4))
      launch_quantize_t<float, true>(Q, ldq, scale, sum, x, T, n, ldx, st);
    else
      launch_quantize_t<float, false>(Q, ldq, scale, sum, x, T, n, ldx, st);
  }
  return check_launch("sg_quantize_tokens");
}

sg_status launch_dequantize_tokens(void* X, int x_dtype, int64_t ldx, const int8_t* Q, int64_t ldq,
                                   const float* scale, int64_t T, int64_t n, hipStream_t st) {
  const int64_t cpr = ceil_div(n, 16);
  int bx = 4;
  while (bx < 256 && bx < cpr) bx *= 2;
  const dim3 block((unsigned)bx, (unsigned)(256 / bx));
  const dim3 grid((unsigned)ceil_div(cpr, bx), (unsigned)std::min<int64_t>(ceil_div(T, 256 / bx), 65535));
  if (x_dtype == SG_BF16) {
    uint16_t* x = static_cast<uint16_t*>(X);
    if (rows_aligned16(X, ldx, 2))
      dequantize_kernel<uint16_t, true><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, T, n);
    else
      dequantize_kernel<uint16_t, false><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, T, n);
  } else {
    float* x = static_cast<float*>(X);
    if (rows_aligned16(X, ldx, 4))
      dequantize_kernel<float, true><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, T, n);
    else
      dequantize_kernel<float, false><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, T, n);
  }
  return check_launch("sg_dequantize_tokens");
}

sg_status launch_pack_w8(int8_t* Wq, int64_t ldw, int32_t* offset, float* w_scale, const uint8_t* codes,
                         const float* scale, const float* zero, int64_t m, int64_t n, hipStream_t st) {
  pack_w8_kernel<<<dim3((unsigned)std::min<int64_t>(m, 1 << 20)), 256, 0, st>>>(Wq, ldw, offset, w_scale, codes, scale,
                                                                               zero, m, n);
  return check_launch("sg_pack_w8");
}

}  // namespace sg
