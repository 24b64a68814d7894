// A layer's activations, gradients and weights in 8-bit floating point.
//
//   rows     blocks of 128 neighbours of a row: Q[t][c], scale[c / 128][t]
//   columns  blocks of 128 neighbours of a column, transposed: Qt[c][t], scale[t / 128][c]
//   weights  blocks of 128 x 128, both ways
//   read back  x[r][c] = code * scale
//
// The scale bytes of one block of the contraction lie side by side for all
// rows, so that a tile of a product fetches them in one piece a stage.
//
// All of these kernels are bound by HBM, after dropout by the generator's multiplies
// beside it.  8192 x 11008 in bf16, beside a copy of the same number of bytes by torch (5.08
// TB/s; the chip's 8 TB/s would take 34, 34, 45, 45 and 34) (us): rows 48 (53), columns 57
// (53), both 80 (71); after dropout 78, 73 and 91; weights both ways 75 (71), read back 45
// (53); both of 515 x 1000, where latency counts, 5.9.
#include "dropout.h"
#include "f8.h"

#include <algorithm>
#include <type_traits>

namespace sg {
namespace {

// Eight elements of a row from column c0 on as fp32 bits; columns from n on
// read as 0 and are not touched in memory.  `inside` (the same for a workgroup):
// all of its columns are below n.
template <typename XT>
__device__ __forceinline__ void load8(const XT* row, int64_t c0, int64_t n, bool inside, uint32_t (&u)[8]) {
  if (inside || c0 + 8 <= n) {
    if constexpr (sizeof(XT) == 2) {
      const u32x4 v = *reinterpret_cast<const u32x4_any*>(row + c0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[2 * k] = v[k] << 16;
        u[2 * k + 1] = v[k] & 0xffff0000u;
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4_any*>(row + c0);
      const u32x4 b = *reinterpret_cast<const u32x4_any*>(row + c0 + 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = a[k];
        u[4 + k] = b[k];
      }
    }
    return;
  }
  // (columns past the last re-read it, without a branch for each)
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const XT v = row[min(c0 + k, n - 1)];
    if constexpr (sizeof(XT) == 2)
      u[k] = c0 + k < n ? (uint32_t)v << 16 : 0u;
    else
      u[k] = c0 + k < n ? __float_as_uint(v) : 0u;
  }
}

// Dropout of eight elements of row t from column c0 on.
__device__ __forceinline__ void drop8(const DropArgs& d, const DropKey& key, int64_t t, int64_t c0, uint32_t (&u)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x4 w = drop_words(key, (uint32_t)t, (uint32_t)(c0 >> 2) + h);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[4 * h + e] = w[e] >= d.threshold ? __float_as_uint(__fmul_rn(__uint_as_float(u[4 * h + e]), d.grow)) : 0u;
  }
}

// As unsigned integers magnitudes order like their values, and NaN and
// infinity lie above every finite one.
__device__ __forceinline__ uint32_t peak8(const uint32_t (&u)[8]) {
  uint32_t p = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) p = max(p, u[e] & 0x7fffffffu);
  return p;
}

// The largest over a row of 16 lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));  // row_ror:8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
}

constexpr uint32_t kInf = 0x7f800000u;

// Codes of eight elements of a block with this peak, `live` of them inside the
// matrix (the others are 0).  A block with a NaN or an infinity is NaN.
template <bool E5>
__device__ __forceinline__ uint2 codes8(const uint32_t (&u)[8], uint32_t peak, uint32_t byte, int live) {
  if (peak >= kInf) {
    const uint64_t m = live >= 8 ? ~0ull : (1ull << (8 * max(live, 0))) - 1;
    const uint64_t w = 0x0101010101010101ull * kF8NaN & m;
    return make_uint2((uint32_t)w, (uint32_t)(w >> 32));
  }
  const float s = f8_down(byte);
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[e]) * s;
  return make_uint2(f8_codes<E5>(f[0], f[1], f[2], f[3]), f8_codes<E5>(f[4], f[5], f[6], f[7]));
}

template <bool E5>
__device__ __forceinline__ uint32_t scale_byte(uint32_t peak) {
  return peak >= kInf ? 127u : f8_scale_of<E5>(peak);
}

// Rows: 16 lanes a block of 128, 16 rows a workgroup at a time.  One row a lane:
// with four in flight (their loads ahead of the first use) 8192 x 11008 takes 54
// instead of 47 us, 512 x 4096 3.3 instead of 2.9.
template <typename XT, bool E5, bool DROP>
__global__ __launch_bounds__(256) void f8_rows_kernel(uint8_t* __restrict__ Q, int64_t ldq,
                                                      uint8_t* __restrict__ scale, int64_t lds,
                                                      const XT* __restrict__ X, int64_t T, int64_t n, int64_t ldx,
                                                      const DropArgs d) {
  const int tid = threadIdx.x;
  const int64_t kb = blockIdx.x;
  const int64_t c0 = kb * kF8Block + (tid & 15) * 8;
  const DropKey key = DROP ? drop_key(d) : DropKey{};
  const bool inside = (kb + 1) * kF8Block <= n;
  for (int64_t t = (int64_t)blockIdx.y * 16 + (tid >> 4); t < T; t += (int64_t)gridDim.y * 16) {  // (whole groups of 16 lanes)
    uint32_t u[8];
    load8<XT>(X + t * ldx, c0, n, inside, u);
    if constexpr (DROP) drop8(d, key, t, c0, u);
    const uint32_t peak = max16(peak8(u));
    const uint32_t byte = scale_byte<E5>(peak);
    *reinterpret_cast<uint2*>(Q + t * ldq + c0) = codes8<E5>(u, peak, byte, (int)min<int64_t>(n - c0, 8));
    if ((tid & 15) == 0) scale[kb * lds + t] = (uint8_t)byte;
  }
}

struct F8Out {
  uint8_t* q;
  int64_t ldq;
  uint8_t* scale;
  int64_t lds;
};

// Codes of four elements.
template <bool E5>
__device__ __forceinline__ uint32_t codes4(const uint32_t (&u)[4], uint32_t peak, uint32_t byte, int live) {
  if (peak >= kInf) return 0x01010101u * kF8NaN & (live >= 4 ? ~0u : (1u << (8 * max(live, 0))) - 1);
  const float s = f8_down(byte);
  return f8_codes<E5>(__uint_as_float(u[0]) * s, __uint_as_float(u[1]) * s, __uint_as_float(u[2]) * s,
                      __uint_as_float(u[3]) * s);
}

// Tiles of 128 x 128, four rows by eight columns a thread: columns, or columns
// and rows, or (WHOLE) one scale for the tile and both ways.  rows.q or cols.q
// may be NULL.  The first row is row0 of the whole matrix.  X is read once and
// stays in registers between the maxima and the codes; eight rows a thread and
// half the threads took 84 instead of 80 us (both of 8192 x 11008) and 7.5 instead of 5.9
// (of 515 x 1000).
template <typename XT, bool E5, bool DROP, bool WHOLE>
__global__ __launch_bounds__(512) void f8_tile_kernel(const F8Out rows, const F8Out cols, const XT* __restrict__ X,
                                                      int64_t T, int64_t n, int64_t ldx, int64_t tiles_n,
                                                      const DropArgs d, int64_t row0) {
  constexpr int RP = 4;
  __shared__ uint32_t s_peak[kF8Block];
  __shared__ __attribute__((aligned(16))) uint8_t s_turn[kF8Block * kF8Block];
  const int tid = threadIdx.x;
  const int64_t kt = blockIdx.x / tiles_n, kc = blockIdx.x - kt * tiles_n;
  const int cl = (tid & 15) * 8, rl = (tid >> 4) * RP;  // in the tile
  const int64_t c0 = kc * kF8Block + cl, t0 = kt * kF8Block + rl;
  const bool inside = (kc + 1) * kF8Block <= n;
  uint32_t u[RP][8];
#pragma unroll
  for (int k = 0; k < RP; ++k) {
    if (t0 + k < T) {
      load8<XT>(X + (t0 + k) * ldx, c0, n, inside, u[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[k][e] = 0u;
    }
  }
  if constexpr (DROP) {
    const DropKey key = drop_key(d);
#pragma unroll
    for (int k = 0; k < RP; ++k) drop8(d, key, row0 + t0 + k, c0, u[k]);  // (zeros stay zeros)
  }
  const int live_c = (int)min<int64_t>(n - c0, 8), live_t = (int)min<int64_t>(T - t0, RP);
  uint32_t whole = 0u;
  if constexpr (WHOLE) {
#pragma unroll
    for (int k = 0; k < RP; ++k) whole = max(whole, peak8(u[k]));
    whole = max16(whole);
    if ((tid & 15) == 0) s_peak[tid >> 4] = whole;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kF8Block / RP; ++w) whole = max(whole, s_peak[w]);
  } else if (cols.q) {
    if (tid < kF8Block) s_peak[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t p = 0u;
#pragma unroll
      for (int k = 0; k < RP; ++k) p = max(p, u[k][e] & 0x7fffffffu);
      atomicMax(&s_peak[cl + e], p);
    }
  }
  if (rows.q) {
#pragma unroll
    for (int k = 0; k < RP; ++k) {
      const uint32_t peak = WHOLE ? whole : max16(peak8(u[k]));
      const uint32_t byte = scale_byte<E5>(peak);
      if (k < live_t) {
        *reinterpret_cast<uint2*>(rows.q + (t0 + k) * rows.ldq + c0) = codes8<E5>(u[k], peak, byte, live_c);
        if ((tid & 15) == 0) rows.scale[kc * rows.lds + t0 + k] = (uint8_t)byte;
      }
    }
  }
  if (!cols.q) return;
  if constexpr (!WHOLE) __syncthreads();
  // A thread's codes of a column are four bytes of 128; they are turned in LDS, so
  // that whole rows of the transposed form are stored.  Piece s (of eight bytes) of
  // column c lies at s ^ ((c / 8) % 16): the 16 columns that lanes write at a time
  // are 8 apart.
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t p = WHOLE ? whole : s_peak[cl + e];
    const uint32_t byte = scale_byte<E5>(p);
    const uint32_t v[4] = {u[0][e], u[1][e], u[2][e], u[3][e]};
    *reinterpret_cast<uint32_t*>(s_turn + (cl + e) * kF8Block + ((rl / 8) ^ (tid & 15)) * 8 + (rl & 4)) =
        codes4<E5>(v, p, byte, live_t);
    if (rl == 0 && e < live_c) cols.scale[kt * cols.lds + c0 + e] = (uint8_t)byte;
  }
  __syncthreads();
  const int64_t tc0 = kc * kF8Block, tt0 = kt * kF8Block;
#pragma unroll
  for (int i = 0; i < RP; ++i) {
    const int c = kF8Block / RP * i + (tid >> 4), piece = tid & 15;
    if (tc0 + c < n)
      *reinterpret_cast<uint2*>(cols.q + (tc0 + c) * cols.ldq + tt0 + piece * 8) =
          *reinterpret_cast<const uint2*>(s_turn + c * kF8Block + (piece ^ ((c >> 3) & 15)) * 8);
  }
}

// Sixteen codes a thread: one load, and whole 16-byte stores at any alignment
// (stored one by one, rows off 16 bytes took 82 instead of 18 us, 8191 x 4095).
// blockDim = (bx, by): bx threads along a row.
template <typename XT, bool E5>
__global__ __launch_bounds__(256) void f8_values_kernel(XT* __restrict__ X, int64_t ldx,
                                                        const uint8_t* __restrict__ Q, int64_t ldq,
                                                        const uint8_t* __restrict__ scale, int64_t lds, int64_t T,
                                                        int64_t n) {
  const int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 16;
  if (c0 >= n) return;
  for (int64_t t = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; t < T; t += (int64_t)gridDim.y * blockDim.y) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(Q + t * ldq + c0);
    const float s = f8_up(scale[c0 / kF8Block * lds + t]);
    floatx4 f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = f8_values<E5>(v[k]) * s;
    XT* o = X + t * ldx + c0;
    if constexpr (sizeof(XT) == 2) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[k >> 1][2 * (k & 1)]) |
               ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f[k >> 1][2 * (k & 1) + 1]) << 16);
      if (c0 + 16 <= n) {
        *reinterpret_cast<u32x4_any*>(o) = u32x4{w[0], w[1], w[2], w[3]};
        *reinterpret_cast<u32x4_any*>(o + 8) = u32x4{w[4], w[5], w[6], w[7]};
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < n) o[e] = (XT)(w[e >> 1] >> (16 * (e & 1)));
      }
    } else {
      if (c0 + 16 <= n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<u32x4_any*>(o + 4 * k) = __builtin_bit_cast(u32x4, f[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c0 + e < n) o[e] = f[e >> 2][e & 3];
      }
    }
  }
}

// A launch holds less than 2^32 threads.
constexpr int64_t kMaxGroups = (int64_t)1 << 22;

template <typename XT, bool E5, bool DROP>
void launch_quantize(const F8Out& rows, const F8Out& cols, const XT* X, int64_t T, int64_t n, int64_t ldx,
                     const DropArgs& d, hipStream_t st) {
  const int64_t kn = ceil_div(n, kF8Block);
  if (!cols.q) {
    const int64_t gy = std::min<int64_t>(65535, kMaxGroups / kn);
    f8_rows_kernel<XT, E5, DROP><<<dim3((unsigned)kn, (unsigned)std::min(ceil_div(T, 16), gy)), 256, 0, st>>>(
        rows.q, rows.ldq, rows.scale, rows.lds, X, T, n, ldx, d);
    return;
  }
  const int64_t most = kMaxGroups / kn * kF8Block;  // rows of X in a launch
  for (int64_t t = 0; t < T; t += most) {
    const int64_t part = std::min(most, T - t);
    F8Out r = rows, c = cols;
    if (r.q) r.q += t * r.ldq, r.scale += t;
    c.q += t, c.scale += t / kF8Block * c.lds;
    f8_tile_kernel<XT, E5, DROP, false><<<(unsigned)(ceil_div(part, kF8Block) * kn), 512, 0, st>>>(
        r, c, X + t * ldx, part, n, ldx, kn, d, t);
  }
}

template <typename XT, bool E5>
void launch_quantize_t(const F8Out& rows, const F8Out& cols, const void* X, int64_t T, int64_t n, int64_t ldx,
                       const DropArgs* d, hipStream_t st) {
  const XT* x = static_cast<const XT*>(X);
  if (d)
    launch_quantize<XT, E5, true>(rows, cols, x, T, n, ldx, *d, st);
  else
    launch_quantize<XT, E5, false>(rows, cols, x, T, n, ldx, DropArgs{}, st);
}

}  // namespace

sg_status launch_quantize_f8(uint8_t* Q, int64_t ldq, uint8_t* q_scale, int64_t ldqs, uint8_t* Qt, int64_t ldqt,
                             uint8_t* qt_scale, int64_t ldqts, int format, const void* X, int x_dtype, int64_t T,
                             int64_t n, int64_t ldx, const DropArgs* drop, hipStream_t st) {
  const F8Out rows{Q, ldq, q_scale, ldqs}, cols{Qt, ldqt, qt_scale, ldqts};
  if (x_dtype == SG_BF16) {
    if (format == SG_E5M2)
      launch_quantize_t<uint16_t, true>(rows, cols, X, T, n, ldx, drop, st);
    else
      launch_quantize_t<uint16_t, false>(rows, cols, X, T, n, ldx, drop, st);
  } else {
    if (format == SG_E5M2)
      launch_quantize_t<float, true>(rows, cols, X, T, n, ldx, drop, st);
    else
      launch_quantize_t<float, false>(rows, cols, X, T, n, ldx, drop, st);
  }
  return check_launch("sg_quantize_f8");
}

sg_status launch_pack_f8(uint8_t* Wq, int64_t ldw, uint8_t* w_scale, int64_t ldws, uint8_t* Wt, int64_t ldwt,
                         uint8_t* wt_scale, int64_t ldwts, const void* W, int w_dtype, int64_t m, int64_t n,
                         int64_t ld, hipStream_t st) {
  const F8Out rows{Wq, ldw, w_scale, ldws}, cols{Wt, ldwt, wt_scale, ldwts};
  const int64_t kn = ceil_div(n, kF8Block);
  const unsigned grid = (unsigned)(ceil_div(m, kF8Block) * kn);  // at most 2^13 x 2^9
  const DropArgs none{};
  if (w_dtype == SG_BF16)
    f8_tile_kernel<uint16_t, false, false, true><<<grid, 512, 0, st>>>(rows, cols, static_cast<const uint16_t*>(W), m, n,
                                                                      ld, kn, none, 0);
  else
    f8_tile_kernel<float, false, false, true><<<grid, 512, 0, st>>>(rows, cols, static_cast<const float*>(W), m, n, ld,
                                                                   kn, none, 0);
  return check_launch("sg_pack_f8");
}

sg_status launch_dequantize_f8(void* X, int x_dtype, int64_t ldx, const uint8_t* Q, int64_t ldq,
                               const uint8_t* scale, int64_t lds, int format, int64_t T, int64_t n, hipStream_t st) {
  const int64_t cpr = ceil_div(n, 16);
  int bx = 4;
  while (bx < 256 && bx < cpr) bx *= 2;
  const dim3 block((unsigned)bx, (unsigned)(256 / bx));
  const int64_t gx = ceil_div(cpr, bx);
  const dim3 grid((unsigned)gx, (unsigned)std::min({ceil_div(T, 256 / bx), (int64_t)65535, kMaxGroups / gx}));
  const bool e5 = format == SG_E5M2;
  auto go = [&](auto* x) {
    typedef typename std::remove_pointer<decltype(x)>::type XT;
    if (e5)
      f8_values_kernel<XT, true><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, lds, T, n);
    else
      f8_values_kernel<XT, false><<<grid, block, 0, st>>>(x, ldx, Q, ldq, scale, lds, T, n);
  };
  if (x_dtype == SG_BF16)
    go(static_cast<uint16_t*>(X));
  else
    go(static_cast<float*>(X));
  return check_launch("sg_dequantize_f8");
}

}  // namespace sg
