// The 8-bit linear layer: its product in integers and its two gradients.
#include "gemm_nt.h"

#include <algorithm>

namespace sg {
namespace {

constexpr int kStreamWaves = 8;

// Every workgroup takes 16 rows of A and 16 * TF rows of B; its waves divide
// the contraction and add their sums up in LDS, in wave order.  Operands go
// from memory straight to the registers the MFMA reads.
template <bool I8, int TF, int EP>
__global__ __launch_bounds__(64 * kStreamWaves) void nt_stream_kernel(const NtArgs g, int vec) {
  typedef typename NtAcc<I8>::type acc_t;
  __shared__ acc_t red[kStreamWaves][TF][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t a0 = (int64_t)blockIdx.x * 16;
  const int64_t b0 = (int64_t)blockIdx.y * (16 * TF);
  const int steps = (int)(g.kbytes / 64);
  const int s0 = (int)((int64_t)steps * wave / kStreamWaves);
  const int s1 = (int)((int64_t)steps * (wave + 1) / kStreamWaves);
  // rows past the end re-read the last one; their sums are not stored
  const int64_t ra = min<int64_t>(a0 + (lane & 15), g.na - 1);
  const unsigned char* pa = g.A + ra * g.lda + (lane >> 4) * 16;
  const unsigned char* pb[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f)
    pb[f] = g.B + min<int64_t>(b0 + 16 * f + (lane & 15), g.nb - 1) * g.ldb + (lane >> 4) * 16;
  acc_t acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = NtAcc<I8>::zero();
  constexpr int U = TF == 1 ? 8 : 4;
  int s = s0;
  for (; s + U <= s1; s += U) {
    u32x4 va[U], vb[U][TF];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      va[u] = *reinterpret_cast<const u32x4*>(pa + (int64_t)(s + u) * 64);
#pragma unroll
      for (int f = 0; f < TF; ++f) vb[u][f] = *reinterpret_cast<const u32x4*>(pb[f] + (int64_t)(s + u) * 64);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int f = 0; f < TF; ++f) acc[f] = NtAcc<I8>::mma(va[u], vb[u][f], acc[f]);
  }
  for (; s < s1; ++s) {
    const u32x4 va = *reinterpret_cast<const u32x4*>(pa + (int64_t)s * 64);
#pragma unroll
    for (int f = 0; f < TF; ++f)
      acc[f] = NtAcc<I8>::mma(va, *reinterpret_cast<const u32x4*>(pb[f] + (int64_t)s * 64), acc[f]);
  }
#pragma unroll
  for (int f = 0; f < TF; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  if (tid < 64 * TF) {
    const int f = tid >> 6;
    acc_t v = red[0][f][lane];
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) v += red[w][f][lane];
    nt_store4<EP>(g, a0 + (lane >> 4) * 4, b0 + 16 * f + (lane & 15), v, vec != 0);
  }
}

constexpr int kBand = 8;  // panels of A whose tiles run together

template <bool I8, int EP, int TA, int TB, int WA, int WB, int RA, int RB, bool BT>
__global__ __launch_bounds__(64 * WA * WB) void nt_tile_kernel(const NtArgs g, NtWide wide, int64_t ta, int64_t tb) {
  typedef NtTile<I8, TA, TB, WA, WB, RA, RB, BT> Tile;
  __shared__ __attribute__((aligned(16))) unsigned char lds[Tile::LDS];
  const int64_t k = nt_xcd_order(blockIdx.x, ta * tb);
  if (k < 0) return;
  int64_t ia, ib;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  typename Tile::acc_t acc[Tile::FA][Tile::FB];
#pragma unroll
  for (int i = 0; i < Tile::FA; ++i)
#pragma unroll
    for (int j = 0; j < Tile::FB; ++j) acc[i][j] = NtAcc<I8>::zero();
  Tile::run(g, lds, ia * TA, ib * TB, 0, (int)(g.kbytes / 64), acc);
  Tile::each(ia * TA, ib * TB, acc, [&](int64_t a, int64_t b, const typename Tile::acc_t(&v)[4]) {
    nt_store16<EP>(g, a, b, v, wide);
  });
}

template <bool I8, int EP, int TA, int TB, int WA, int WB, int RA, int RB, bool BT = false>
void launch_tiles(const NtArgs& g, const NtWide& wide, hipStream_t st) {
  const int64_t ta = ceil_div(g.na, TA), tb = ceil_div(g.nb, TB);
  nt_tile_kernel<I8, EP, TA, TB, WA, WB, RA, RB, BT>
      <<<(unsigned)(ceil_div(ta * tb, 8) * 8), 64 * WA * WB, 0, st>>>(g, wide, ta, tb);
}

// The tile: the largest one that still makes a workgroup for most CUs.  On
// 4096 x 4096 weights the integer product takes 11.3 us with 64x64, 15.6 us
// with 128x64 and 44 us with 256x256 tiles at 256 tokens, 16.6 / 16.7 / 44 us
// at 512, 52 / 44 / 50 us (256x128: 35 us) at 2048, and 124 us with 256x256
// against 135 us with 256x128 at 8192.
constexpr int64_t kFill = 160;

template <bool I8, int EP>
sg_status launch_nt(const NtArgs& g, const char* what, hipStream_t st) {
  const NtWide wide = nt_wide(g);
  auto tiles = [&](int64_t ta, int64_t tb) { return ceil_div(g.na, ta) * ceil_div(g.nb, tb); };
  if (g.nb > 64) {
    if (tiles(256, 256) >= kFill)
      launch_tiles<I8, EP, 256, 256, 2, 4, 3, 2>(g, wide, st);
    else if (tiles(256, 128) >= kFill)
      launch_tiles<I8, EP, 256, 128, 4, 2, 3, 3>(g, wide, st);
    else if (tiles(128, 64) >= kFill)
      launch_tiles<I8, EP, 128, 64, 2, 2, 3, 3>(g, wide, st);
    else
      launch_tiles<I8, EP, 64, 64, 1, 4, 4, 4>(g, wide, st);
    return check_launch(what);
  }
  const dim3 grid((unsigned)ceil_div(g.na, 16), (unsigned)ceil_div(g.nb, g.nb <= 16 ? 16 : 64));
  if (g.nb <= 16)
    nt_stream_kernel<I8, 1, EP><<<grid, 64 * kStreamWaves, 0, st>>>(g, wide.out4);
  else
    nt_stream_kernel<I8, 4, EP><<<grid, 64 * kStreamWaves, 0, st>>>(g, wide.out4);
  return check_launch(what);
}

// ---------------------------------------------------------------------------
// Operands of the gradients, in bf16 with the contraction along the rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float code_at(const u32x4& v, int e) {
  return (float)((int32_t)(v[e >> 2] << (24 - 8 * (e & 3))) >> 24);
}

// dst[c][r] = src[r][c] in bf16, c < C, r < Rp (Rp = R rounded up to 32
// elements, zero from R on).  CODES: src holds signed bytes in 64-byte padded
// rows that stand for scale[r] * (code + offset[r]) (offset NULL: 0); else
// bf16 rows of any pitch.
template <bool CODES>
__global__ __launch_bounds__(256) void transpose_bf16_kernel(uint16_t* __restrict__ dst, int64_t Rp,
                                                             const void* __restrict__ src, int64_t lds,
                                                             const float* __restrict__ scale,
                                                             const int32_t* __restrict__ offset, int64_t R,
                                                             int64_t C) {
  __shared__ uint16_t tile[64][72];  // [c][r]
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  const int tid = threadIdx.x;
  for (int64_t r0 = (int64_t)blockIdx.y * 64; r0 < Rp; r0 += (int64_t)gridDim.y * 64) {
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int64_t r = r0 + lr;
    if constexpr (CODES) {
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      float s = 0.0f, off = 0.0f;
      const bool live = r < R && c0 + lc < C;
      if (live) {
        v = *reinterpret_cast<const u32x4*>(static_cast<const int8_t*>(src) + r * lds + c0 + lc);
        s = scale[r];
        off = offset ? (float)offset[r] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) tile[lc + e][lr] = live ? (uint16_t)bf16_of(s * (code_at(v, e) + off)) : 0;
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(src) + r * lds + c0 + lc;
#pragma unroll
      for (int e = 0; e < 16; ++e) tile[lc + e][lr] = (r < R && c0 + lc + e < C) ? p[e] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int item = tid + 256 * k;
      const int c = item >> 3, rr = (item & 7) * 8;
      if (c0 + c < C && r0 + rr < Rp)
        *reinterpret_cast<u32x4*>(dst + (c0 + c) * Rp + r0 + rr) = *reinterpret_cast<const u32x4*>(&tile[c][rr]);
    }
    __syncthreads();
  }
}

// dst[t][k] = src[t][k] for k < K, 0 up to Kp.
__global__ __launch_bounds__(256) void pad_rows_kernel(uint16_t* __restrict__ dst, int64_t Kp,
                                                       const uint16_t* __restrict__ src, int64_t lds, int64_t T,
                                                       int64_t K) {
  const int64_t cpr = Kp / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < T * cpr; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / cpr, k0 = (i - t * cpr) * 8;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = k0 + 2 * e < K ? src[t * lds + k0 + 2 * e] : 0;
      const uint32_t hi = k0 + 2 * e + 1 < K ? src[t * lds + k0 + 2 * e + 1] : 0;
      w[e] = lo | (hi << 16);
    }
    *reinterpret_cast<u32x4*>(dst + t * Kp + k0) = u32x4{w[0], w[1], w[2], w[3]};
  }
}

void launch_pad_rows(uint16_t* dst, int64_t Kp, const uint16_t* src, int64_t lds, int64_t T, int64_t K, hipStream_t st) {
  const int64_t items = T * (Kp / 8);
  pad_rows_kernel<<<(unsigned)std::min<int64_t>(ceil_div(items, 256), 1 << 20), 256, 0, st>>>(dst, Kp, src, lds, T, K);
}

template <bool CODES>
void launch_transpose(uint16_t* dst, int64_t Rp, const void* src, int64_t lds, const float* scale,
                      const int32_t* offset, int64_t R, int64_t C, hipStream_t st) {
  const dim3 grid((unsigned)ceil_div(C, 64), (unsigned)std::min<int64_t>(ceil_div(Rp, 64), 65535));
  transpose_bf16_kernel<CODES><<<grid, 256, 0, st>>>(dst, Rp, src, lds, scale, offset, R, C);
}

size_t rows_bytes(int64_t rows, int64_t kp) { return (size_t)round_up(rows * kp * 2, 256); }

}  // namespace

size_t linear_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

sg_status launch_linear_w8a8(const LinearArgs& a, void*, hipStream_t st) {
  NtArgs g{};
  g.A = reinterpret_cast<const unsigned char*>(a.Wq);
  g.B = reinterpret_cast<const unsigned char*>(a.Q);
  g.lda = a.ldw;
  g.ldb = a.ldq;
  g.na = a.m;
  g.nb = a.T;
  g.kbytes = round_up(a.n, 64);
  g.out = a.Y;
  g.out_dtype = a.y_dtype;
  g.ldo = a.ldy;
  g.a_off = a.w_offset;
  g.a_scale = a.w_scale;
  g.b_scale = a.x_scale;
  g.b_sum = a.x_sum;
  return launch_nt<true, EP_LINEAR>(g, "sg_linear_w8a8", st);
}

// Workspace: the weights in bf16 [n x m_pad]; a padded copy of dY.
size_t grad_input_ws_bytes(int64_t m, int64_t n, int64_t T) {
  const int64_t mp = round_up(m, 32);
  return rows_bytes(n, mp) + rows_bytes(T, mp);
}

sg_status launch_grad_input(const GradInputArgs& a, void* ws, hipStream_t st) {
  const int64_t mp = round_up(a.m, 32);
  uint16_t* wt = static_cast<uint16_t*>(ws);
  launch_transpose<true>(wt, mp, a.Wq, a.ldw, a.w_scale, a.w_offset, a.m, a.n, st);
  const uint16_t* dy = a.dY;
  int64_t ldy = a.lddy;
  if (mp != a.m || a.lddy % 8 != 0 || reinterpret_cast<uintptr_t>(dy) % 16 != 0) {
    uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + rows_bytes(a.n, mp));
    launch_pad_rows(copy, mp, dy, ldy, a.T, a.m, st);
    dy = copy;
    ldy = mp;
  }
  NtArgs g{};
  g.A = reinterpret_cast<const unsigned char*>(wt);
  g.B = reinterpret_cast<const unsigned char*>(dy);
  g.lda = mp * 2;
  g.ldb = ldy * 2;
  g.na = a.n;
  g.nb = a.T;
  g.kbytes = mp * 2;
  g.out = a.dX;
  g.out_dtype = a.dx_dtype;
  g.ldo = a.lddx;
  return launch_nt<false, EP_PLAIN>(g, "sg_linear_w8_grad_input", st);
}

// Workspace: the checkpoint's tensor in bf16 with the tokens along the rows;
// a copy of dY whose rows can be read in 16-byte pieces.
size_t grad_weight_ws_bytes(int64_t m, int64_t n, int64_t T) {
  return rows_bytes(n, round_up(T, 32)) + rows_bytes(T, round_up(m, 8));
}

sg_status launch_grad_weight(const GradWeightArgs& a, void* ws, hipStream_t st) {
  const int64_t tp = round_up(a.T, 32), mp = round_up(a.m, 8);
  uint16_t* xt = static_cast<uint16_t*>(ws);
  const uint16_t* dy = a.dY;
  int64_t ldy = a.lddy;
  if (tp > 0) {
    launch_transpose<true>(xt, tp, a.Q, a.ldq, a.x_scale, nullptr, a.T, a.n, st);
    if (mp != a.m || ldy % 8 != 0 || reinterpret_cast<uintptr_t>(dy) % 16 != 0) {
      uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + rows_bytes(a.n, tp));
      launch_pad_rows(copy, mp, dy, ldy, a.T, a.m, st);
      dy = copy;
      ldy = mp;
    }
  }
  NtArgs g{};
  g.A = reinterpret_cast<const unsigned char*>(xt);
  g.B = reinterpret_cast<const unsigned char*>(dy);
  g.lda = tp * 2;
  g.ldb = ldy * 2;
  g.na = a.n;
  g.nb = a.m;
  g.kbytes = tp * 2;
  g.krows = a.T;
  g.bcols = mp;
  g.out = a.dW;
  g.out_dtype = a.dw_dtype;
  g.ldo = a.lddw;
  g.mask = a.mask;
  g.accumulate = a.accumulate;
  const NtWide wide = nt_wide(g);
  if (ceil_div(g.na, 256) * ceil_div(g.nb, 256) >= kFill)
    launch_tiles<false, EP_MASKED, 256, 256, 2, 4, 3, 2, true>(g, wide, st);
  else
    launch_tiles<false, EP_MASKED, 128, 128, 2, 2, 2, 2, true>(g, wide, st);
  return check_launch("sg_linear_w8_grad_weight");
}

}  // namespace sg
