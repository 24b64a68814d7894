// The 8-bit linear layer: its product in integers and its two gradients.
//
//   Y[t][r]  = x_scale[t] w_scale[r] sum_c q[t][c] (code[r][c] - zero[r])
//   dX[t][c] = sum_r dY[t][r] bf16(w_scale[r] (code[r][c] - zero[r]))
//   dW[r][c] = kept[r][c] sum_t dY[t][r] bf16(x_scale[t] q[t][c])
//
// With the zero point taken out, sum_c q (code - zero) = sum_c q (code - 128) +
// (128 - zero) sum_c q, the product is one of signed bytes: MFMA in integers,
// exact sums, one correction from the token's sum of codes.  The gradients are
// products of bf16 values (the codes' values rounded to bf16, as the definition
// has them) with fp32 sums.
//
// Every output is a sum over rows of A (the layer's or the checkpoint's codes)
// and rows of B (tokens, or output channels for dW); out[b][a] has a running
// fastest, so A's rows go to the MFMA's rows and a lane ends up with
// neighbouring outputs.
#include "gemm_codes.h"

#include <algorithm>

namespace sg {
namespace {

// Few rows of B: every workgroup takes 16 * CF rows of A and all of B's (16 *
// TF at most); its W waves divide the contraction and add their sums up in
// LDS, in wave order.  Operands go from memory straight to the registers that
// the MFMA reads, U steps ahead of their products.  A (the weights) is read
// once: bound by HBM.
template <bool I8, int EP, int CF, int TF, int W, int U>
__global__ __launch_bounds__(64 * W) void nt_stream_kernel(const NtArgs g, NtWide wide) {
  typedef typename NtAcc<I8>::type acc_t;
  __shared__ acc_t red[W][CF * TF][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t a0 = (int64_t)blockIdx.x * (16 * CF);
  const int steps = (int)(g.kbytes / 64);
  const int s0 = steps * wave / W, s1 = steps * (wave + 1) / W;
  // the outputs of this thread, if it has any: every (c, f) has 64 lanes' fours
  constexpr int ITEMS = 64 * CF * TF, PER = (ITEMS + 64 * W - 1) / (64 * W);
  auto column = [&](int i) { return a0 + 16 * ((i >> 6) / TF) + ((i & 63) >> 4) * 4; };
  auto token = [&](int i) { return (int64_t)(16 * ((i >> 6) % TF) + (i & 15)); };
  NtSide<EP, 4> side[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (tid + k * 64 * W < ITEMS) side[k].load(g, column(tid + k * 64 * W), token(tid + k * 64 * W), wide);
  // rows past the end re-read the last one; their sums are not stored
  const unsigned char *pa[CF], *pb[TF];
#pragma unroll
  for (int c = 0; c < CF; ++c)
    pa[c] = g.A + min<int64_t>(a0 + 16 * c + (lane & 15), g.na - 1) * g.lda + (lane >> 4) * 16 + (int64_t)s0 * 64;
#pragma unroll
  for (int f = 0; f < TF; ++f)
    pb[f] = g.B + min<int64_t>(16 * f + (lane & 15), g.nb - 1) * g.ldb + (lane >> 4) * 16 + (int64_t)s0 * 64;
  acc_t acc[CF][TF];
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int f = 0; f < TF; ++f) acc[c][f] = NtAcc<I8>::zero();
  u32x4 va[U][CF], vb[U][TF];
  auto load = [&](int u, int s) {
#pragma unroll
    for (int c = 0; c < CF; ++c) va[u][c] = *reinterpret_cast<const u32x4*>(pa[c] + (int64_t)s * 64);
#pragma unroll
    for (int f = 0; f < TF; ++f) vb[u][f] = *reinterpret_cast<const u32x4*>(pb[f] + (int64_t)s * 64);
  };
  auto multiply = [&](const u32x4 (&a)[CF], const u32x4 (&b)[TF]) {
#pragma unroll
    for (int c = 0; c < CF; ++c)
#pragma unroll
      for (int f = 0; f < TF; ++f) acc[c][f] = NtAcc<I8>::mma(a[c], b[f], acc[c][f]);
  };
  const int n = s1 - s0;
  int s = 0;
  if (n >= U) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, u);
    for (; s + 2 * U <= n; s += U) {
      u32x4 ca[U][CF], cb[U][TF];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int c = 0; c < CF; ++c) ca[u][c] = va[u][c];
#pragma unroll
        for (int f = 0; f < TF; ++f) cb[u][f] = vb[u][f];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) load(u, s + U + u);
#pragma unroll
      for (int u = 0; u < U; ++u) multiply(ca[u], cb[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(va[u], vb[u]);
    s += U;
  }
  const int rest = n - s;  // fewer than U
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (u < rest) load(u, s + u);
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (u < rest) multiply(va[u], vb[u]);
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int f = 0; f < TF; ++f) red[wave][c * TF + f][lane] = acc[c][f];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int i = tid + k * 64 * W;
    if (i >= ITEMS) break;
    acc_t v[1] = {red[0][i >> 6][i & 63]};
#pragma unroll
    for (int w = 1; w < W; ++w) v[0] += red[w][i >> 6][i & 63];
    nt_store<EP, 4>(g, column(i), token(i), v, wide, side[k]);
  }
}

template <bool I8, int EP, int TF>
void launch_stream(const NtArgs& g, const NtWide& wide, hipStream_t st) {
  // Measured with one token (16 for the first two), weights from HBM: 8192 x
  // 28672 bytes 44.8 us with two row fragments a wave and four waves against
  // 54.6 with one, 8192 x 8192 15.0 against 17.2; but 11008 x 4096 12.0
  // against 10.5, and 4096 x 4096 6.5 against 5.2 us: two fragments pay where
  // they still make a workgroup for every CU and the waves have long runs.
  // One fragment, four against eight waves: 11008 x 4096 10.5 / 11.0, 4096 x
  // 11008 12.5 / 11.2 us.
  constexpr int U = TF == 4 ? 2 : 4;
  if (g.na >= 32 * kNumCU && g.kbytes >= 8192)
    nt_stream_kernel<I8, EP, 2, TF, 4, U><<<(unsigned)ceil_div(g.na, 32), 256, 0, st>>>(g, wide);
  else if (g.na >= 32 * kNumCU)
    nt_stream_kernel<I8, EP, 1, TF, 4, 4><<<(unsigned)ceil_div(g.na, 16), 256, 0, st>>>(g, wide);
  else
    nt_stream_kernel<I8, EP, 1, TF, 8, 4><<<(unsigned)ceil_div(g.na, 16), 512, 0, st>>>(g, wide);
}

// panels of A whose tiles run together (large products: 4 to 8 within 2%, 16 up to 5% slower)
constexpr int kBand = 8;

// One tile a workgroup.  Large products are bound by the matrix cores and the
// power they draw: 8192 x 11008 outputs of 4096 products take 317 us in bytes
// (2.33 POP/s; the cores are busy 66-69% of the cycles at 2.0 GHz, and the clock
// falls when they are busier) and 505 us in bf16 over 11008 (1.46 PFLOP/s).
//
// Split: every tile's contraction is divided over `splits` workgroups, whose
// sums go to `part` (one 16-byte slot a fragment and thread); the join kernel
// adds them up in split order.
template <typename Tile, int EP, bool SPLIT>
__global__ __launch_bounds__(Tile::THREADS) void nt_tile_kernel(const NtArgs g, NtWide wide, int64_t ta, int64_t tb,
                                                                int splits, void* part) {
  typedef typename Tile::acc_t acc_t;
  __shared__ __attribute__((aligned(16))) unsigned char lds[Tile::LDS];
  int64_t k = nt_xcd_order(blockIdx.x, SPLIT ? ta * tb * splits : ta * tb);
  if (k < 0) return;
  const int steps = (int)(g.kbytes / 64);
  int s0 = 0, t1 = steps, split = 0;
  if constexpr (SPLIT) {
    const int stages = (steps + 1) / 2;
    split = (int)(k / (ta * tb));
    k -= split * (ta * tb);
    s0 = (int)((int64_t)stages * split / splits);
    t1 = min(steps, 2 * (int)((int64_t)stages * (split + 1) / splits));
  }
  int64_t ia, ib;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  constexpr bool kOne = Tile::GA * Tile::FB == 1;
  NtSide<EP, 16> side;
  if (kOne && !SPLIT && nt_aligned<EP>(g, wide))
    Tile::each(ia * Tile::TA, ib * Tile::TB, [&](int, int, int64_t a, int64_t b) { side.load(g, a, b, wide); });
  acc_t acc[Tile::FA][Tile::FB];
#pragma unroll
  for (int i = 0; i < Tile::FA; ++i)
#pragma unroll
    for (int j = 0; j < Tile::FB; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
  Tile::run(g, lds, ia * Tile::TA, ib * Tile::TB, s0, t1, acc);
  if constexpr (SPLIT) {
    acc_t* slot = static_cast<acc_t*>(part) +
                  ((k * splits + split) * (Tile::FA * Tile::FB)) * Tile::THREADS + threadIdx.x;
#pragma unroll
    for (int i = 0; i < Tile::FA; ++i)
#pragma unroll
      for (int j = 0; j < Tile::FB; ++j) slot[(i * Tile::FB + j) * Tile::THREADS] = acc[i][j];
  } else if (nt_aligned<EP>(g, wide)) {
    Tile::each(ia * Tile::TA, ib * Tile::TB, [&](int h, int j, int64_t a, int64_t b) {
      const acc_t v[4] = {acc[4 * h][j], acc[4 * h + 1][j], acc[4 * h + 2][j], acc[4 * h + 3][j]};
      if constexpr (!kOne) side.load(g, a, b, wide);
      nt_store<EP, 16>(g, a, b, v, wide, side);
    });
  } else {
    static_assert(Tile::LDS >= Tile::THREADS / 64 * kTurnBytes, "the stages' LDS turns the sums");
    __syncthreads();  // every wave is past its last read of the stages
    unsigned char* const turn = lds + (threadIdx.x >> 6) * kTurnBytes;
    const int lane = threadIdx.x & 63;
    Tile::each(ia * Tile::TA, ib * Tile::TB, [&](int h, int j, int64_t a, int64_t b) {
      const acc_t v[4] = {acc[4 * h][j], acc[4 * h + 1][j], acc[4 * h + 2][j], acc[4 * h + 3][j]};
      nt_store_rows<EP>(g, a - (lane >> 4) * 16, b - (lane & 15), v, turn);
    });
  }
}

// One workgroup per tile and (h, j): the sums of its splits, in their order.
template <typename Tile, int EP>
__global__ __launch_bounds__(Tile::THREADS) void nt_join_kernel(const NtArgs g, NtWide wide, int64_t ta, int64_t tb,
                                                                int splits, const void* part) {
  typedef typename Tile::acc_t acc_t;
  __shared__ __attribute__((aligned(16))) unsigned char turn[Tile::THREADS / 64 * kTurnBytes];
  const int64_t k = blockIdx.x;
  const int lane = threadIdx.x & 63;
  int64_t ia, ib;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  Tile::each(ia * Tile::TA, ib * Tile::TB, [&](int h, int j, int64_t a, int64_t b) {
    const int64_t wa0 = a - (lane >> 4) * 16, wb0 = b - (lane & 15);  // the wave's corner
    if (h * Tile::FB + j != (int)blockIdx.y || wb0 >= g.nb || wa0 >= g.na) return;
    acc_t v[4];
    for (int s = 0; s < splits; ++s) {
      const acc_t* slot = static_cast<const acc_t*>(part) +
                          ((k * splits + s) * (Tile::FA * Tile::FB)) * Tile::THREADS + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const acc_t w = slot[((4 * h + i) * Tile::FB + j) * Tile::THREADS];
        v[i] = s == 0 ? w : v[i] + w;
      }
    }
    if (nt_aligned<EP>(g, wide)) {
      NtSide<EP, 16> side;
      side.load(g, a, b, wide);
      nt_store<EP, 16>(g, a, b, v, wide, side);
    } else {
      nt_store_rows<EP>(g, wa0, wb0, v, turn + (threadIdx.x >> 6) * kTurnBytes);
    }
  });
}

// The tiles there are, largest first; the last three take A as codes.
enum { NT_256x256 = 0, NT_256x128, NT_128x64, NT_64x64, NT_CODES_128x128, NT_CODES_128x64, NT_CODES_64x64, NT_STREAM };
struct NtPlan {
  int tile;
  int splits;
  size_t ws_bytes;  // partial sums
  bool codes() const { return tile >= NT_CODES_128x128 && tile <= NT_CODES_64x64; }
};

struct NtTileCost {
  int ta, tb;
  int per_cu;     // workgroups that fit a CU
  double us[2];   // a 128-byte stage with one and with two workgroups on every CU
};
// Stages measured on layers of 4096 channels (MFMA alone would take 0.85 us a
// stage of a 256 x 256 tile at 2.4 GHz).  The constants below are common to all
// tiles, which flatters the largest: its first stages, output and launch take
// 12-15 us a round.  The estimate ranks tiles well where many rounds or many
// stages count; with few of both it can miss: 512 tokens' weight gradient at
// 4096 x 4096 is put at 17.6 us and takes 26.9.
constexpr NtTileCost kTiles[7] = {{256, 256, 1, {1.70, 0}},   {256, 128, 1, {0.93, 0}},   {128, 64, 2, {0.39, 0.60}},
                                  {64, 64, 2, {0.245, 0.41}}, {128, 128, 1, {0.86, 0}},   {128, 64, 1, {0.68, 0}},
                                  {64, 64, 2, {0.55, 0.80}}};
constexpr double kLaunch = 4.0;      // a tile's fill, epilogue and launch
constexpr double kRound = 2.0;       // a later round's fill and epilogue
constexpr double kJoin = 4.5;        // a second launch
constexpr double kJoinRate = 3.0e6;  // bytes of partial sums a microsecond, written and read

// The tile and the splits that should take the least time: rounds of
// workgroups, each for its share of the stages, plus the join; for the tiles
// [first, last).
NtPlan nt_plan(int64_t na, int64_t nb, int64_t kbytes, int first, int last, double* us_out = nullptr) {
  NtPlan p{first, 1, 0};
  const int64_t stages = std::max<int64_t>(1, ceil_div(kbytes, 128));
  double best = 1e300;
  for (int t = first; t < last; ++t) {
    const NtTileCost& c = kTiles[t];
    const int64_t tiles = ceil_div(na, c.ta) * ceil_div(nb, c.tb);
    for (int s = 1; s <= 16; s *= 2) {
      if (s > 1 && (stages / s < 8 || tiles * s > 2 * kNumCU)) break;
      const int64_t wgs = tiles * s;
      const bool one = c.per_cu == 1 || wgs <= kNumCU;
      const double rounds = (double)ceil_div(wgs, one ? kNumCU : 2 * kNumCU);
      double us = kLaunch + kRound * (rounds - 1) + rounds * (double)ceil_div(stages, s) * c.us[one ? 0 : 1];
      const size_t bytes = s > 1 ? (size_t)(wgs * c.ta * c.tb * 4) : 0;
      if (s > 1) us += kJoin + 2.0 * (double)bytes / kJoinRate;
      if (us < best * 0.999) {
        best = us;
        p = NtPlan{t, s, bytes};
      }
    }
  }
  if (us_out) *us_out = best;
  return p;
}

// A launch holds less than 2^32 threads; tiles have at most 512.
constexpr int64_t kMaxWorkgroups = (int64_t)1 << 22;

// The product of `rows` rows of B from b0 on (a multiple of 64).
template <typename Tile>
NtArgs nt_rows_of(const NtArgs& g, int64_t b0, int64_t rows) {
  NtArgs r = g;
  r.nb = rows;
  if (Tile::BT) {
    r.B += b0 * 2;
    r.bcols -= b0;
  } else {
    r.B += b0 * g.ldb;
  }
  r.out = static_cast<char*>(g.out) + b0 * g.ldo * (g.out_dtype == SG_F32 ? 4 : 2);
  if (g.b_scale) r.b_scale += b0;
  if (g.b_sum) r.b_sum += b0;
  if (g.mask) r.mask += b0 * g.na;
  return r;
}

template <typename Tile, int EP>
void launch_tiles(const NtArgs& g, const NtWide& wide, const NtPlan& p, void* part, hipStream_t st) {
  const int64_t ta = ceil_div(g.na, Tile::TA), tb = ceil_div(g.nb, Tile::TB);
  if (p.splits > 1) {  // (of few tiles)
    const unsigned grid = (unsigned)(ceil_div(ta * tb * p.splits, 8) * 8);
    nt_tile_kernel<Tile, EP, true><<<grid, Tile::THREADS, 0, st>>>(g, wide, ta, tb, p.splits, part);
    nt_join_kernel<Tile, EP><<<dim3((unsigned)(ta * tb), Tile::GA * Tile::FB), Tile::THREADS, 0, st>>>(
        g, wide, ta, tb, p.splits, part);
    return;
  }
  const int64_t most = kMaxWorkgroups / ta;  // panels of B in a launch
  for (int64_t b = 0; b < tb; b += most) {
    const int64_t n = std::min(most, tb - b), b0 = b * Tile::TB;
    const unsigned grid = (unsigned)(ceil_div(ta * n, 8) * 8);
    nt_tile_kernel<Tile, EP, false><<<grid, Tile::THREADS, 0, st>>>(
        nt_rows_of<Tile>(g, b0, std::min<int64_t>(g.nb - b0, n * Tile::TB)), wide, ta, n, 1, nullptr);
  }
}

// The gradients' products: A in bf16 rows, or (plans of code tiles) as codes.
template <int EP, bool BT>
sg_status launch_grad(const NtArgs& g, const NtPlan& p, void* part, const char* what, hipStream_t st) {
  constexpr bool OFFSET = !BT;  // weights have zero points, tokens have none
  const NtWide wide = nt_wide(g);
  switch (p.tile) {
    case NT_256x256: launch_tiles<NtTile<false, 256, 256, 2, 4, 3, 2, BT>, EP>(g, wide, p, part, st); break;
    case NT_256x128: launch_tiles<NtTile<false, 256, 128, 4, 2, 3, 3, BT>, EP>(g, wide, p, part, st); break;
    case NT_128x64: launch_tiles<NtTile<false, 128, 64, 2, 4, 3, 3, BT>, EP>(g, wide, p, part, st); break;
    case NT_64x64: launch_tiles<NtTile<false, 64, 64, 1, 4, 4, 4, BT>, EP>(g, wide, p, part, st); break;
    case NT_CODES_128x128: launch_tiles<CodeTile<128, 128, 2, 4, 4, BT, OFFSET>, EP>(g, wide, p, part, st); break;
    case NT_CODES_128x64: launch_tiles<CodeTile<128, 64, 2, 4, 4, BT, OFFSET>, EP>(g, wide, p, part, st); break;
    default: launch_tiles<CodeTile<64, 64, 1, 4, 4, BT, OFFSET>, EP>(g, wide, p, part, st);
  }
  return check_launch(what);
}

// ---------------------------------------------------------------------------
// Operands of the gradients, in bf16 with the contraction along the rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ float code_at(const u32x4& v, int e) {
  return (float)((int32_t)(v[e >> 2] << (24 - 8 * (e & 3))) >> 24);
}

// Rows copied to where they can be read in 16-byte pieces, zero-padded.
struct PadRows {
  uint16_t* dst;  // [rows x pitch], pitch a multiple of 8
  int64_t pitch;
  const uint16_t* src;  // [rows x cols], any pitch and alignment; NULL: nothing to copy
  int64_t lds, rows, cols;
};

// wt[c][r] = bf16(scale[r] * (codes[r][c] + offset[r])) for c < C and r < Rp,
// 0 for r >= R: signed bytes in 64-byte padded rows turned to bf16 with the
// other index running (offset NULL: 0).  The first workgroups do this in tiles
// of 64 x 64 through LDS, the others copy the rows of `pad`.  Bound by HBM: 3
// bytes a code, 11008 x 4096 in 30 us (4.5 TB/s).
__global__ __launch_bounds__(256) void operands_kernel(uint16_t* __restrict__ wt, int64_t Rp,
                                                       const int8_t* __restrict__ codes, int64_t ldc,
                                                       const float* __restrict__ scale,
                                                       const int32_t* __restrict__ offset, int64_t R, int64_t C,
                                                       int64_t tblocks, const PadRows pad) {
  __shared__ uint16_t tile[64][72];  // [c][r]
  const int tid = threadIdx.x;
  if (blockIdx.x >= tblocks) {
    const int64_t cpr = pad.pitch / 8;
    const int64_t stride = (gridDim.x - tblocks) * 256;
    for (int64_t i = (blockIdx.x - tblocks) * 256 + tid; i < pad.rows * cpr; i += stride) {
      const int64_t t = i / cpr, k0 = (i - t * cpr) * 8;
      const uint16_t* p = pad.src + t * pad.lds + k0;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = k0 + 2 * e < pad.cols ? p[2 * e] : 0;
        const uint32_t hi = k0 + 2 * e + 1 < pad.cols ? p[2 * e + 1] : 0;
        w[e] = lo | (hi << 16);
      }
      *reinterpret_cast<u32x4*>(pad.dst + t * pad.pitch + k0) = u32x4{w[0], w[1], w[2], w[3]};
    }
    return;
  }
  const int64_t tc = (C + 63) / 64, tr = (Rp + 63) / 64;
  for (int64_t i = blockIdx.x; i < tc * tr; i += tblocks) {
    const int64_t r0 = i / tc * 64, c0 = i % tc * 64;
    const int lr = tid >> 2, lc = (tid & 3) * 16;
    const int64_t r = r0 + lr;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    float s = 0.0f, off = 0.0f;
    const bool live = r < R && c0 + lc < C;
    if (live) {
      v = *reinterpret_cast<const u32x4*>(codes + r * ldc + c0 + lc);
      s = scale[r];
      off = offset ? (float)offset[r] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) tile[lc + e][lr] = live ? (uint16_t)bf16_of(s * (code_at(v, e) + off)) : 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int item = tid + 256 * k;
      const int c = item >> 3, rr = (item & 7) * 8;
      if (c0 + c < C && r0 + rr < Rp)
        *reinterpret_cast<u32x4*>(wt + (c0 + c) * Rp + r0 + rr) = *reinterpret_cast<const u32x4*>(&tile[c][rr]);
    }
    __syncthreads();
  }
}

void launch_operands(uint16_t* wt, int64_t Rp, const int8_t* codes, int64_t ldc, const float* scale,
                     const int32_t* offset, int64_t R, int64_t C, const PadRows& pad, hipStream_t st) {
  const int64_t tblocks = std::min<int64_t>(ceil_div(C, 64) * ceil_div(Rp, 64), 1 << 20);
  const int64_t pblocks = pad.src ? std::min<int64_t>(ceil_div(pad.rows * (pad.pitch / 8), 256), 1 << 16) : 0;
  operands_kernel<<<(unsigned)(tblocks + pblocks), 256, 0, st>>>(wt, Rp, codes, ldc, scale, offset, R, C, tblocks, pad);
}

size_t rows_bytes(int64_t rows, int64_t kp) { return (size_t)round_up(rows * kp * 2, 256); }


// Few tokens stream the weights; what few are was measured: 4096 x 4096
// weights with 32 tokens take 8.9 us streamed and 10.1 us in 64x64 tiles, with
// 64 tokens 12.5 and 10.2; 11008 x 4096 with 32 tokens 19.7 and 11.0 (enough
// tiles for most CUs); 1000 x 1000 with 64 tokens 5.3 and 6.0.  With 17 to 32
// tokens the border of 160 tiles lies between the two measured layers (64 and
// 172 tiles); where between them was not measured.
NtPlan linear_plan(int64_t m, int64_t n, int64_t T) {
  const int64_t kbytes = round_up(n, 64);
  if (T <= 16 || (T <= 32 && ceil_div(m, 64) < 160) || (T <= 64 && m * kbytes <= (4 << 20)))
    return NtPlan{NT_STREAM, 1, 0};
  return nt_plan(m, T, kbytes, NT_256x256, NT_CODES_128x128);
}

// A gradient whose A is na columns of codes over kr contraction rows: either
// turned to bf16 rows by a launch of its own (0.6 us a million codes), or by
// code tiles, once for every tile.  The bf16 rows are as long as the
// contraction, and a row's offset from its tile's corner is kept in 32 bits:
// past 2^23 tokens (255 rows of 2^24 bytes) the weight gradient is left to code
// tiles, whose rows are the caller's.  8.5 million tokens of 512 x 1024 weights
// take 14.3 ms so; 128-row tiles, whose offsets would still fit, took 28.8.
constexpr int64_t kMaxRowBytes = (int64_t)1 << 24;
NtPlan grad_plan(int64_t na, int64_t nb, int64_t kr) {
  double rows_us, codes_us;
  const int64_t kbytes = round_up(kr, 32) * 2;
  const NtPlan codes = nt_plan(na, nb, kbytes, NT_CODES_128x128, NT_STREAM, &codes_us);
  if (kbytes > kMaxRowBytes) return codes;
  const NtPlan rows = nt_plan(na, nb, kbytes, NT_256x256, NT_CODES_128x128, &rows_us);
  return rows_us + 3.0 + 0.62e-6 * (double)(na * kr) < codes_us ? rows : codes;
}

}  // namespace

// Workspace: the partial sums of split tiles.
size_t linear_ws_bytes(int64_t m, int64_t n, int64_t T) { return T > 0 ? linear_plan(m, n, T).ws_bytes : 0; }

sg_status launch_linear_w8a8(const LinearArgs& a, void* ws, hipStream_t st) {
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
  const NtWide wide = nt_wide(g);
  const NtPlan p = linear_plan(a.m, a.n, a.T);
  switch (p.tile) {
    case NT_256x256: launch_tiles<NtTile<true, 256, 256, 2, 4, 3, 2>, EP_LINEAR>(g, wide, p, ws, st); break;
    case NT_256x128: launch_tiles<NtTile<true, 256, 128, 4, 2, 3, 3>, EP_LINEAR>(g, wide, p, ws, st); break;
    case NT_128x64: launch_tiles<NtTile<true, 128, 64, 2, 4, 3, 3>, EP_LINEAR>(g, wide, p, ws, st); break;
    case NT_64x64: launch_tiles<NtTile<true, 64, 64, 1, 4, 4, 4>, EP_LINEAR>(g, wide, p, ws, st); break;
    default:
      if (a.T <= 16)
        launch_stream<true, EP_LINEAR, 1>(g, wide, st);
      else if (a.T <= 32)
        launch_stream<true, EP_LINEAR, 2>(g, wide, st);
      else
        launch_stream<true, EP_LINEAR, 4>(g, wide, st);
  }
  return check_launch("sg_linear_w8a8");
}

// Workspace: a copy of dY whose rows can be read in 16-byte pieces with the
// contraction padded to 64 bytes; partial sums; the weights in bf16 [n x m_pad]
// unless the plan takes codes.
size_t grad_input_ws_bytes(int64_t m, int64_t n, int64_t T) {
  if (T == 0) return 0;
  const int64_t mp = round_up(m, 32);
  const NtPlan p = grad_plan(n, T, m);
  return rows_bytes(T, mp) + p.ws_bytes + (p.codes() ? 0 : rows_bytes(n, mp));
}

sg_status launch_grad_input(const GradInputArgs& a, void* ws, hipStream_t st) {
  const int64_t mp = round_up(a.m, 32);
  const NtPlan p = grad_plan(a.n, a.T, a.m);
  char* const part = static_cast<char*>(ws) + rows_bytes(a.T, mp);
  uint16_t* const wt = reinterpret_cast<uint16_t*>(part + p.ws_bytes);
  const uint16_t* dy = a.dY;
  int64_t ldy = a.lddy;
  PadRows pad{};
  if (mp != a.m || ldy % 8 != 0 || reinterpret_cast<uintptr_t>(dy) % 16 != 0) {
    pad = PadRows{static_cast<uint16_t*>(ws), mp, dy, ldy, a.T, a.m};
    dy = pad.dst;
    ldy = mp;
  }
  if (!p.codes() || pad.src)
    launch_operands(wt, mp, a.Wq, a.ldw, a.w_scale, a.w_offset, a.m, p.codes() ? 0 : a.n, pad, st);
  NtArgs g{};
  if (p.codes()) {
    g.A = reinterpret_cast<const unsigned char*>(a.Wq);
    g.lda = a.ldw;
    g.krows = a.m;
    g.k_scale = a.w_scale;
    g.k_off = a.w_offset;
  } else {
    g.A = reinterpret_cast<const unsigned char*>(wt);
    g.lda = mp * 2;
  }
  g.B = reinterpret_cast<const unsigned char*>(dy);
  g.ldb = ldy * 2;
  g.na = a.n;
  g.nb = a.T;
  g.kbytes = mp * 2;
  g.out = a.dX;
  g.out_dtype = a.dx_dtype;
  g.ldo = a.lddx;
  return launch_grad<EP_PLAIN, false>(g, p, part, "sg_linear_w8_grad_input", st);
}

// Workspace: a copy of dY whose rows can be read in 16-byte pieces; partial
// sums; the checkpoint's tensor in bf16 with the tokens along the rows unless
// the plan takes codes.
size_t grad_weight_ws_bytes(int64_t m, int64_t n, int64_t T) {
  if (T == 0) return 0;
  const NtPlan p = grad_plan(n, m, T);
  return rows_bytes(T, round_up(m, 8)) + p.ws_bytes + (p.codes() ? 0 : rows_bytes(n, round_up(T, 32)));
}

sg_status launch_grad_weight(const GradWeightArgs& a, void* ws, hipStream_t st) {
  const int64_t tp = round_up(a.T, 32), mp = round_up(a.m, 8);
  // (no tokens: the tiles take no stage and write zeros)
  const NtPlan p = a.T > 0 ? grad_plan(a.n, a.m, a.T) : NtPlan{NT_64x64, 1, 0};
  char* const part = static_cast<char*>(ws) + rows_bytes(a.T, mp);
  uint16_t* const xt = reinterpret_cast<uint16_t*>(part + p.ws_bytes);
  const uint16_t* dy = a.dY;
  int64_t ldy = a.lddy;
  if (a.T > 0) {
    PadRows pad{};
    if (mp != a.m || ldy % 8 != 0 || reinterpret_cast<uintptr_t>(dy) % 16 != 0) {
      pad = PadRows{static_cast<uint16_t*>(ws), mp, dy, ldy, a.T, a.m};
      dy = pad.dst;
      ldy = mp;
    }
    if (!p.codes() || pad.src)
      launch_operands(xt, tp, a.Q, a.ldq, a.x_scale, nullptr, a.T, p.codes() ? 0 : a.n, pad, st);
  }
  NtArgs g{};
  if (p.codes()) {
    g.A = reinterpret_cast<const unsigned char*>(a.Q);
    g.lda = a.ldq;
    g.k_scale = a.x_scale;
  } else {
    g.A = reinterpret_cast<const unsigned char*>(xt);
    g.lda = tp * 2;
  }
  g.B = reinterpret_cast<const unsigned char*>(dy);
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
  return launch_grad<EP_MASKED, true>(g, p, part, "sg_linear_w8_grad_weight", st);
}

}  // namespace sg
