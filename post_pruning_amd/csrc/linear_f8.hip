// The linear layer in 8-bit floating point: its product and its two gradients,
// one product of two matrices with other operands each.
//
//   Y[t][r]  = sum_c x^[t][c] w^[r][c]            A = weights            B = tokens
//   dX[t][c] = drop(sum_r dy^[t][r] w^[r][c])     A = weights, transposed  B = gradients
//   dW[r][c] = kept[r][c] sum_t dy^[t][r] x^[t][c]  A = inputs, transposed   B = gradients, transposed
//
// where v^ = code 2^e with an e for every 128 of the contraction.
#include "gemm_f8.h"

#include <algorithm>

namespace sg {
namespace {

// Few rows of B: every workgroup takes 16 CF rows of A and all of B's (16 TF at
// most); its W waves divide the contraction and add their sums up in LDS, in wave
// order.  Operands go from memory straight to registers, U blocks of 128 ahead of
// their products.  A (the weights) is read once: bound by HBM (8192 x 28672 with 16
// tokens 47 us, 5.0 TB/s); a layer that the caches hold, by the chain of one wave's
// loads and the join (4096 x 4096, one token, 5 us).
template <bool WIDE, bool E5, int CF, int TF, int W, int U>
__global__ __launch_bounds__(64 * W) void f8_stream_kernel(const F8Args p, NtWide wide) {
  __shared__ floatx4 red[W][CF * TF][64];
  const NtArgs& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t a0 = (int64_t)blockIdx.x * (16 * CF);
  const int steps = (int)(g.kbytes / 128);
  const int s0 = (int)((int64_t)steps * wave / W), n = (int)((int64_t)steps * (wave + 1) / W) - s0;
  // rows past the end re-read the last one; their sums are not stored
  const unsigned char *pa[CF], *pb[TF];
  const uint8_t *qa[CF], *qb[TF];
#pragma unroll
  for (int c = 0; c < CF; ++c) {
    pa[c] = g.A + min<int64_t>(a0 + 16 * c + (lane & 15), g.na - 1) * g.lda + (lane >> 4) * 16 + (int64_t)s0 * 128;
    qa[c] = p.a_scale + s0 * p.a_lds + min<int64_t>(a0 + 16 * c + (lane & 15), g.na - 1);
  }
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    const int64_t r = min<int64_t>(16 * f + (lane & 15), g.nb - 1);
    pb[f] = g.B + r * g.ldb + (lane >> 4) * 16 + (int64_t)s0 * 128;
    qb[f] = p.b_scale + s0 * p.b_lds + r;
  }
  floatx4 acc[CF][TF];
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int f = 0; f < TF; ++f) acc[c][f] = floatx4{0.f, 0.f, 0.f, 0.f};
  struct Block {
    f8_frag a[CF], b[TF];
    uint32_t ea[CF], eb[TF];
  };
  auto frag = [](const unsigned char* q) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(q), hi = *reinterpret_cast<const u32x4*>(q + 64);
    return f8_frag{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto load = [&](Block& v, int s) {
#pragma unroll
    for (int c = 0; c < CF; ++c) {
      v.a[c] = frag(pa[c] + (int64_t)s * 128);
      v.ea[c] = qa[c][s * p.a_lds];
    }
#pragma unroll
    for (int f = 0; f < TF; ++f) {
      v.b[f] = frag(pb[f] + (int64_t)s * 128);
      v.eb[f] = qb[f][s * p.b_lds];
    }
  };
  auto multiply = [&](const Block& v) {
    if constexpr (WIDE) {
      F8Wide wb[TF];
#pragma unroll
      for (int f = 0; f < TF; ++f) wb[f] = f8_widen<E5>(v.b[f], f8_scale_float<0>(v.eb[f]));
#pragma unroll
      for (int c = 0; c < CF; ++c)
        f8_dot_wide<TF>(f8_widen<false>(v.a[c], f8_scale_float<0>(v.ea[c])), wb, acc[c]);
    } else {
#pragma unroll
      for (int c = 0; c < CF; ++c)
#pragma unroll
        for (int f = 0; f < TF; ++f)
          acc[c][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v.a[c], v.b[f], acc[c][f], 0, E5 ? 1 : 0, 0,
                                                                       (int)v.ea[c], 0, (int)v.eb[f]);
    }
  };
  Block v[U];
  int s = 0;
  if (n >= U) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(v[u], u);
    for (; s + 2 * U <= n; s += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Block now = v[u];
        load(v[u], s + U + u);
        multiply(now);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(v[u]);
    s += U;
  }
  const int rest = n - s;  // fewer than U
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (u < rest) load(v[u], s + u);
#pragma unroll
  for (int u = 0; u < U - 1; ++u)
    if (u < rest) multiply(v[u]);
#pragma unroll
  for (int c = 0; c < CF; ++c)
#pragma unroll
    for (int f = 0; f < TF; ++f) red[wave][c * TF + f][lane] = acc[c][f];
  __syncthreads();
  const DropKey key = p.has_drop ? drop_key(p.drop) : DropKey{};
  for (int i = tid; i < 64 * CF * TF; i += 64 * W) {
    floatx4 o[1] = {red[0][i >> 6][i & 63]};
#pragma unroll
    for (int w = 1; w < W; ++w) o[0] += red[w][i >> 6][i & 63];
    const int64_t a = a0 + 16 * ((i >> 6) / TF) + ((i & 63) >> 4) * 4, b = 16 * ((i >> 6) % TF) + (i & 15);
    if (p.has_drop) f8_drop<4>(p, key, a, b, o);
    NtSide<EP_MASKED, 4> side;
    side.load(g, a, b, wide);
    nt_store<EP_MASKED, 4>(g, a, b, o, wide, side);
  }
}

template <bool WIDE, bool E5, int TF>
void launch_stream(const F8Args& p, hipStream_t st) {
  // Measured (bf16, weights from HBM), two row fragments and four waves / one and
  // four / one and eight: 8192 rows x 28672 with 16 tokens 48.5 / 63.4 / 62.0 us, with one 43.3 /
  // 46.7 / 43.8; 11008 x 4096 with one - / 12.0 / 14.4; 4096 x 4096 with one 7.8 / 7.1 / 7.3.
  const NtWide wide = nt_wide(p.g);
  constexpr int U = TF == 4 ? 2 : 4;
  const unsigned ga = (unsigned)ceil_div(p.g.na, 16);
  if (p.g.na >= 32 * kNumCU && p.g.kbytes >= 8192)
    f8_stream_kernel<WIDE, E5, 2, TF, 4, U><<<(ga + 1) / 2, 256, 0, st>>>(p, wide);
  else if (p.g.na >= 32 * kNumCU)
    f8_stream_kernel<WIDE, E5, 1, TF, 4, U><<<ga, 256, 0, st>>>(p, wide);
  else
    f8_stream_kernel<WIDE, E5, 1, TF, 8, U><<<ga, 512, 0, st>>>(p, wide);
}
template <bool E5, int TF>
void launch_stream(const F8Args& p, hipStream_t st) {
  if (p.g.out_dtype == SG_F32)
    launch_stream<true, E5, TF>(p, st);
  else
    launch_stream<false, E5, TF>(p, st);
}

// The product of `rows` rows of B from b0 on.
F8Args f8_rows_of(const F8Args& p, int64_t b0, int64_t rows) {
  F8Args r = p;
  r.g.nb = rows;
  r.g.B += b0 * p.g.ldb;
  r.b_scale += b0;
  r.g.out = static_cast<char*>(p.g.out) + b0 * p.g.ldo * (p.g.out_dtype == SG_F32 ? 4 : 2);
  if (p.g.mask) r.g.mask += b0 * p.g.na;
  r.row0 += b0;
  return r;
}

// Panels of A whose tiles run together.  8192 rows x 11008 x 4096 and 8192 x 4096 x 11008
// with 4, 8 and 16 (us): 272, 268 and 273; 320, 317 and 324.
constexpr int kBand = 8;

// One tile a workgroup (what bounds them: F8Tile).  Split: every tile's contraction is divided over `splits`
// workgroups, whose sums go to `part` (one 16-byte slot a fragment and thread);
// the join kernel adds them up in split order.
template <typename Tile, bool SPLIT>
__global__ __launch_bounds__(Tile::THREADS) void f8_tiles_kernel(const F8Args p, int64_t ta, int64_t tb,
                                                                 int splits, floatx4* part) {
  __shared__ __attribute__((aligned(16))) unsigned char lds[Tile::LDS];
  int64_t k = nt_xcd_order(blockIdx.x, SPLIT ? ta * tb * splits : ta * tb);
  if (k < 0) return;
  const int steps = (int)(p.g.kbytes / 128);
  int s0 = 0, s1 = steps, split = 0;
  if constexpr (SPLIT) {
    split = (int)(k / (ta * tb));
    k -= split * (ta * tb);
    s0 = (int)((int64_t)steps * split / splits);
    s1 = (int)((int64_t)steps * (split + 1) / splits);
  }
  int64_t ia, ib;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  floatx4 acc[Tile::FA][Tile::FB];
#pragma unroll
  for (int i = 0; i < Tile::FA; ++i)
#pragma unroll
    for (int j = 0; j < Tile::FB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  {
    const Tile tile(p, lds, ia * Tile::TA, ib * Tile::TB, s0, s1 - s0);
    tile.run(acc);
  }
  if constexpr (SPLIT) {
    floatx4* slot = part + ((k * splits + split) * (Tile::FA * Tile::FB)) * Tile::THREADS + threadIdx.x;
#pragma unroll
    for (int i = 0; i < Tile::FA; ++i)
#pragma unroll
      for (int j = 0; j < Tile::FB; ++j) slot[(i * Tile::FB + j) * Tile::THREADS] = acc[i][j];
    return;
  }
  F8Kept<Tile> kept;
  if (p.has_drop) kept.make(p, drop_key(p.drop), ia * Tile::TA, ib * Tile::TB);
  Tile::template each<Tile::ITEMS>([&](auto iq) {
    constexpr int q = decltype(iq)::value, h = q / Tile::FB, j = q % Tile::FB;
    int64_t a, b;
    Tile::item(ia * Tile::TA, ib * Tile::TB, q, a, b);
    floatx4 v[4] = {acc[4 * h][j], acc[4 * h + 1][j], acc[4 * h + 2][j], acc[4 * h + 3][j]};
    if (p.has_drop) f8_drop16(p, kept.of(q), v);
    f8_store16(p.g, a, b, v);
  });
}

// One workgroup per tile and item: the sums of its splits, in their order.
template <typename Tile>
__global__ __launch_bounds__(Tile::THREADS) void f8_join_kernel(const F8Args p, int64_t ta, int64_t tb,
                                                                int splits, const floatx4* part) {
  const int64_t k = blockIdx.x;
  const int q = (int)blockIdx.y, h = q / Tile::FB, j = q % Tile::FB;
  int64_t ia, ib, a, b;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  Tile::item(ia * Tile::TA, ib * Tile::TB, q, a, b);
  if (a >= p.g.na) return;  // (whole quads)
  floatx4 v[4];
  for (int s = 0; s < splits; ++s) {
    const floatx4* slot = part + ((k * splits + s) * (Tile::FA * Tile::FB)) * Tile::THREADS + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const floatx4 w = slot[((4 * h + i) * Tile::FB + j) * Tile::THREADS];
      v[i] = s == 0 ? w : v[i] + w;
    }
  }
  if (p.has_drop) f8_drop16(p, f8_kept16(p, drop_key(p.drop), a, b), v);
  f8_store16(p.g, a, b, v);
}

// The tiles there are, largest first: those of the matrix instruction for 8-bit
// floating point, then those of widened codes.
enum { F8_256x256 = 0, F8_256x128, F8_128x128, F8_64x64, F8_WIDE_256x128, F8_WIDE_128x128, F8_WIDE_64x64, F8_STREAM };
struct F8Plan {
  int tile;
  int splits;
  size_t ws_bytes;  // partial sums
};

struct F8TileCost {
  int ta, tb;
  int per_cu;        // workgroups that fit a CU
  double base;       // launch, first stages and output
  double few, full;  // a stage with few workgroups, and with all of a round
};
// Microseconds, measured at 8, 32 and 86 stages with 64 to 8192 rows of B (the
// products of a stage of 256 x 256 alone take 0.85 at 2.4 GHz).
constexpr F8TileCost kTiles[7] = {{256, 256, 1, 8.0, 1.10, 1.45}, {256, 128, 1, 6.0, 0.60, 0.90},
                                  {128, 128, 1, 5.0, 0.38, 0.52}, {64, 64, 2, 4.3, 0.28, 0.42},
                                  {256, 128, 1, 6.5, 1.28, 1.75}, {128, 128, 1, 5.0, 0.78, 1.08},
                                  {64, 64, 2, 4.3, 0.46, 0.76}};
constexpr double kJoin = 4.0;        // a second launch
constexpr double kJoinRate = 5.0e6;  // bytes of partial sums a microsecond, written and read

// The tile and the splits that should take the least time: rounds of
// workgroups, each for its share of the stages, plus the join.
//
// Few rows of B stream A, measured against the best of the tiles (bf16, us): 4096 x
// 4096 with 32 rows 9.2 and 11.8, 11008 x 4096 20.2 and 13.2 (enough tiles for most
// CUs), 4096 x 11008 18.3 and 17.0; with 64 rows 2048 x 2048 7.8 and 8.2, 4096 x 4096
// 12.2 and 12.1.
//
// A wave of the stream takes its share of the contraction alone, 0.6 (one row of B) to
// 2.2 us (64 rows) for 128 of each wave; where A's rows do not fill the CUs, split tiles
// divide a long one further.  Stream and split tiles (bf16, us), contraction in brackets:
// 64 rows of A by 16 of B 10.5 and 13.5 (8192), 17.8 and 14.0 (16384), 31.8 and 16.3
// (32768), 117 and 29 (131072); 2048 by 16 17.7 and 18.4 (16384), 34 and 26 (32768); 64 by
// 17 11.7 and 13.3 (8192), 20.1 and 14.4 (16384); 64 by 64 12.4 and 11.5 (4096), 21.9 and 13.9
// (8192), 285 and 29 (131072).
F8Plan f8_plan(int64_t na, int64_t nb, int64_t k, bool wide) {
  if ((nb <= 16 && (na >= 16 * kNumCU || k <= 16384)) || (nb <= 32 && na * k <= (16 << 20) && k <= 16384) ||
      (nb <= 64 && na * k <= (4 << 20) && k <= 4096))
    return F8Plan{F8_STREAM, 1, 0};
  const int first = wide ? F8_WIDE_256x128 : F8_256x256, last = wide ? F8_STREAM : F8_WIDE_256x128;
  F8Plan p{first, 1, 0};
  const int64_t stages = std::max<int64_t>(1, ceil_div(k, 128));
  double best = 1e300;
  for (int t = first; t < last; ++t) {
    const F8TileCost& c = kTiles[t];
    const int64_t tiles = ceil_div(na, c.ta) * ceil_div(nb, c.tb), most = (int64_t)kNumCU * c.per_cu;
    for (int s = 1; s <= 16; s *= 2) {
      if (s > 1 && (stages / s < 4 || tiles * s > 2 * kNumCU)) break;
      const int64_t wgs = tiles * s, rounds = ceil_div(wgs, most);
      // how full the rounds are
      const double load = (double)wgs / (double)(rounds * most);
      const double stage = c.few + (c.full - c.few) * load;
      double us = c.base * (1.0 + 0.7 * (double)(rounds - 1)) + (double)(rounds * ceil_div(stages, s)) * stage;
      const size_t bytes = s > 1 ? (size_t)(wgs * c.ta * c.tb * 4) : 0;
      if (s > 1) us += kJoin + 2.0 * (double)bytes / kJoinRate;
      if (us < best * 0.999) {
        best = us;
        p = F8Plan{t, s, bytes};
      }
    }
  }
  return p;
}

// A launch holds less than 2^32 threads; workgroups have at most 512.
constexpr int64_t kMaxWorkgroups = (int64_t)1 << 22;

template <typename Tile>
void launch_tiles(const F8Args& p, const F8Plan& plan, void* ws, hipStream_t st) {
  const int64_t ta = ceil_div(p.g.na, Tile::TA), tb = ceil_div(p.g.nb, Tile::TB);
  if (plan.splits > 1) {  // (of few tiles)
    floatx4* const part = static_cast<floatx4*>(ws);
    const unsigned grid = (unsigned)(ceil_div(ta * tb * plan.splits, 8) * 8);
    f8_tiles_kernel<Tile, true><<<grid, Tile::THREADS, 0, st>>>(p, ta, tb, plan.splits, part);
    f8_join_kernel<Tile><<<dim3((unsigned)(ta * tb), Tile::ITEMS), Tile::THREADS, 0, st>>>(p, ta, tb, plan.splits, part);
    return;
  }
  const int64_t most = kMaxWorkgroups / ta;  // panels of B in a launch
  for (int64_t b = 0; b < tb; b += most) {
    const int64_t n = std::min(most, tb - b), b0 = b * Tile::TB;
    const unsigned grid = (unsigned)(ceil_div(ta * n, 8) * 8);
    f8_tiles_kernel<Tile, false><<<grid, Tile::THREADS, 0, st>>>(
        f8_rows_of(p, b0, std::min<int64_t>(p.g.nb - b0, n * Tile::TB)), ta, n, 1, nullptr);
  }
}

template <bool E5>
void launch_f8_t(const F8Args& p, const F8Plan& plan, void* ws, hipStream_t st) {
  switch (plan.tile) {
    case F8_256x256: launch_tiles<F8Tile<false, E5, 256, 256, 2, 4, 2>>(p, plan, ws, st); break;
    case F8_256x128: launch_tiles<F8Tile<false, E5, 256, 128, 4, 2, 3>>(p, plan, ws, st); break;
    case F8_128x128: launch_tiles<F8Tile<false, E5, 128, 128, 2, 4, 4>>(p, plan, ws, st); break;
    case F8_64x64: launch_tiles<F8Tile<false, E5, 64, 64, 1, 4, 4>>(p, plan, ws, st); break;
    case F8_WIDE_256x128: launch_tiles<F8Tile<true, E5, 256, 128, 4, 2, 3>>(p, plan, ws, st); break;
    case F8_WIDE_128x128: launch_tiles<F8Tile<true, E5, 128, 128, 2, 4, 4>>(p, plan, ws, st); break;
    case F8_WIDE_64x64: launch_tiles<F8Tile<true, E5, 64, 64, 1, 4, 4>>(p, plan, ws, st); break;
    default:  // at most 64 rows of B
      if (p.g.nb <= 16)
        launch_stream<E5, 1>(p, st);
      else if (p.g.nb <= 32)
        launch_stream<E5, 2>(p, st);
      else
        launch_stream<E5, 4>(p, st);
  }
}

}  // namespace

// Workspace: the partial sums of split tiles, for either type of the output.
size_t linear_f8_ws_bytes(int64_t na, int64_t nb, int64_t k) {
  return std::max(f8_plan(na, nb, k, false).ws_bytes, f8_plan(na, nb, k, true).ws_bytes);
}

sg_status launch_linear_f8(const F8LinearArgs& a, void* ws, const char* what, hipStream_t st) {
  F8Args p{};
  p.g.A = a.A;
  p.g.lda = a.lda;
  p.g.na = a.na;
  p.g.B = a.B;
  p.g.ldb = a.ldb;
  p.g.nb = a.nb;
  p.g.kbytes = round_up(a.k, SG_F8_BLOCK);
  p.g.out = a.out;
  p.g.out_dtype = a.out_dtype;
  p.g.ldo = a.ldo;
  p.g.mask = a.mask;
  p.g.accumulate = a.accumulate;
  p.a_scale = a.a_scale;
  p.a_lds = a.a_lds;
  p.b_scale = a.b_scale;
  p.b_lds = a.b_lds;
  p.has_drop = a.drop != nullptr;
  if (a.drop) p.drop = *a.drop;
  const F8Plan plan = f8_plan(a.na, a.nb, a.k, a.out_dtype == SG_F32);
  if (a.b_format == SG_E5M2)
    launch_f8_t<true>(p, plan, ws, st);
  else
    launch_f8_t<false>(p, plan, ws, st);
  return check_launch(what);
}

}  // namespace sg
