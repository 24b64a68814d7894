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

// Few rows of B: every workgroup takes 16 rows of A and all of B's (16 TF at most); its W waves
// divide the contraction and add their sums up in LDS, in wave order.  Operands
// go from memory straight to registers.
template <bool E5, int TF, int W>
__global__ __launch_bounds__(64 * W) void f8_stream_kernel(const F8Args p, NtWide wide) {
  __shared__ floatx4 red[W][TF][64];
  const NtArgs& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t a0 = (int64_t)blockIdx.x * 16;
  const int steps = (int)(g.kbytes / 128);
  const int s0 = (int)((int64_t)steps * wave / W), s1 = (int)((int64_t)steps * (wave + 1) / W);
  // rows past the end re-read the last one; their sums are not stored
  const int64_t ra = min<int64_t>(a0 + (lane & 15), g.na - 1);
  const unsigned char* pa = g.A + ra * g.lda + (lane >> 4) * 16;
  const unsigned char* pb[TF];
  int64_t rb[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    rb[f] = min<int64_t>(16 * f + (lane & 15), g.nb - 1);
    pb[f] = g.B + rb[f] * g.ldb + (lane >> 4) * 16;
  }
  const int64_t rc = min<int64_t>(a0 + (lane >> 4) * 4, (g.na - 1) & ~(int64_t)3);  // (scale rows are padded to 16)
  floatx4 acc[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) acc[f] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto frag = [](const unsigned char* q) {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(q), hi = *reinterpret_cast<const u32x4*>(q + 64);
    return f8_frag{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  for (int s = s0; s < s1; ++s) {
    const f8_frag a = frag(pa + (int64_t)s * 128);
    const uint32_t ea = *reinterpret_cast<const uint32_t*>(p.a_scale + s * p.a_lds + rc);
    const F8Wide wa = f8_widen<false>(a);
#pragma unroll
    for (int f = 0; f < TF; ++f) {
      const F8Wide wb = f8_widen<E5>(frag(pb[f] + (int64_t)s * 128));
      const int eb = p.b_scale[s * p.b_lds + rb[f]];
      const floatx4 part = f8_dot_wide(wa, wb);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = f8_add_scaled(acc[f][i], part[i], (int)((ea >> (8 * i)) & 255u) + eb);
    }
  }
#pragma unroll
  for (int f = 0; f < TF; ++f) red[wave][f][lane] = acc[f];
  __syncthreads();
  const DropKey key = p.has_drop ? drop_key(p.drop) : DropKey{};
  for (int i = tid; i < 64 * TF; i += 64 * W) {
    floatx4 v[1] = {red[0][i >> 6][i & 63]};
#pragma unroll
    for (int w = 1; w < W; ++w) v[0] += red[w][i >> 6][i & 63];
    const int64_t a = a0 + ((i & 63) >> 4) * 4, b = 16 * (i >> 6) + (i & 15);
    if (p.has_drop) f8_drop<4>(p, key, a, b, v);
    NtSide<EP_MASKED, 4> side;
    side.load(g, a, b, wide);
    nt_store<EP_MASKED, 4>(g, a, b, v, wide, side);
  }
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

// panels of A whose tiles run together
constexpr int kBand = 8;

// One tile a workgroup.  Split: every tile's contraction is divided over `splits`
// workgroups, whose sums go to `part` (one 16-byte slot a fragment and thread);
// the join kernel adds them up in split order.
template <typename Tile, bool SPLIT>
__global__ __launch_bounds__(Tile::THREADS) void f8_tiles_kernel(const F8Args p, NtWide wide, int64_t ta, int64_t tb,
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
  const bool aligned = nt_aligned<EP_MASKED>(p.g, wide);
  static_assert(Tile::LDS >= Tile::THREADS / 64 * kTurnBytes, "the stages' LDS turns the sums");
  if (!aligned) __syncthreads();  // every wave is past its last read of the stages
  unsigned char* const turn = lds + (threadIdx.x >> 6) * kTurnBytes;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int q = 0; q < Tile::ITEMS; ++q) {
    const int h = q / Tile::FB, j = q % Tile::FB;
    int64_t a, b;
    Tile::item(ia * Tile::TA, ib * Tile::TB, q, a, b);
    floatx4 v[4] = {acc[4 * h][j], acc[4 * h + 1][j], acc[4 * h + 2][j], acc[4 * h + 3][j]};
    if (p.has_drop) f8_drop16(p, kept.of(q), v);
    if (aligned) {
      NtSide<EP_MASKED, 16> side;
      side.load(p.g, a, b, wide);
      nt_store<EP_MASKED, 16>(p.g, a, b, v, wide, side);
    } else {
      nt_store_rows<EP_MASKED>(p.g, a - (lane >> 4) * 16, b - (lane & 15), v, turn);
    }
  }
}

// One workgroup per tile and item: the sums of its splits, in their order.
template <typename Tile>
__global__ __launch_bounds__(Tile::THREADS) void f8_join_kernel(const F8Args p, NtWide wide, int64_t ta, int64_t tb,
                                                                int splits, const floatx4* part) {
  __shared__ __attribute__((aligned(16))) unsigned char turn[Tile::THREADS / 64 * kTurnBytes];
  const int64_t k = blockIdx.x;
  const int q = (int)blockIdx.y, h = q / Tile::FB, j = q % Tile::FB;
  const int lane = threadIdx.x & 63;
  int64_t ia, ib, a, b;
  nt_tile_of(k, ta, tb, kBand, ia, ib);
  Tile::item(ia * Tile::TA, ib * Tile::TB, q, a, b);
  const int64_t wa0 = a - (lane >> 4) * 16, wb0 = b - (lane & 15);  // the wave's corner
  if (wb0 >= p.g.nb || wa0 >= p.g.na) return;
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
  if (nt_aligned<EP_MASKED>(p.g, wide)) {
    NtSide<EP_MASKED, 16> side;
    side.load(p.g, a, b, wide);
    nt_store<EP_MASKED, 16>(p.g, a, b, v, wide, side);
  } else {
    nt_store_rows<EP_MASKED>(p.g, wa0, wb0, v, turn + (threadIdx.x >> 6) * kTurnBytes);
  }
}

// The tiles there are, largest first: those of the matrix instruction for 8-bit
// floating point, then those of widened codes.
enum { F8_256x256 = 0, F8_256x128, F8_128x128, F8_64x64, F8_WIDE_128x128, F8_WIDE_64x64, F8_STREAM };
struct F8Plan {
  int tile;
  int splits;
  size_t ws_bytes;  // partial sums
};

struct F8TileCost {
  int ta, tb;
  int per_cu;    // workgroups that fit a CU
  double us[2];  // a stage with one and with two workgroups on every CU
};
constexpr F8TileCost kTiles[6] = {{256, 256, 1, {1.40, 0}},  {256, 128, 1, {0.80, 0}}, {128, 128, 1, {0.50, 0}},
                                  {64, 64, 2, {0.25, 0.40}}, {128, 128, 1, {0.90, 0}}, {64, 64, 2, {0.35, 0.60}}};
constexpr double kLaunch = 4.0;      // a tile's fill, epilogue and launch
constexpr double kRound = 2.0;       // a later round's fill and epilogue
constexpr double kJoin = 4.5;        // a second launch
constexpr double kJoinRate = 3.0e6;  // bytes of partial sums a microsecond, written and read

// The tile and the splits that should take the least time.
F8Plan f8_plan(int64_t na, int64_t nb, int64_t k, bool wide) {
  if (nb <= 16 || (nb <= 64 && na * k <= (4 << 20))) return F8Plan{F8_STREAM, 1, 0};
  const int first = wide ? F8_WIDE_128x128 : F8_256x256, last = wide ? F8_STREAM : F8_WIDE_128x128;
  F8Plan p{first, 1, 0};
  const int64_t stages = std::max<int64_t>(1, ceil_div(k, 128));
  double best = 1e300;
  for (int t = first; t < last; ++t) {
    const F8TileCost& c = kTiles[t];
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
  const NtWide wide = nt_wide(p.g);
  const int64_t ta = ceil_div(p.g.na, Tile::TA), tb = ceil_div(p.g.nb, Tile::TB);
  if (plan.splits > 1) {  // (of few tiles)
    floatx4* const part = static_cast<floatx4*>(ws);
    const unsigned grid = (unsigned)(ceil_div(ta * tb * plan.splits, 8) * 8);
    f8_tiles_kernel<Tile, true><<<grid, Tile::THREADS, 0, st>>>(p, wide, ta, tb, plan.splits, part);
    f8_join_kernel<Tile><<<dim3((unsigned)(ta * tb), Tile::ITEMS), Tile::THREADS, 0, st>>>(p, wide, ta, tb,
                                                                                                 plan.splits, part);
    return;
  }
  const int64_t most = kMaxWorkgroups / ta;  // panels of B in a launch
  for (int64_t b = 0; b < tb; b += most) {
    const int64_t n = std::min(most, tb - b), b0 = b * Tile::TB;
    const unsigned grid = (unsigned)(ceil_div(ta * n, 8) * 8);
    f8_tiles_kernel<Tile, false><<<grid, Tile::THREADS, 0, st>>>(
        f8_rows_of(p, b0, std::min<int64_t>(p.g.nb - b0, n * Tile::TB)), wide, ta, n, 1, nullptr);
  }
}

template <bool E5>
void launch_f8_t(const F8Args& p, const F8Plan& plan, void* ws, hipStream_t st) {
  switch (plan.tile) {
    case F8_256x256: launch_tiles<F8Tile<false, E5, 256, 256, 2, 4, 2>>(p, plan, ws, st); break;
    case F8_256x128: launch_tiles<F8Tile<false, E5, 256, 128, 4, 2, 3>>(p, plan, ws, st); break;
    case F8_128x128: launch_tiles<F8Tile<false, E5, 128, 128, 2, 4, 4>>(p, plan, ws, st); break;
    case F8_64x64: launch_tiles<F8Tile<false, E5, 64, 64, 1, 4, 4>>(p, plan, ws, st); break;
    case F8_WIDE_128x128: launch_tiles<F8Tile<true, E5, 128, 128, 2, 4, 4>>(p, plan, ws, st); break;
    case F8_WIDE_64x64: launch_tiles<F8Tile<true, E5, 64, 64, 1, 4, 4>>(p, plan, ws, st); break;
    default: {  // at most 64 rows of B
      const NtWide wide = nt_wide(p.g);
      const unsigned ga = (unsigned)ceil_div(p.g.na, 16);
      if (p.g.nb <= 16)
        f8_stream_kernel<E5, 1, 8><<<ga, 512, 0, st>>>(p, wide);
      else
        f8_stream_kernel<E5, 4, 4><<<ga, 256, 0, st>>>(p, wide);
    }
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
