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

// Few rows of B: every workgroup takes 16 rows of A and 16 TF of B; its W waves
// divide the contraction and add their sums up in LDS, in wave order.  Operands
// go from memory straight to registers.
template <bool E5, int TF, int W>
__global__ __launch_bounds__(64 * W) void f8_stream_kernel(const F8Args p, NtWide wide) {
  __shared__ floatx4 red[W][TF][64];
  const NtArgs& g = p.g;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t a0 = (int64_t)blockIdx.x * 16, b0 = (int64_t)blockIdx.y * (16 * TF);
  const int steps = (int)(g.kbytes / 128);
  const int s0 = (int)((int64_t)steps * wave / W), s1 = (int)((int64_t)steps * (wave + 1) / W);
  // rows past the end re-read the last one; their sums are not stored
  const int64_t ra = min<int64_t>(a0 + (lane & 15), g.na - 1);
  const unsigned char* pa = g.A + ra * g.lda + (lane >> 4) * 16;
  const unsigned char* pb[TF];
  int64_t rb[TF];
#pragma unroll
  for (int f = 0; f < TF; ++f) {
    rb[f] = min<int64_t>(b0 + 16 * f + (lane & 15), g.nb - 1);
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
    const int64_t a = a0 + ((i & 63) >> 4) * 4, b = b0 + 16 * (i >> 6) + (i & 15);
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

template <bool E5>
void launch_f8_t(const F8Args& p, void*, hipStream_t st) {
  const NtWide wide = nt_wide(p.g);
  const int64_t ga = ceil_div(p.g.na, 16);
  if (p.g.nb <= 16) {
    f8_stream_kernel<E5, 1, 8><<<dim3((unsigned)ga, 1), 512, 0, st>>>(p, wide);
    return;
  }
  // a launch holds less than 2^32 threads
  const int64_t most = std::min<int64_t>(65535, ((int64_t)1 << 23) / ga) * 64;
  for (int64_t b = 0; b < p.g.nb; b += most) {
    const int64_t rows = std::min(most, p.g.nb - b);
    f8_stream_kernel<E5, 4, 4><<<dim3((unsigned)ga, (unsigned)ceil_div(rows, 64)), 256, 0, st>>>(f8_rows_of(p, b, rows),
                                                                                                wide);
  }
}

}  // namespace

size_t linear_f8_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

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
  if (a.b_format == SG_E5M2)
    launch_f8_t<true>(p, ws, st);
  else
    launch_f8_t<false>(p, ws, st);
  return check_launch(what);
}

}  // namespace sg
