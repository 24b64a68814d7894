// Products of two matrices whose rows both run along the contraction:
//   out[b][a] = epilogue( sum_k A[a][k] B[b][k] )
// in signed bytes (int32 sums) or bf16 (fp32 sums).  Both element types are
// moved as 64-byte row pieces: one MFMA step takes 16 bytes of a row a lane
// (v_mfma_i32_16x16x64_i8: 64 elements, v_mfma_f32_16x16x32_bf16: 32).
// A's rows are the MFMA's rows, so a lane ends up with four neighbouring
// outputs of one row of `out`.
#pragma once

#include "sg_internal.h"

#include <type_traits>

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
  int64_t krows, bcols; // B[k][b] (tiles with BT): its rows, its columns rounded up to 8
  const float* k_scale;   // A as bytes A[k][a] (code tiles): of each of its krows rows
  const int32_t* k_off;
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

// How far the outputs may be stored in wide pieces.
struct NtWide {
  int out4;    // four neighbouring outputs at once
  int out16;   // 16 bytes at once
  int mask16;  // 16 mask bytes at once
  int mask4;   // four mask bytes at once
};
inline NtWide nt_wide(const NtArgs& g) {
  const int64_t e = g.out_dtype == SG_F32 ? 4 : 2;
  const uintptr_t p = reinterpret_cast<uintptr_t>(g.out);
  NtWide w;
  w.out4 = p % (4 * e) == 0 && g.ldo % 4 == 0;
  w.out16 = p % 16 == 0 && (g.ldo * e) % 16 == 0;
  w.mask16 = g.mask && reinterpret_cast<uintptr_t>(g.mask) % 16 == 0 && g.na % 16 == 0;
  w.mask4 = g.mask && reinterpret_cast<uintptr_t>(g.mask) % 4 == 0 && g.na % 4 == 0;
  return w;
}

// What the epilogue of N neighbouring outputs of row b from column a on reads
// besides the sums.  Tiles with one such group a lane load it before their
// products: after them its latency would be bare (a microsecond from HBM).
template <int EP, int N>
struct NtSide {
  float a_scale[EP == EP_LINEAR ? N : 1];
  int32_t a_off[EP == EP_LINEAR ? N : 1];
  float b_scale;
  int32_t b_sum;
  uint32_t pruned;  // bit i: mask[b][a + i]

  __device__ __forceinline__ void load(const NtArgs& g, int64_t a, int64_t b, const NtWide& wide) {
    pruned = 0u;
    if (b >= g.nb || a >= g.na) return;
    if constexpr (EP == EP_LINEAR) {
      b_scale = g.b_scale[b];
      b_sum = g.b_sum[b];
      if (a + N <= g.na) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          a_scale[i] = g.a_scale[a + i];
          a_off[i] = g.a_off[a + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int64_t c = min<int64_t>(a + i, g.na - 1);
          a_scale[i] = g.a_scale[c];
          a_off[i] = g.a_off[c];
        }
      }
    }
    if constexpr (EP == EP_MASKED) {
      if (g.mask) {
        const uint8_t* m = g.mask + b * g.na + a;
        if (N == 16 && (wide.mask16 || wide.mask4) && a + 16 <= g.na) {
          u32x4 w;
          if (wide.mask16) {
            w = *reinterpret_cast<const u32x4*>(m);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(m)[i];
          }
#pragma unroll
          for (int i = 0; i < N; ++i) pruned |= ((w[(i >> 2) & 3] >> (8 * (i & 3))) & 0xffu) ? 1u << i : 0u;
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (a + i < g.na && m[i]) pruned |= 1u << i;
        }
      }
    }
  }
};

// The gradient of a pruned weight; -0 where it is added, which leaves a zero of
// either sign as it is.
template <int EP>
__device__ __forceinline__ float nt_pruned(const NtArgs& g) {
  return EP == EP_MASKED && g.accumulate ? -0.0f : 0.0f;
}

// N neighbouring outputs of row b from column a on (those inside the matrix),
// from sums in fours.
template <int EP, int N, typename V4>
__device__ __forceinline__ void nt_store(const NtArgs& g, int64_t a, int64_t b, const V4 (&v)[N / 4],
                                         const NtWide& wide, const NtSide<EP, N>& side) {
  if (b >= g.nb || a >= g.na) return;
  const int cnt = (int)min<int64_t>(g.na - a, N);
  const bool add = EP == EP_MASKED && g.accumulate;
  const float none = nt_pruned<EP>(g);
  float o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (EP == EP_LINEAR) {
      // wraps like sums of two's complement; the total fits (n <= 65536).  The
      // channel's scale first: a sum times the scale of a huge token could
      // leave the range that the output stays in
      const uint32_t tot = (uint32_t)v[i >> 2][i & 3] + (uint32_t)side.a_off[i] * (uint32_t)side.b_sum;
      o[i] = (float)(int32_t)tot * side.a_scale[i] * side.b_scale;
    } else {
      o[i] = v[i >> 2][i & 3];
    }
    if (EP == EP_MASKED && ((side.pruned >> i) & 1u)) o[i] = none;
  }
  const bool whole = cnt == N && wide.out4;
  if (g.out_dtype == SG_F32) {
    float* p = static_cast<float*>(g.out) + b * g.ldo + a;
    if (whole) {
#pragma unroll
      for (int f = 0; f < N / 4; ++f) {
        floatx4 w = floatx4{o[4 * f], o[4 * f + 1], o[4 * f + 2], o[4 * f + 3]};
        if (add) w += *reinterpret_cast<const floatx4*>(p + 4 * f);
        *reinterpret_cast<floatx4*>(p + 4 * f) = w;
      }
      return;
    }
    if (add) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < cnt) o[i] += p[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) p[i] = o[i];
    return;
  }
  uint16_t* p = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
  if (whole) {
    if (add) {
#pragma unroll
      for (int f = 0; f < N / 4; ++f) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + 4 * f);
        o[4 * f] += __uint_as_float(w.x << 16);
        o[4 * f + 1] += __uint_as_float(w.x & 0xffff0000u);
        o[4 * f + 2] += __uint_as_float(w.y << 16);
        o[4 * f + 3] += __uint_as_float(w.y & 0xffff0000u);
      }
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = bf16_of(o[2 * i]) | (bf16_of(o[2 * i + 1]) << 16);
    if (N == 16 && wide.out16) {
#pragma unroll
      for (int f = 0; f < N / 8; ++f)
        *reinterpret_cast<u32x4*>(p + 8 * f) = u32x4{w[4 * f], w[4 * f + 1], w[4 * f + 2], w[4 * f + 3]};
    } else {
#pragma unroll
      for (int f = 0; f < N / 4; ++f) *reinterpret_cast<uint2*>(p + 4 * f) = make_uint2(w[2 * f], w[2 * f + 1]);
    }
    return;
  }
  if (add) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) o[i] += bf16_to_f32(p[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < cnt) p[i] = (uint16_t)bf16_of(o[i]);
}

// Whether rows of `out` (and of the mask) can be reached in pieces of four:
// then a lane stores its 16 neighbours (a masked bf16 gradient of 5256 x 7636
// from 467 tokens: 98 us, one by one 219).
template <int EP>
__device__ __forceinline__ bool nt_aligned(const NtArgs& g, const NtWide& wide) {
  return wide.out4 && (EP != EP_MASKED || !g.mask || wide.mask16 || wide.mask4);
}

// A wave's sums of 16 rows from b0 on of 64 columns from a0 on, held as 16
// neighbouring columns a lane, for outputs whose rows lie unaligned: turned in
// `turn` so that 64 lanes store 64 neighbouring outputs of a row.  Stored from
// where they are, 4 or 2 bytes in every 64, 3841 x 1273 fp32 outputs of 736
// products took 40 us, so 23; a bf16 weight gradient of 4099 x 1001 36, so 30;
// only outputs of a few us lose (515 x 771 bf16: 7.4, so 7.9).
constexpr int kTurnPitch = 68;                        // 32-bit words a row
constexpr int kTurnBytes = 16 * kTurnPitch * 4;       // a wave's
template <int EP, typename V4>
__device__ __forceinline__ void nt_store_rows(const NtArgs& g, int64_t a0, int64_t b0, const V4 (&v)[4],
                                              unsigned char* turn) {
  if (a0 >= g.na || b0 >= g.nb) return;  // (the whole wave)
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    *reinterpret_cast<V4*>(turn + ((lane & 15) * kTurnPitch + (lane >> 4) * 16 + 4 * e) * 4) = v[e];
  asm volatile("" ::: "memory");  // a wave's LDS accesses keep their order
  const int64_t a = a0 + lane;
  const bool ok = a < g.na;
  float a_scale = 0.0f;
  uint32_t a_off = 0u;
  if (EP == EP_LINEAR && ok) {
    a_scale = g.a_scale[a];
    a_off = (uint32_t)g.a_off[a];
  }
  const int rows = (int)min<int64_t>(16, g.nb - b0);
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(turn + (r * kTurnPitch + lane) * 4);
    if (!ok) continue;
    const int64_t b = b0 + r;
    float o;
    if constexpr (EP == EP_LINEAR)
      o = (float)(int32_t)(w + a_off * (uint32_t)g.b_sum[b]) * a_scale * g.b_scale[b];
    else
      o = __uint_as_float(w);
    if (EP == EP_MASKED && g.mask && g.mask[b * g.na + a]) o = nt_pruned<EP>(g);
    if (g.out_dtype == SG_F32) {
      float* p = static_cast<float*>(g.out) + b * g.ldo + a;
      *p = (EP == EP_MASKED && g.accumulate) ? *p + o : o;
    } else {
      uint16_t* p = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
      *p = (uint16_t)bf16_of((EP == EP_MASKED && g.accumulate) ? bf16_to_f32(*p) + o : o);
    }
  }
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// Tiles in LDS
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void nt_lds_void;
typedef short nt_short4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) nt_short4 nt_lds_short4;

// One LDS-DMA copy: lane l moves 16 bytes from base + off (its own offset) to
// LDS byte address lds + 16 l.  In inline assembly so that the compiler adds
// no waits of its own for copies in flight; it has no register results, and
// every wait for it is written out.  An instruction that writes M0 needs a wait
// state before the copy; inside this block the compiler would not add it.
__device__ __forceinline__ void nt_copy16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

// Workgroup barrier without the fence that would wait for copies in flight.
__device__ __forceinline__ void nt_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Waits until at most N copies of this wave are on their way and, with LDS,
// until its LDS reads have returned (N = 63: only those; s_waitcnt: vmcnt in bits 0-3 and 14-15,
// lgkmcnt in bits 8-11).
template <int N, bool LDS = false>
__device__ __forceinline__ void nt_wait() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x70 | (LDS ? 0 : 0xf00));
  asm volatile("" ::: "memory");
}

// B's panel of a tile: TB rows of B, a stage of 128 bytes of the contraction of
// each (a whole cache line: pieces of 64 bytes fetch the line twice, 30 against
// 52 bytes a clock and CU were measured), two MFMA steps.
//
// In LDS its rows lie 128 bytes apart, and 16-byte piece p of row r holds piece
// p ^ ((r >> 1) & 7) of the row, so that the 16 lanes of a read that take one
// piece of 16 rows touch every bank once.
//
// BT (bf16 only): B comes with the contraction along its columns, B[k][b], and
// is copied as it lies: a stage is 64 rows k of TB elements, and the fragments
// are gathered by the transposing LDS read (4 rows x 4 columns over 16 lanes).
// 16-byte piece p of row k holds piece p ^ 2 tau(k), so that the 8 rows a
// half-wave touches (k = 0 .. 3 and 8 .. 11, and so on) lie in different banks:
// tau = (k & 3) | ((k & 8) >> 1), with 64 columns ((k >> 1) & 1) | ((k & 8) >>
// 2), two rows filling the banks.  Rows from the end of the contraction on are
// cleared in LDS; columns past B's last re-read its last 8 and feed only sums
// that are not stored.
template <int TB, int WAVES, int WB, bool BT>
struct NtPanelB {
  static constexpr int BYTES = TB * 128;       // a stage in LDS
  static constexpr int COPIES = TB / 8 / WAVES;  // copy instructions of a wave and stage
  static constexpr int FB = TB / WB / 16;
  static_assert(FB >= 1 && TB % (8 * WAVES) == 0 && (!BT || TB == 64 || TB % 128 == 0), "panel shape");

  const unsigned char* base;
  int64_t ldb, krows;
  int64_t k0;  // first contraction row (BT)
  uint32_t off[COPIES];
  int n, wave, lane;
  bool half;
  int at, tau;  // where this lane reads, and its swizzle (BT)

  static __device__ __forceinline__ int tau_of(int k) {
    return TB == 64 ? ((k >> 1) & 1) | ((k & 8) >> 2) : (k & 3) | ((k & 8) >> 1);
  }
  __device__ __forceinline__ int row_of(int k) const {  // panel row (BT: contraction row) of this lane's copy k
    return BT ? ((wave * COPIES + k) * 64 + lane) / (TB / 8) : (wave * COPIES + k) * 8 + (lane >> 3);
  }
  __device__ __forceinline__ int piece_of(int k) const { return (lane & 7) ^ ((row_of(k) >> 1) & 7); }

  // Stages of s0 .. s0 + n - 1; half: the last one has one step.
  __device__ __forceinline__ void init(const NtArgs& g, int64_t b0, int s0, int stages, bool odd) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    n = stages;
    half = odd;
    ldb = g.ldb;
    krows = g.krows;
    k0 = (int64_t)s0 * 64;
    base = BT ? g.B + k0 * ldb : g.B + b0 * ldb + (int64_t)s0 * 128;
#pragma unroll
    for (int k = 0; k < COPIES; ++k) {
      const int r = row_of(k);
      if constexpr (BT) {
        const int64_t col = b0 + 8 * ((((wave * COPIES + k) * 64 + lane) % (TB / 8)) ^ (2 * tau_of(r)));
        off[k] = (uint32_t)(r * ldb + 2 * (col + 8 <= g.bcols ? col : g.bcols - 8));
      } else {
        // rows past the panel's end re-read the last one
        off[k] = (uint32_t)(min<int64_t>(r, g.nb - b0 - 1) * ldb + piece_of(k) * 16);
      }
    }
    const int row = lane & 15, piece = lane >> 4;
    if constexpr (BT) {
      // a transposing read points at row 8 (lane / 16) + (lane % 16) / 4 (and 4
      // rows further) and 4 columns of a fragment
      const int tr = 8 * piece + (row >> 2);
      tau = tau_of(tr);
      at = tr * (TB * 2) + (row & 3) * 8;
    } else {
      tau = 0;
      at = ((wave % WB) * (TB / WB) + row) * 128 + ((piece ^ (row >> 1)) << 4);
    }
  }
  // Copy k of stage s to the slot at LDS address `to`.  ends: the stage may be
  // the last one, of which a row may hold only the first 64 bytes (the other
  // half re-reads them and is not used) and which (BT) the contraction may end
  // in (the rows past it re-read the last one).
  template <bool ends>
  __device__ __forceinline__ void copy(int s, uint32_t to, int k) const {
    uint32_t o = off[k];
    if (ends && s == n - 1) {
      if constexpr (BT) {
        const int64_t past = k0 + (int64_t)s * 64 + row_of(k) - (krows - 1);
        if (past > 0) o -= (uint32_t)(past * ldb);
      } else {
        if (half && piece_of(k) >= 4) o -= 64;
      }
    }
    nt_copy16(BT ? base + (int64_t)s * 64 * ldb : base + (int64_t)s * 128, o,
              __builtin_amdgcn_readfirstlane(to + (uint32_t)((wave * COPIES + k) * 1024)));
  }
  // Fragment q of step h of the stage in `slot`.
  __device__ __forceinline__ u32x4 fetch(const unsigned char* slot, int h, int q) const {
    if constexpr (BT) {
      const unsigned char* p = slot + at + h * (32 * TB * 2) + ((((wave % WB) * FB + q) ^ tau) << 5);
      const nt_short4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((nt_lds_short4*)p);
      const nt_short4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((nt_lds_short4*)(p + 4 * (TB * 2)));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      // (the second step's pieces are 4 .. 7: bit 6 of the offset flips)
      return *reinterpret_cast<const u32x4*>(slot + (at ^ (h * 64)) + q * 2048);
    }
  }
  // BT: clears the rows of the last stage past the end of the contraction.
  __device__ __forceinline__ void clear_tail(unsigned char* slot) const {
    if constexpr (BT) {
      const int64_t valid = krows - k0 - (int64_t)(n - 1) * 64;
      if (valid < 64) {
        for (int e = (int)valid * (TB / 8) + (int)threadIdx.x; e < 64 * (TB / 8); e += 64 * WAVES)
          *reinterpret_cast<u32x4*>(slot + e * 16) = u32x4{0u, 0u, 0u, 0u};
        __syncthreads();
      }
    }
  }
};

// A tile of TA rows of A by TB rows of B, WA x WB waves, each with FA x FB
// fragments of 16 x 16 sums (32 x 32 MFMAs were 4-10% slower).  RA stages of A's panel and RB of B's rotate
// through LDS.  While the products of one step run from registers, the
// fragments of the next are read from LDS, and the younger stages are on their
// way.  A 256 x 256 tile with three stages of A and two of B fills the 160 KB;
// its eight waves keep 128 sums and two steps' fragments a lane in registers.
// 128-byte stages took the 8192 x 4096 x 4096 product in bytes from 145 to 124
// us, the copies spread between the products one round of it from 47 to 44.
//
// A's panel lies in LDS like B's, but fragment f of a 64-row group takes rows
// 16 (i / 4) + 4 f + i % 4, i = 0 .. 15 (a lane then ends up with 16
// neighbouring outputs over the four fragments), and the swizzle is p ^ (2 ((r
// >> 4) & 3) + ((r >> 1) & 1)).
template <bool I8, int TA_, int TB_, int WA_, int WB_, int RA_, int RB_, bool BT_ = false>
struct NtTile {
  static constexpr int TA = TA_, TB = TB_, WA = WA_, WB = WB_, RA = RA_, RB = RB_;
  static constexpr bool BT = BT_;
  static constexpr int WAVES = WA * WB, THREADS = 64 * WAVES;
  typedef NtPanelB<TB, WAVES, WB, BT> PanelB;
  static constexpr int FA = TA / WA / 16, FB = PanelB::FB;
  static constexpr int GA = FA / 4;  // 64-row groups of a wave
  static constexpr int ASTAGE = TA * 128, BSTAGE = PanelB::BYTES;
  static constexpr int LDS = RA * ASTAGE + RB * BSTAGE;
  static constexpr int CA = TA / 8 / WAVES, CB = PanelB::COPIES;  // copy instructions of a wave and stage
  static_assert(FA % 4 == 0 && TA % (8 * WAVES) == 0 && !(I8 && BT), "tile shape");
  static_assert(RB >= 2 && (RA == RB || RA == RB + 1) && LDS <= 160 * 1024, "stages");
  // copies that may be on their way when the next stage has to be in: those
  // issued after it
  static constexpr int YOUNGER = (RA - 2) * CA + (RB - 2) * CB;
  static_assert((RA - 1) * CA + (RB - 1) * CB < 64, "the copies on their way are counted in 6 bits");
  typedef typename NtAcc<I8>::type acc_t;

  struct Frags {
    u32x4 a[FA], b[FB];
  };

  // Sums of the tile with corner (a0, b0) over steps [2 s0, t1) of 64 bytes.
  static __device__ __forceinline__ void run(const NtArgs& g, unsigned char* lds, int64_t a0, int64_t b0, int s0, int t1,
                                             acc_t (&acc)[FA][FB]) {
    const int n = (t1 + 1) / 2 - s0;  // stages
    if (n <= 0) return;
    const bool half = t1 & 1;  // the last stage has one step
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t lds0 = (uint32_t)(uintptr_t)(nt_lds_void*)lds;
    unsigned char* const ldsb = lds + RA * ASTAGE;
    PanelB pb;
    pb.init(g, b0, s0, n, half);
    uint32_t offa[CA];
    const unsigned char* const basea = g.A + a0 * g.lda + (int64_t)s0 * 128;
    auto piece_a = [&](int k) {
      const int r = (wave * CA + k) * 8 + (lane >> 3);
      return (lane & 7) ^ (2 * ((r >> 4) & 3) + ((r >> 1) & 1));
    };
#pragma unroll
    for (int k = 0; k < CA; ++k) {
      const int64_t r = (wave * CA + k) * 8 + (lane >> 3);
      offa[k] = (uint32_t)(min<int64_t>(r, g.na - a0 - 1) * g.lda + piece_a(k) * 16);
    }
    auto copy_a = [&](int s, int slot, int k, auto ends) {
      uint32_t o = offa[k];
      if (decltype(ends)::value && half && s == n - 1 && piece_a(k) >= 4) o -= 64;
      nt_copy16(basea + (int64_t)s * 128, o,
                __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(slot * ASTAGE + (wave * CA + k) * 1024)));
    };
    auto copy_b = [&](int s, int slot, int k, auto ends) {
      pb.template copy<decltype(ends)::value>(s, lds0 + (uint32_t)(RA * ASTAGE + slot * BSTAGE), k);
    };
    const int row = lane & 15;
    const int ra = (wave / WB) * (TA / WA) + (row >> 2) * 16 + (row & 3);
    const int pa = ra * 128 + (((lane >> 4) ^ (2 * (row >> 2) + ((row >> 1) & 1))) << 4);
    int ua = 0, ub = 0;  // slots of the stage being read
    // fragment q of step h of that stage: B's, then A's
    auto fetch = [&](int h, int q, Frags& f) {
      if (q < FB) {
        f.b[q] = pb.fetch(ldsb + ub * BSTAGE, h, q);
      } else {
        const int i = q - FB;
        f.a[i] = *reinterpret_cast<const u32x4*>(lds + ua * ASTAGE + (pa ^ (h * 64)) + (i >> 2) * 8192 + (i & 3) * 512);
      }
    };
    auto up = [](int slot, int slots) { return slot + 1 == slots ? 0 : slot + 1; };
    auto fetch_all = [&](int h, Frags& f) {
#pragma unroll
      for (int q = 0; q < FA + FB; ++q) fetch(h, q, f);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = NtAcc<I8>::mma(f.a[i], f.b[j], acc[i][j]);
    };
    // The products of one step, with the LDS reads of the next one and NC
    // copies spread between them: copies issued in one go stall the wave on the
    // address unit (16 clocks each, shared by the CU's waves).
    auto step = [&](const Frags& now, int h, Frags& next, auto nc, auto&& copy) {
      constexpr int NC = decltype(nc)::value;
      constexpr int RG = FA * 3 / 4;  // the reads return under the last quarter's products
#pragma unroll
      for (int i = 0; i < FA; ++i) {
#pragma unroll
        for (int q = min(i, RG) * (FA + FB) / RG; q < min(i + 1, RG) * (FA + FB) / RG; ++q) fetch(h, q, next);
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = NtAcc<I8>::mma(now.a[i], now.b[j], acc[i][j]);
#pragma unroll
        for (int k = i * NC / FA; k < (i + 1) * NC / FA; ++k) copy(k);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::true_type ends{};
    constexpr std::false_type inside{};
    // Stage s of A's panel is copied during the first step of stage s - RA + 1,
    // stage s of B's during the second step of stage s - RB: their slots are
    // free from the second step of stage s - RA and s - RB on.
#pragma unroll
    for (int k = 0; k < RB; ++k) {
      if (k < RA - 1 && k < n) {
#pragma unroll
        for (int c = 0; c < CA; ++c) copy_a(k, k, c, ends);
      }
      if (k < n) {
#pragma unroll
        for (int c = 0; c < CB; ++c) copy_b(k, k, c, ends);
      }
    }
    if (n >= RB)
      nt_wait<(RA - 2) * CA + (RB - 1) * CB>();
    else
      nt_wait<0>();
    nt_barrier();
    if (n == 1) pb.clear_tail(ldsb + ub * BSTAGE);
    Frags f0, f1;
    fetch_all(0, f0);
    int s = 0;
    int qa = RA - 1, qb = 0;  // slots of the next copies
    // First step of a stage: its second step's fragments are read meanwhile.
    // Second step: the copies of stage s + 1 are in and the fragments of stage
    // s in registers; past the barrier that holds for every wave.
    for (; s + RB + 2 <= n; ++s) {
      nt_wait<63, true>();
      __builtin_amdgcn_sched_barrier(0);
      step(f0, 1, f1, std::integral_constant<int, CA>{}, [&](int k) { copy_a(s + RA - 1, qa, k, inside); });
      qa = up(qa, RA);
      nt_wait<YOUNGER, true>();
      nt_barrier();
      ua = up(ua, RA);
      ub = up(ub, RB);
      __builtin_amdgcn_sched_barrier(0);
      step(f1, 0, f0, std::integral_constant<int, CB>{}, [&](int k) { copy_b(s + RB, qb, k, inside); });
      qb = up(qb, RB);
    }
    for (; s < n; ++s) {
      const bool two = s < n - 1 || !half;
      if (s + RA - 1 < n) {
#pragma unroll
        for (int k = 0; k < CA; ++k) copy_a(s + RA - 1, qa, k, ends);
        qa = up(qa, RA);
      }
      if (two) fetch_all(1, f1);
      multiply(f0);
      if (s < n - 1) {
        if (s + RA - 1 < n)
          nt_wait<YOUNGER, true>();
        else
          nt_wait<0, true>();
        nt_barrier();
        ua = up(ua, RA);
        ub = up(ub, RB);
        if (s + RB < n) {
#pragma unroll
          for (int k = 0; k < CB; ++k) copy_b(s + RB, qb, k, ends);
          qb = up(qb, RB);
        }
        if (s == n - 2) pb.clear_tail(ldsb + ub * BSTAGE);
        fetch_all(0, f0);
      }
      if (two) multiply(f1);
    }
  }

  // Calls f(h, j, a, b) for the wave's 64-row groups h and fragments j of B's
  // panel: this lane's sums acc[4 h .. 4 h + 3][j] are those of 16 neighbouring
  // columns from a on of row b.
  template <typename F>
  static __device__ __forceinline__ void each(int64_t a0, int64_t b0, F&& f) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wa = wave / WB, wb = wave % WB;
#pragma unroll
    for (int h = 0; h < GA; ++h)
#pragma unroll
      for (int j = 0; j < FB; ++j)
        f(h, j, a0 + wa * (TA / WA) + h * 64 + (lane >> 4) * 16, b0 + wb * (TB / WB) + j * 16 + (lane & 15));
  }
};

// The k-th tile in an order that keeps tiles sharing panels together: bands of
// `band` panels of A, and inside a band the panels of B one after another.
__device__ __forceinline__ void nt_tile_of(int64_t k, int64_t ta, int64_t tb, int band, int64_t& ia, int64_t& ib) {
  const int64_t per = (int64_t)band * tb;
  const int64_t q = k / per;
  const int64_t w = ta - q * band < band ? ta - q * band : band;
  const int64_t r = k - q * per;
  ib = r / w;
  ia = q * band + (r - ib * w);
}

// Workgroups go round-robin over the 8 XCDs; XCD x takes a contiguous eighth
// of the tile order, so that the workgroups of one L2 share panels.
__device__ __forceinline__ int64_t nt_xcd_order(int64_t bid, int64_t cnt) {
  const int64_t x = bid & 7, i = bid >> 3;
  const int64_t k0 = cnt * x / 8, k1 = cnt * (x + 1) / 8;
  return i < k1 - k0 ? k0 + i : -1;
}

}  // namespace sg
