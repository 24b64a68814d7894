// Products of two matrices whose rows both run along the contraction:
//   out[b][a] = epilogue( sum_k A[a][k] B[b][k] )
// in signed bytes (int32 sums) or bf16 (fp32 sums).  Both element types are
// moved as 64-byte row pieces: one MFMA step takes 16 bytes of a row a lane
// (v_mfma_i32_16x16x64_i8: 64 elements, v_mfma_f32_16x16x32_bf16: 32).
// A's rows are the MFMA's rows, so a lane ends up with four neighbouring
// outputs of one row of `out`.
#pragma once

#include "sg_internal.h"

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

// Four neighbouring outputs of row b from column a on (those inside the
// matrix), from four sums.
template <int EP, typename V4>
__device__ __forceinline__ void nt_store4(const NtArgs& g, int64_t a, int64_t b, V4 v, bool vec) {
  if (b >= g.nb || a >= g.na) return;
  const int cnt = (int)(g.na - a < 4 ? g.na - a : 4);
  float f[4];
  if constexpr (EP == EP_LINEAR) {
    const float sb = g.b_scale[b];
    const int32_t qb = g.b_sum[b];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t ai = a + (i < cnt ? i : 0);
      // wraps like the sums of two's complement; the total fits (n <= 65536)
      const uint32_t tot = (uint32_t)v[i] + (uint32_t)g.a_off[ai] * (uint32_t)qb;
      // the channel's scale first: a sum times the scale of a huge token could
      // leave the range that the output stays in
      f[i] = (float)(int32_t)tot * g.a_scale[ai] * sb;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
  if constexpr (EP == EP_MASKED) {
    if (g.mask) {
      const uint8_t* mk = g.mask + b * g.na + a;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt && mk[i]) f[i] = 0.0f;
    }
  }
  if (g.out_dtype == SG_F32) {
    float* o = static_cast<float*>(g.out) + b * g.ldo + a;
    if (vec && cnt == 4) {
      floatx4 w = floatx4{f[0], f[1], f[2], f[3]};
      if (EP == EP_MASKED && g.accumulate) w += *reinterpret_cast<const floatx4*>(o);
      *reinterpret_cast<floatx4*>(o) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) o[i] = f[i] + ((EP == EP_MASKED && g.accumulate) ? o[i] : 0.0f);
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
    if (EP == EP_MASKED && g.accumulate) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) f[i] += bf16_to_f32(o[i]);
    }
    if (vec && cnt == 4) {
      const uint2 w = make_uint2(bf16_of(f[0]) | (bf16_of(f[1]) << 16), bf16_of(f[2]) | (bf16_of(f[3]) << 16));
      *reinterpret_cast<uint2*>(o) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < cnt) o[i] = (uint16_t)bf16_of(f[i]);
    }
  }
}

// How far the outputs may be stored in wide pieces.
struct NtWide {
  int out4;    // four neighbouring outputs at once
  int out16;   // 16 bytes at once, 16 neighbouring outputs
  int mask16;  // 16 mask bytes at once
};
inline NtWide nt_wide(const NtArgs& g) {
  const int64_t e = g.out_dtype == SG_F32 ? 4 : 2;
  const uintptr_t p = reinterpret_cast<uintptr_t>(g.out);
  NtWide w;
  w.out4 = p % (4 * e) == 0 && g.ldo % 4 == 0;
  w.out16 = p % 16 == 0 && (g.ldo * e) % 16 == 0;
  w.mask16 = g.mask && reinterpret_cast<uintptr_t>(g.mask) % 16 == 0 && g.na % 16 == 0;
  return w;
}

// Sixteen neighbouring outputs of row b from column a on.
template <int EP, typename V4>
__device__ __forceinline__ void nt_store16(const NtArgs& g, int64_t a, int64_t b, const V4 (&v)[4], const NtWide& wide) {
  if (b >= g.nb || a >= g.na) return;
  const bool whole = a + 16 <= g.na && wide.out16 && (EP != EP_MASKED || !g.mask || wide.mask16);
  if (!whole) {
#pragma unroll
    for (int f = 0; f < 4; ++f) nt_store4<EP>(g, a + 4 * f, b, v[f], wide.out4 != 0);
    return;
  }
  float o[16];
  if constexpr (EP == EP_LINEAR) {
    const float sb = g.b_scale[b];
    const uint32_t qb = (uint32_t)g.b_sum[b];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t tot = (uint32_t)v[i >> 2][i & 3] + (uint32_t)g.a_off[a + i] * qb;
      o[i] = (float)(int32_t)tot * g.a_scale[a + i] * sb;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = v[i >> 2][i & 3];
  }
  if constexpr (EP == EP_MASKED) {
    if (g.mask) {
      const u32x4 mk = *reinterpret_cast<const u32x4*>(g.mask + b * g.na + a);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((mk[i >> 2] >> (8 * (i & 3))) & 0xffu) o[i] = 0.0f;
    }
  }
  if (g.out_dtype == SG_F32) {
    float* p = static_cast<float*>(g.out) + b * g.ldo + a;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      floatx4 w = floatx4{o[4 * f], o[4 * f + 1], o[4 * f + 2], o[4 * f + 3]};
      if (EP == EP_MASKED && g.accumulate) w += *reinterpret_cast<const floatx4*>(p + 4 * f);
      *reinterpret_cast<floatx4*>(p + 4 * f) = w;
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
    if (EP == EP_MASKED && g.accumulate) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] += bf16_to_f32(p[i]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = bf16_of(o[8 * h + 2 * i]) | (bf16_of(o[8 * h + 2 * i + 1]) << 16);
      *reinterpret_cast<u32x4*>(p + 8 * h) = w;
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles in LDS
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) void nt_lds_void;

// One LDS-DMA copy: lane l moves 16 bytes from base + off (its own offset) to
// LDS byte address lds + 16 l.  In inline assembly so that the compiler adds
// no waits of its own for copies in flight; it has no register results, and
// every wait for it is written out.
__device__ __forceinline__ void nt_copy16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
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

template <int N>
__device__ __forceinline__ void nt_wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A tile of TA rows of A by TB rows of B, WA x WB waves, each with FA x FB
// fragments of 16 x 16 sums.  A stage is 64 bytes of the contraction of every
// row of both panels; four stages rotate through LDS.  While the products of
// stage s run from registers, the fragments of stage s + 1 are read from LDS
// and stages s + 2 .. s + 4 are on their way.
//
// In LDS a panel's rows lie 64 bytes apart, and 16-byte piece p of row r holds
// piece p ^ sw(r) of the row, so that the 16 lanes of a read that take one
// piece of 16 rows touch every bank once.  sw = (r >> 4) & 3 in A's panel,
// whose fragment f of a 64-row group takes rows 16 (i / 4) + 4 f + i % 4, i =
// 0 .. 15 (a lane then ends up with 16 neighbouring outputs over the four
// fragments); sw = (r >> 2) & 3 in B's, whose fragments take 16 rows in order.
template <bool I8, int TA_, int TB_, int WA_, int WB_>
struct NtTile {
  static constexpr int TA = TA_, TB = TB_, WA = WA_, WB = WB_;
  static constexpr int WAVES = WA * WB, THREADS = 64 * WAVES;
  static constexpr int FA = TA / WA / 16, FB = TB / WB / 16;
  static constexpr int GA = FA / 4;  // 64-row groups of a wave
  static constexpr int STAGE = (TA + TB) * 64;
  static constexpr int COPIES = (TA + TB) / 16 / WAVES;  // copy instructions of a wave and stage
  static_assert(FA % 4 == 0 && (TA + TB) % (16 * WAVES) == 0 && (TA / 16) % COPIES == 0, "tile shape");
  typedef typename NtAcc<I8>::type acc_t;

  struct Frags {
    u32x4 a[FA], b[FB];
  };

  // Sums over stages [s0, s1) of the tile with corner (a0, b0).
  static __device__ __forceinline__ void run(const NtArgs& g, unsigned char* lds, int64_t a0, int64_t b0, int s0, int s1,
                                             acc_t (&acc)[FA][FB]) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wa = wave / WB, wb = wave % WB;
    // copy role: COPIES blocks of 16 rows a wave, all of one panel
    const int blk0 = wave * COPIES;
    const bool is_a = blk0 < TA / 16;
    const unsigned char* base = is_a ? g.A + a0 * g.lda : g.B + b0 * g.ldb;
    const int64_t ld = is_a ? g.lda : g.ldb;
    const int64_t rows = is_a ? g.na - a0 : g.nb - b0;  // rows past the end re-read the last one
    uint32_t off[COPIES];
#pragma unroll
    for (int k = 0; k < COPIES; ++k) {
      const int r = (blk0 + k - (is_a ? 0 : TA / 16)) * 16 + (lane >> 2);
      const int sw = is_a ? (r >> 4) & 3 : (r >> 2) & 3;
      const int64_t rr = r < rows ? r : rows - 1;
      off[k] = (uint32_t)(rr * ld + (((lane & 3) ^ sw) << 4));
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(nt_lds_void*)lds;
    const uint32_t dst0 = lds0 + (uint32_t)blk0 * 1024u;
    auto copy = [&](int s) {
      const unsigned char* p = base + (int64_t)s * 64;
      const uint32_t d = dst0 + (uint32_t)((s - s0) & 3) * (uint32_t)STAGE;
#pragma unroll
      for (int k = 0; k < COPIES; ++k) nt_copy16(p, off[k], __builtin_amdgcn_readfirstlane(d + (uint32_t)k * 1024u));
    };
    const int row = lane & 15, piece = lane >> 4;
    const int ra = wa * (TA / WA) + (row >> 2) * 16 + (row & 3);
    const int rb = wb * (TB / WB) + row;
    const int pa = ra * 64 + ((piece ^ ((row >> 2) & 3)) << 4);
    const int pb = (TA + rb) * 64 + ((piece ^ ((row >> 2) & 3)) << 4);
    auto fetch = [&](int s, Frags& f) {
      const unsigned char* st = lds + ((s - s0) & 3) * STAGE;
#pragma unroll
      for (int j = 0; j < FB; ++j) f.b[j] = *reinterpret_cast<const u32x4*>(st + pb + j * 1024);
#pragma unroll
      for (int i = 0; i < FA; ++i)
        f.a[i] = *reinterpret_cast<const u32x4*>(st + pa + (i >> 2) * 4096 + (i & 3) * 256);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = NtAcc<I8>::mma(f.a[i], f.b[j], acc[i][j]);
    };
    const int n = s1 - s0;
    if (n <= 0) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) copy(s0 + k);
    if (n >= 4)
      nt_wait_copies<3 * COPIES>();
    else if (n == 3)
      nt_wait_copies<2 * COPIES>();
    else if (n == 2)
      nt_wait_copies<COPIES>();
    else
      nt_wait_copies<0>();
    nt_barrier();
    Frags f0, f1;
    fetch(s0, f0);
    // Step s: this wave's copies of stage s + 1 are in (two younger stages may
    // be on their way) and its fragments of stage s are in registers; past
    // the barrier that holds for every wave, so stage s's buffer is free for
    // stage s + 4 and stage s + 1 can be read.
    auto step = [&](int s, const Frags& now, Frags& next) {
      nt_wait_copies<2 * COPIES>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      nt_barrier();
      copy(s + 4);
      fetch(s + 1, next);
      multiply(now);
    };
    int s = s0;
    for (; s + 6 <= s1; s += 2) {
      step(s, f0, f1);
      step(s + 1, f1, f0);
    }
    // the last stages: nothing more to copy past s1
    auto last = [&](int q, const Frags& now, Frags& next) {
      const int younger = min(q + 3, s1 - 1) - (q + 1);
      if (younger >= 2)
        nt_wait_copies<2 * COPIES>();
      else if (younger == 1)
        nt_wait_copies<COPIES>();
      else
        nt_wait_copies<0>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      nt_barrier();
      if (q + 4 < s1) copy(q + 4);
      if (q + 1 < s1) fetch(q + 1, next);
      multiply(now);
    };
    for (; s < s1; s += 2) {
      last(s, f0, f1);
      if (s + 1 < s1) last(s + 1, f1, f0);
    }
  }

  // Calls store(a, b, v) for the tile's sums, 16 neighbouring columns a of a row b at a time.
  template <typename F>
  static __device__ __forceinline__ void each(int64_t a0, int64_t b0, const acc_t (&acc)[FA][FB], F&& store) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wa = wave / WB, wb = wave % WB;
#pragma unroll
    for (int h = 0; h < GA; ++h)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
        const acc_t v[4] = {acc[4 * h][j], acc[4 * h + 1][j], acc[4 * h + 2][j], acc[4 * h + 3][j]};
        store(a0 + wa * (TA / WA) + h * 64 + (lane >> 4) * 16, b0 + wb * (TB / WB) + j * 16 + (lane & 15), v);
      }
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
