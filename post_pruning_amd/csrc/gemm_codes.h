// Products whose A comes as signed bytes with the contraction along their
// columns and a scale (and an offset) for each contraction row:
//   out[b][a] = sum_k bf16(scale[k] * (A[k][a] + offset[k])) B[b][k]
// (or B[k][b]).  The bytes are turned to bf16 on their way through LDS, once a
// workgroup, so that no bf16 copy of A is made in memory: with few rows of B
// that copy is most of the work.  4096 x 4096 codes with 64 rows of B take 17 us
// (25 with the copy), 8192 x 28672 about 90 us (307).  A stage is a chain of LDS
// reads, conversions and a barrier (0.55 us for 64 x 64), which bounds it; with
// many rows of B every tile converts again, and the copy wins.
#pragma once

#include "gemm_nt.h"

namespace sg {

// One LDS-DMA copy of 4 bytes a lane (s_nop: as in nt_copy16).
__device__ __forceinline__ void nt_copy4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

// A tile of TA columns of A by TB rows of B, WA x WB waves.  A stage is 64
// contraction rows.  RB stages of B's panel, of A's bytes and of their scales
// rotate through LDS; every lane copies 16 bytes of one row of A a stage and
// reads the same 16 back two stages ahead, so those need no barrier.  During the
// first step of stage s it turns its bytes of stage s + 1 to bf16 and writes
// them to one of two panels, which the waves gather fragments from by
// transposing reads.
//
// A panel's rows k hold 32-byte groups of 16 columns, each as four 8-byte
// pieces.  Fragment f of a 64-column group takes piece f of its four groups (a
// lane then ends up with 16 neighbouring outputs over the four fragments).
// The 8 rows that a half-wave reads (k = 0 .. 3 and 8 .. 11, and so on) would
// all touch the same banks, so group p of row k lies at p ^ 4 ((k >> 3) & 1)
// and piece f at f ^ (k & 3); with 64 columns two rows fill the banks, groups
// stay, and piece f lies at f ^ (((k >> 1) & 1) + 2 ((k >> 3) & 1)).
template <int TA_, int TB_, int WA_, int WB_, int RB_, bool BT_, bool OFFSET_>
struct CodeTile {
  static constexpr int TA = TA_, TB = TB_, WA = WA_, WB = WB_, RB = RB_;
  static constexpr bool BT = BT_, OFFSET = OFFSET_;
  static constexpr int WAVES = WA * WB, THREADS = 64 * WAVES;
  typedef NtPanelB<TB, WAVES, WB, BT> PanelB;
  static constexpr int FA = TA / WA / 16, FB = PanelB::FB, GA = FA / 4;
  static constexpr int APANEL = TA * 128;                                // 64 rows in bf16
  static constexpr int RAW = TA * 64 + WAVES * (OFFSET ? 512 : 256);     // bytes of A, then scales
  static constexpr int BSTAGE = PanelB::BYTES;
  static constexpr int LDS = 2 * APANEL + RB * (RAW + BSTAGE);
  static constexpr int CB = PanelB::COPIES, COPIES = CB + (OFFSET ? 3 : 2);  // of a wave and stage
  static_assert(TA * 64 == 1024 * WAVES && FA == 4 && RB >= 4 && LDS <= 160 * 1024, "tile shape");
  static_assert((RB - 1) * COPIES < 64, "the copies on their way are counted in 6 bits");
  typedef floatx4 acc_t;

  struct Frags {
    u32x4 a[FA], b[FB];
  };

  // Sums of the tile with corner (a0, b0) over steps [2 s0, t1) of 32 rows.
  static __device__ __forceinline__ void run(const NtArgs& g, unsigned char* lds, int64_t a0, int64_t b0, int s0, int t1,
                                             acc_t (&acc)[FA][FB]) {
    const int n = (t1 + 1) / 2 - s0;  // stages
    if (n <= 0) return;
    const bool half = t1 & 1;  // the last stage has one step
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t lds0 = (uint32_t)(uintptr_t)(nt_lds_void*)lds;
    constexpr int RAW0 = 2 * APANEL, B0 = RAW0 + RB * RAW, SCALES = TA * 64;
    PanelB pb;
    pb.init(g, b0, s0, n, half);
    // this lane's 16 bytes of a stage: row kr, columns a0 + 16 p ..
    const int kr = (wave * 64 + lane) / (TA / 16), p = (wave * 64 + lane) % (TA / 16);
    const int64_t k0 = (int64_t)s0 * 64;
    const int64_t wide = (g.na + 63) / 64 * 64;  // the rows' bytes
    const unsigned char* const basea = g.A + k0 * g.lda;
    const uint32_t offa = (uint32_t)(kr * g.lda + min<int64_t>(a0 + 16 * p, wide - 16));
    const float* const scale = g.k_scale + k0;
    const int32_t* const offset = OFFSET ? g.k_off + k0 : nullptr;
    // copy c of stage s: B's panel, then the bytes, their scales and offsets;
    // ends: rows past the end of the contraction re-read the last one
    auto copy = [&](int s, int slot, int c, auto ends) {
      if (c < CB) {
        pb.template copy<decltype(ends)::value>(s, lds0 + (uint32_t)(B0 + slot * BSTAGE), c);
        return;
      }
      const uint32_t to = lds0 + (uint32_t)(RAW0 + slot * RAW);
      int64_t past = 0;
      if (decltype(ends)::value && s == n - 1) past = max<int64_t>(0, k0 + (int64_t)s * 64 + kr - (g.krows - 1));
      if (c == CB)
        nt_copy16(basea + (int64_t)s * 64 * g.lda, offa - (uint32_t)(past * g.lda),
                  __builtin_amdgcn_readfirstlane(to + (uint32_t)(wave * 1024)));
      else if (c == CB + 1)
        nt_copy4(scale + (int64_t)s * 64, (uint32_t)(kr - past) * 4,
                 __builtin_amdgcn_readfirstlane(to + (uint32_t)(SCALES + wave * 256)));
      else
        nt_copy4(offset + (int64_t)s * 64, (uint32_t)(kr - past) * 4,
                 __builtin_amdgcn_readfirstlane(to + (uint32_t)(SCALES + (WAVES + wave) * 256)));
    };
    struct Raw {
      u32x4 v;
      float s, o;
    };
    auto read_raw = [&](int s, int slot) {
      const unsigned char* q = lds + RAW0 + slot * RAW;
      Raw r;
      r.v = *reinterpret_cast<const u32x4*>(q + (wave * 64 + lane) * 16);
      r.s = *reinterpret_cast<const float*>(q + SCALES + (wave * 64 + lane) * 4);
      const int32_t o = OFFSET ? *reinterpret_cast<const int32_t*>(q + SCALES + ((WAVES + wave) * 64 + lane) * 4) : 0;
      r.o = (float)(o - 128);
      // rows past the end count as 0 (whatever scale the last one has)
      if (s == n - 1 && k0 + (int64_t)s * 64 + kr >= g.krows) {
        r.v = u32x4{0u, 0u, 0u, 0u};
        r.s = 0.0f;
        r.o = -128.0f;
      }
      return r;
    };
    auto xor_group = [](int k) { return TA == 64 ? 0 : ((k >> 3) & 1) << 2; };
    auto xor_piece = [](int k) { return TA == 64 ? ((k >> 1) & 1) | ((k >> 2) & 2) : k & 3; };
    const int at_w = kr * (TA * 2) + ((p ^ xor_group(kr)) << 5) + (xor_piece(kr) << 3);
    // piece f of this lane's 16 columns
    auto write_piece = [&](const Raw& r, int f, int panel) {
      // a byte with its sign bit flipped is the code + 128 (one conversion
      // each); r.o has the 128 taken off, so the sum is exact
      const uint32_t u = r.v[f] ^ 0x80808080u;
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = r.s * ((float)((u >> (8 * e)) & 0xffu) + r.o);
      *reinterpret_cast<uint2*>(lds + panel * APANEL + (at_w ^ (f << 3))) =
          make_uint2(bf16_of(x[0]) | (bf16_of(x[1]) << 16), bf16_of(x[2]) | (bf16_of(x[3]) << 16));
    };
    const int row = lane & 15;
    const int tr = 8 * (lane >> 4) + (row >> 2);
    const int at_r = tr * (TA * 2) + (((wave / WB) * 4 ^ xor_group(tr)) << 5) + ((row & 3) << 5) + (xor_piece(tr) << 3);
    int ub = 0, panel = 0;  // B's slot and A's panel of the stage being read
    // fragment q of step h of that stage: B's, then A's
    auto fetch = [&](int h, int q, Frags& f) {
      if (q < FB) {
        f.b[q] = pb.fetch(lds + B0 + ub * BSTAGE, h, q);
      } else {
        const unsigned char* a = lds + panel * APANEL + h * (32 * TA * 2) + (at_r ^ ((q - FB) << 3));
        const nt_short4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((nt_lds_short4*)a);
        const nt_short4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((nt_lds_short4*)(a + 4 * (TA * 2)));
        f.a[q - FB] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    };
    auto up = [](int slot) { return slot + 1 == RB ? 0 : slot + 1; };
    auto fetch_all = [&](int h, Frags& f) {
#pragma unroll
      for (int q = 0; q < FA + FB; ++q) fetch(h, q, f);
    };
    auto multiply = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = NtAcc<false>::mma(f.a[i], f.b[j], acc[i][j]);
    };
    // The products of one step with the reads of the next one's fragments and
    // `more(i)` between them.
    auto step = [&](const Frags& now, int h, Frags& next, auto&& more) {
#pragma unroll
      for (int i = 0; i < FA; ++i) {
#pragma unroll
        for (int q = min(i, 3) * (FA + FB) / 3; q < min(i + 1, 3) * (FA + FB) / 3; ++q) fetch(h, q, next);
#pragma unroll
        for (int j = 0; j < FB; ++j) acc[i][j] = NtAcc<false>::mma(now.a[i], now.b[j], acc[i][j]);
        more(i);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::true_type ends{};
    constexpr std::false_type inside{};
#pragma unroll
    for (int k = 0; k < RB; ++k)
      if (k < n) {
#pragma unroll
        for (int c = 0; c < COPIES; ++c) copy(k, k, c, ends);
      }
    if (n >= RB)
      nt_wait<(RB - 2) * COPIES>();
    else
      nt_wait<0>();
    Raw r = read_raw(0, 0);
#pragma unroll
    for (int f = 0; f < 4; ++f) write_piece(r, f, 0);
    if (n > 1) r = read_raw(1, 1);
    nt_wait<63, true>();
    nt_barrier();
    if (n == 1) pb.clear_tail(lds + B0);
    Frags f0, f1;
    fetch_all(0, f0);
    int s = 0, q = 0;  // q: the slot of stage s, and of stage s + RB
    // First step: the bytes of stage s + 1, in registers, become bf16 in the
    // other panel, whose last reads ended before the barrier of stage s - 1.
    // Second step: this wave's copies of stage s + 2 are in (RB - 3 younger
    // stages may be on their way) and its bytes are read; past the barrier
    // stage s + 1 can be gathered, and stage s's slots are free.
    for (; s + RB + 2 <= n; ++s) {
      nt_wait<63, true>();
      __builtin_amdgcn_sched_barrier(0);
      step(f0, 1, f1, [&](int i) { write_piece(r, i, panel ^ 1); });
      nt_wait<(RB - 3) * COPIES, true>();
      nt_barrier();
      panel ^= 1;
      ub = up(ub);
      __builtin_amdgcn_sched_barrier(0);
      r = read_raw(s + 2, up(up(q)));
      step(f1, 0, f0, [&](int i) {
#pragma unroll
        for (int c = i * COPIES / FA; c < (i + 1) * COPIES / FA; ++c) copy(s + RB, q, c, inside);
      });
      q = up(q);
    }
    for (; s < n; ++s) {
      const bool two = s < n - 1 || !half;
      if (two) fetch_all(1, f1);
      multiply(f0);
      if (s < n - 1) {
#pragma unroll
        for (int f = 0; f < 4; ++f) write_piece(r, f, panel ^ 1);
        if (s + RB - 1 < n)
          nt_wait<(RB - 3) * COPIES, true>();
        else
          nt_wait<0, true>();
        nt_barrier();
        panel ^= 1;
        ub = up(ub);
        if (s + 2 < n) r = read_raw(s + 2, up(up(q)));
        if (s + RB < n) {
#pragma unroll
          for (int c = 0; c < COPIES; ++c) copy(s + RB, q, c, ends);
        }
        q = up(q);
        if (s == n - 2) pb.clear_tail(lds + B0 + ub * BSTAGE);
        fetch_all(0, f0);
      }
      if (two) multiply(f1);
    }
  }

  // As NtTile's.
  template <typename F>
  static __device__ __forceinline__ void each(int64_t a0, int64_t b0, F&& f) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wa = wave / WB, wb = wave % WB;
#pragma unroll
    for (int j = 0; j < FB; ++j)
      f(0, j, a0 + wa * 64 + (lane >> 4) * 16, b0 + wb * (TB / WB) + j * 16 + (lane & 15));
  }
};

}  // namespace sg
