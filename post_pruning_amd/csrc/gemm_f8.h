// Products of two matrices in 8-bit floating point whose rows both run along
// the contraction, with a scale for every 128 of it:
//   out[b][a] = epilogue( sum_k A[a][k] 2^ea[k/128][a] B[b][k] 2^eb[k/128][b] )
// A is e4m3, B e4m3 or e5m2.  A's rows are the MFMA's rows, so a lane ends up
// with neighbouring outputs of one row of `out`.
#pragma once

#include "dropout.h"
#include "gemm_nt.h"

namespace sg {

struct F8Args {
  // A, B, na, nb, lda, ldb, out, out_dtype, ldo, mask, accumulate; kbytes a
  // multiple of 128, zero-padded in both operands
  NtArgs g;
  const uint8_t *a_scale, *b_scale;  // bytes e + 127, [kbytes / 128] rows of a_lds and b_lds bytes
  int64_t a_lds, b_lds;
  int has_drop;  // dropout of the outputs, of which the first row is row0 of the whole
  int64_t row0;
  DropArgs drop;
};

typedef int f8_frag __attribute__((ext_vector_type(8)));  // 32 codes of a row: 16-byte pieces p and p + 4 of 128 bytes

// Exact products with fp32 sums: the codes are widened to bf16, which holds them
// and their block's scale exactly (values below 2^-126 to a multiple of 2^-133).  `scale`: the
// float whose exponent is the scale byte.
//
// The matrix instruction for 8-bit floating point, which bf16 outputs use, holds partial
// sums in fewer bits: it cuts every eight neighbours of the contraction toward zero
// to multiples of 2^(E - 13), E the largest sum of exponents of two codes (subnormal ones
// at the least exponent) whose product is not zero; the sums of the eights are added in the
// width of fp32.
// Measured with single products, and on whole results: 1.5e-5 to 7e-5 of their norm for
// normal and lognormal inputs (bf16's rounding: 1.7e-3; with it 1.65919e-3 instead of
// 1.65891e-3 at 8192 x 4096 x 11008), a bias of 3e-6 toward zero where every product is positive.  For
// that it runs at twice the rate: 8192 x 4096 x 4096 in about 111 us, widened 222.
struct F8Wide {
  bf16x8 v[4];
};
template <bool E5>
__device__ __forceinline__ F8Wide f8_widen(const f8_frag& f, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  F8Wide w;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    bf16x2 lo, hi;
    if constexpr (E5) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f[q], scale, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((uint32_t)f[q], scale, true);
    } else {
      lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[q], scale, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)f[q], scale, true);
    }
    const int at = 4 * (q & 1);
    w.v[q >> 1][at] = lo[0];
    w.v[q >> 1][at + 1] = lo[1];
    w.v[q >> 1][at + 2] = hi[0];
    w.v[q >> 1][at + 3] = hi[1];
  }
  return w;
}
// Byte I of a word of scale bytes as such a float.
template <int I>
__device__ __forceinline__ float f8_scale_float(uint32_t word) {
  constexpr int UP = I < 3 ? 23 - 8 * I : 0;
  return __uint_as_float((I < 3 ? word << UP : word >> 1) & 0x7f800000u);
}
// The products of a widened row fragment of A with N of B, four accumulations
// each; those of different fragments between them hide one's latency.
template <int N>
__device__ __forceinline__ void f8_dot_wide(const F8Wide& a, const F8Wide (&b)[N], floatx4 (&acc)[N]) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[q], b[j].v[q], acc[j], 0, 0, 0);
}

// Dropout of N neighbouring outputs of row b from column a on (a a multiple of 4).
template <int N, typename V4>
__device__ __forceinline__ void f8_drop(const F8Args& f, const DropKey& key, int64_t a, int64_t b, V4 (&v)[N / 4]) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const u32x4 w = drop_words(key, (uint32_t)(f.row0 + b), (uint32_t)(a >> 2) + q);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[q][e] = w[e] >= f.drop.threshold ? v[q][e] * f.drop.grow : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Tiles in LDS
// ---------------------------------------------------------------------------

// One LDS-DMA copy of 4 bytes a lane (see nt_copy16).
__device__ __forceinline__ void f8_copy4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}

// A tile of TA rows of A by TB rows of B, WA x WB waves, each with FA x FB
// fragments of 16 x 16 sums.  A stage is 128 of the contraction, one MFMA step:
// TA + TB rows of 128 bytes and their scale bytes.  R stages rotate through LDS.
//
// In LDS rows lie 128 bytes apart, 16-byte piece p of row r at piece p ^ sw(r), so
// that the 16 lanes of a read that take one piece of 16 rows touch every bank
// once (no conflicts measured).  Fragment f of a 64-row group of A takes rows 16 (i / 4) + 4 f + i % 4, i = 0
// .. 15 (a lane then ends up with 16 neighbouring outputs over the four
// fragments), sw = 2 ((r >> 4) & 3) + ((r >> 1) & 1); fragment j of B rows 16 j + i,
// sw = (r >> 1) & 7.  The matrix instruction takes the scale of lane i's row
// from one byte of a register: the four of a group are gathered into one.
//
// 256 x 256 (2 x 4 waves, R = 2: all that LDS holds) is for many tiles: 8192 x 4096 x
// 11008 in 300-324 us, 2.28-2.46 PFLOP/s, matrix cores busy for two thirds of the CUs'
// busy cycles at 1.95 GHz.  The chip's power bounds it: in timing copies of it (8192 x
// 11008 x 4096) the products alone take 205 us at 2.1 GHz, with the LDS reads 230, with
// copies from one row 246, from a hot L2 257, all 277.
// The smaller ones are for fewer tiles than CUs; a 64 x 64 stage is a chain of LDS reads and
// barriers (8.5 us for eight stages; without any copy 13.5 of 14 us for 32), which deeper
// rings and fragments read a stage ahead did not shorten.  WIDE multiplies four times as
// many instructions of half the length: 8192 x 4096 x 4096 in 222-230 us, 1.2 PFLOP/s.
template <bool WIDE_, bool E5_, int TA_, int TB_, int WA_, int WB_, int R_>
struct F8Tile {
  static constexpr bool WIDE = WIDE_, E5 = E5_;
  static constexpr int TA = TA_, TB = TB_, WA = WA_, WB = WB_, R = R_;
  static constexpr int WAVES = WA * WB, THREADS = 64 * WAVES;
  static constexpr int FA = TA / WA / 16, FB = TB / WB / 16, GA = FA / 4;
  static constexpr int ASTAGE = TA * 128, BSTAGE = TB * 128, STAGE = ASTAGE + BSTAGE;
  // scale bytes behind the stages: every wave copies those of 64 rows to a piece of its own
  static constexpr int SCALES = R * STAGE, SSTAGE = WAVES * 256;
  static constexpr int LDS = SCALES + R * SSTAGE;
  static constexpr int CA = TA / 8 / WAVES, CB = TB / 8 / WAVES;  // copy instructions of a wave and stage
  static constexpr int COPIES = 1 + CA + CB;
  static constexpr bool SAME_A = CA == 1 || WAVES % 8 == 0, SAME_B = CB == 1 || WAVES % 2 == 0;
  static_assert(FA % 4 == 0 && FB >= 1 && FB <= 4 && CA >= 1 && CB >= 1 && SAME_B, "tile shape");
  static_assert(TA % 64 == 0 && TB % 64 == 0 && TA + TB <= 64 * WAVES && LDS <= 160 * 1024, "stages");
  static_assert((R - 1) * COPIES < 64, "the copies on their way are counted in 6 bits");

  const F8Args& p;
  unsigned char* const lds;
  const int lane, wave;
  uint32_t lds0;
  int64_t a0, b0;
  int s0, n;  // first stage, stages
  const unsigned char *base_a, *base_b;
  const uint8_t* base_s;  // the scales that this wave copies
  int64_t pitch_s;
  uint32_t row_a, row_b, piece_a[SAME_A ? 1 : CA], piece_b;  // byte offset of this lane's row of copy 0, and of its piece
  uint32_t last_a, last_b, step_a, step_b;  // offset of the operand's last row of the tile; of a copy's rows from the next's
  uint32_t off_s;
  int at_a, at_b, at_ea, at_eb;

  __device__ __forceinline__ F8Tile(const F8Args& p_, unsigned char* lds_, int64_t a0_, int64_t b0_, int s0_, int n_)
      : p(p_), lds(lds_), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6))),
        a0(a0_), b0(b0_), s0(s0_), n(n_) {
    lds0 = (uint32_t)(uintptr_t)(nt_lds_void*)lds;
    base_a = p.g.A + a0 * p.g.lda + (int64_t)s0 * 128;
    base_b = p.g.B + b0 * p.g.ldb + (int64_t)s0 * 128;
    // Copy k of a wave takes rows 8 (WAVES k + wave) on: with eight waves a lane's
    // piece is the same for all k.  Rows past an operand's end re-read its last one; their
    // sums are not stored.
    const int r = wave * 8 + (lane >> 3);
    row_a = (uint32_t)(r * p.g.lda);
    row_b = (uint32_t)(r * p.g.ldb);
#pragma unroll
    for (int k = 0; k < (SAME_A ? 1 : CA); ++k) {
      const int rk = r + 8 * WAVES * k;
      piece_a[k] = ((lane & 7) ^ (2 * ((rk >> 4) & 3) + ((rk >> 1) & 1))) * 16;
    }
    piece_b = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
    last_a = (uint32_t)((min<int64_t>(TA, p.g.na - a0) - 1) * p.g.lda);
    last_b = (uint32_t)((min<int64_t>(TB, p.g.nb - b0) - 1) * p.g.ldb);
    step_a = (uint32_t)(8 * WAVES * p.g.lda);
    step_b = (uint32_t)(8 * WAVES * p.g.ldb);
    // Scales: four bytes in each of the first 16 lanes, the others repeat them; rows
    // of scales are padded to 16.
    const int chunk = min(wave, (TA + TB) / 64 - 1);
    const bool of_b = chunk >= TA / 64;
    const int64_t first = of_b ? b0 + 64 * (chunk - TA / 64) : a0 + 64 * chunk;
    const int64_t rows = of_b ? p.g.nb : p.g.na;
    pitch_s = of_b ? p.b_lds : p.a_lds;
    base_s = (of_b ? p.b_scale : p.a_scale) + s0 * pitch_s;
    off_s = (uint32_t)min<int64_t>(first + (lane & 15) * 4, (rows - 1) & ~(int64_t)3);
    const int i = lane & 15, g = lane >> 4;
    at_a = (wave / WB) * (TA / WA) * 128 + ((i >> 2) * 16 + (i & 3)) * 128 + ((g ^ (2 * (i >> 2) + ((i >> 1) & 1))) << 4);
    at_b = ASTAGE + ((wave % WB) * (TB / WB) + i) * 128 + ((g ^ ((i >> 1) & 7)) << 4);
    // (pieces p and p + 4: bit 6 of the offset flips)
    at_ea = (wave / WB) * (TA / WA) * 4 + 16 * (i >> 2);
    const int rb = (wave % WB) * (TB / WB);
    at_eb = TA * 4 + (rb >> 6) * 256 + (rb & 63) + i;
  }

  // Copy k of stage s to its slot: the scales come first.
  __device__ __forceinline__ void copy(int s, int slot, int k) const {
    const uint32_t to = lds0 + (uint32_t)(slot * STAGE);
    if (k == 0)
      f8_copy4(base_s + s * pitch_s, off_s,
               __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(SCALES + slot * SSTAGE + wave * 256)));
    else if (k <= CA)
      nt_copy16(base_a + (int64_t)s * 128, min(row_a + (k - 1) * step_a, last_a) + piece_a[SAME_A ? 0 : k - 1],
                __builtin_amdgcn_readfirstlane(to + (uint32_t)((WAVES * (k - 1) + wave) * 1024)));
    else
      nt_copy16(base_b + (int64_t)s * 128, min(row_b + (k - 1 - CA) * step_b, last_b) + piece_b,
                __builtin_amdgcn_readfirstlane(to + (uint32_t)(ASTAGE + (WAVES * (k - 1 - CA) + wave) * 1024)));
  }
  // Waits until at most LEFT copies of this wave are on their way and its LDS reads
  // have returned.
  template <int LEFT>
  static __device__ __forceinline__ void arrive() {
    nt_wait<LEFT, true>();
  }

  __device__ __forceinline__ f8_frag read(int at, int add) const {
    const u32x4 lo = *reinterpret_cast<const u32x4*>(lds + at + add), hi = *reinterpret_cast<const u32x4*>(lds + (at ^ 64) + add);
    return f8_frag{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }
  static __device__ __forceinline__ int up(int slot) { return slot + 1 == R ? 0 : slot + 1; }

  __device__ __forceinline__ void first_copies() const {
#pragma unroll
    for (int s = 0; s < R; ++s)
      if (s < n) {
#pragma unroll
        for (int k = 0; k < COPIES; ++k) copy(s, s, k);
      }
    if (n >= R)
      arrive<(R - 1) * COPIES>();
    else
      arrive<0>();
    nt_barrier();
  }

  // Copies wait on their latency, so they are issued as early as their slot allows.
  // Waves with two 64-row groups have B's fragments, the first group's and all
  // scales in registers after the first pair of rows: what replaces them is copied
  // from then on (the scales, every second copy of A, all of B), the second group's from the last pair on.
  static constexpr int EARLY = GA == 2 ? 1 + CA / 2 + CB : 0;
  static_assert(GA == 1 || (CA % 2 == 0 && WAVES == 8), "a copy of A is of one 64-row group");
  static constexpr int early(int k) { return k == 0 ? 0 : k <= CA / 2 ? 2 * k - 1 : k + CA / 2; }
  static constexpr int late(int k) { return GA == 2 ? 2 * k + 2 : k; }

  // Sums of the tile's stages.  The products go by pairs of rows of fragments: the
  // next pair's fragments of A are read meanwhile, and under the last pair the
  // next stage's of B, each when its predecessor's last product has been issued (two
  // whole sets of fragments beside 128 sums would not fit).  From the last pair
  // on, reads are of the next stage, and this one's slot is free for the copies of
  // the stage R on.
  //
  // A loop's body is one block of code without branches: the compiler would move
  // products, which touch no memory, across them.
  __device__ __forceinline__ void run(floatx4 (&acc)[FA][FB]) const {
    if (n <= 0) return;
    first_copies();
    f8_frag fa[4], fb[FB];
    uint32_t ea[GA], eb;
    u32x4 raw_a[GA];
    F8Wide wb[WIDE ? FB : 1];
    // Scales of 64-row group h of A as they are read: byte i % 4 of word f for lane i's row
    // of fragment f; packed, byte f of one word, as the matrix instruction takes them.  Read
    // early and packed late, so that the packing does not wait.
    auto read_a = [&](int slot, int h) {
      raw_a[h] = *reinterpret_cast<const u32x4*>(lds + at_ea + (SCALES + slot * SSTAGE + h * 256));
    };
    auto pack_a = [&](int h) {
      const uint32_t sh = (lane & 3) * 8;
      const u32x4 w = raw_a[h] >> sh;
      ea[h] = (w[0] & 255u) | ((w[1] & 255u) << 8) | ((w[2] & 255u) << 16) | (w[3] << 24);
    };
    uint32_t raw_b[FB];
    auto read_b = [&](int slot) {
      const unsigned char* e = lds + at_eb + (SCALES + slot * SSTAGE);
#pragma unroll
      for (int j = 0; j < FB; ++j) raw_b[j] = e[16 * j];
    };
    auto pack_b = [&]() {  // byte j: row 16 j + lane % 16
      eb = raw_b[0];
#pragma unroll
      for (int j = 1; j < FB; ++j) eb |= raw_b[j] << (8 * j);
    };
    auto frag_a = [&](int slot, int i) { return read(at_a, slot * STAGE + (i >> 2) * 8192 + (i & 3) * 512); };
    auto frag_b = [&](int slot, int j) { return read(at_b, slot * STAGE + j * 2048); };
    read_a(0, 0);
    read_b(0);
    pack_a(0);
    pack_b();
#pragma unroll
    for (int j = 0; j < FB; ++j) fb[j] = frag_b(0, j);
    fa[0] = frag_a(0, 0);
    fa[1] = frag_a(0, 1);
    int s = 0, slot = 0;
    auto stage = [&](auto more) {
      constexpr bool MORE = decltype(more)::value;  // the stage R on is copied
      const int ahead = up(slot);
      if constexpr (WIDE) {
        each<FB>([&](auto jq) {
          constexpr int J = decltype(jq)::value;
          wb[J] = f8_widen<E5>(fb[J], f8_scale_float<J>(eb));
        });
      }
      auto pair = [&](auto iq) {
        constexpr int I = decltype(iq)::value, G = I >> 2;
        constexpr bool LAST = I == FA - 2;
        if constexpr (LAST) {
          // every wave has read this stage, and its copies of the next are in
          arrive<MORE ? (R - 2) * COPIES + EARLY : 0>();
          nt_barrier();
          __builtin_amdgcn_sched_barrier(0);
          read_b(ahead);
          read_a(ahead, 0);
        } else if constexpr (GA == 2 && I == 0) {
          read_a(slot, 1);
        }
        if constexpr (MORE && GA == 2 && I == 2) {
          // every wave has read what the early copies replace
          nt_wait<63, true>();
          nt_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        const int from = LAST ? ahead : slot;
        constexpr int NEXT = LAST ? 0 : I + 2;
        fa[NEXT & 3] = frag_a(from, NEXT);
        if constexpr (WIDE && LAST) {
#pragma unroll
          for (int j = 0; j < FB; ++j) fb[j] = frag_b(ahead, j);
        }
        // (the copies of what follows go between the products)
        auto copies = [&](int part, int parts) {
          if constexpr (MORE && LAST) {
#pragma unroll
            for (int k = part * (COPIES - EARLY) / parts; k < (part + 1) * (COPIES - EARLY) / parts; ++k)
              copy(s + R, slot, late(k));
          }
          if constexpr (MORE && GA == 2 && I == 2) {
#pragma unroll
            for (int k = part * EARLY / parts; k < (part + 1) * EARLY / parts; ++k) copy(s + R, slot, early(k));
          }
        };
        if constexpr (WIDE) {
          f8_dot_wide<FB>(f8_widen<false>(fa[I & 3], f8_scale_float<I & 3>(ea[G])), wb, acc[I]);
          fa[(NEXT + 1) & 3] = frag_a(from, NEXT + 1);
          copies(0, 2);
          __builtin_amdgcn_sched_barrier(0);
          f8_dot_wide<FB>(f8_widen<false>(fa[(I + 1) & 3], f8_scale_float<(I + 1) & 3>(ea[G])), wb, acc[I + 1]);
          copies(1, 2);
          __builtin_amdgcn_sched_barrier(0);
        } else {
          each<FB>([&](auto jq) {
            constexpr int J = decltype(jq)::value;
            product<I, J>(fa[I & 3], fb[J], ea[G], eb, acc[I][J]);
            if constexpr (J == 0) fa[(NEXT + 1) & 3] = frag_a(from, NEXT + 1);
            product<I + 1, J>(fa[(I + 1) & 3], fb[J], ea[G], eb, acc[I + 1][J]);
            if constexpr (LAST) fb[J] = frag_b(ahead, J);
            copies(J, FB);
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        if constexpr (GA == 2 && I == 2) pack_a(1);
        if constexpr (LAST) {
          pack_a(0);
          pack_b();
        }
      };
      each<FA / 2>([&](auto iq) { pair(std::integral_constant<int, 2 * decltype(iq)::value>{}); });
      slot = ahead;
      ++s;
    };
    while (s + R < n) stage(std::true_type{});
    while (s < n) stage(std::false_type{});  // (after the last stage what is read is not used)
  }
  template <int N, int I = 0, typename F>
  static __device__ __forceinline__ void each(F&& f) {
    if constexpr (I < N) {
      f(std::integral_constant<int, I>{});
      each<N, I + 1>(f);
    }
  }
  template <int I, int J>
  static __device__ __forceinline__ void product(const f8_frag& a, const f8_frag& b, uint32_t ea, uint32_t eb,
                                                 floatx4& acc) {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, E5 ? 1 : 0, I & 3, (int)ea, J, (int)eb);
  }

  // Item q of the wave: this lane's sums acc[4 h .. 4 h + 3][j], h = q / FB, j = q % FB, are
  // those of 16 neighbouring columns from a on of row b.
  static constexpr int ITEMS = GA * FB;
  static __device__ __forceinline__ void item(int64_t a0, int64_t b0, int q, int64_t& a, int64_t& b) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    a = a0 + (wave / WB) * (TA / WA) + (q / FB) * 64 + (lane >> 4) * 16;
    b = b0 + (wave % WB) * (TB / WB) + (q % FB) * 16 + (lane & 15);
  }
};

// Which of 16 neighbouring outputs of row b from column a on a dropout keeps.
__device__ __forceinline__ uint32_t f8_kept16(const F8Args& p, const DropKey& key, int64_t a, int64_t b) {
  uint32_t bits = 0u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const u32x4 w = drop_words(key, (uint32_t)(p.row0 + b), (uint32_t)(a >> 2) + q);
#pragma unroll
    for (int e = 0; e < 4; ++e) bits |= w[e] >= p.drop.threshold ? 1u << (4 * q + e) : 0u;
  }
  return bits;
}
// The bits of all items of a lane, 16 each, the first lowest.  A rolled loop: the
// generator's code unrolled over eight items would keep the sums from their registers.
template <typename Tile>
struct F8Kept {
  static constexpr int WORDS = (Tile::ITEMS + 1) / 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ void make(const F8Args& p, const DropKey& key, int64_t a0, int64_t b0) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
#pragma unroll 1
    for (int q = 0; q < 2 * WORDS; ++q) {
      int64_t a, b;
      Tile::item(a0, b0, q, a, b);
      const uint32_t bits = q < Tile::ITEMS ? f8_kept16(p, key, a, b) : 0u;
#pragma unroll
      for (int i = 0; i + 1 < WORDS; ++i) w[i] = (w[i] >> 16) | (w[i + 1] << 16);
      w[WORDS - 1] = (w[WORDS - 1] >> 16) | (bits << 16);
    }
  }
  __device__ __forceinline__ uint32_t of(int q) const { return w[q >> 1] >> (16 * (q & 1)); }
};
__device__ __forceinline__ void f8_drop16(const F8Args& p, uint32_t bits, floatx4 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e >> 2][e & 3] = (bits >> e) & 1u ? v[e >> 2][e & 3] * p.drop.grow : 0.0f;
}

// Four lanes of a quad trade what they hold: v[f] of lane r becomes v[r] of lane f.
__device__ __forceinline__ float f8_xor(float v, std::integral_constant<int, 1>) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 0xf, 0xf, false));  // quad_perm 1, 0, 3, 2
}
__device__ __forceinline__ float f8_xor(float v, std::integral_constant<int, 2>) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4e, 0xf, 0xf, false));  // quad_perm 2, 3, 0, 1
}
template <int BIT>
__device__ __forceinline__ void f8_trade(floatx4& low, floatx4& high) {
  const bool up = threadIdx.x & BIT;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float got = f8_xor(up ? low[e] : high[e], std::integral_constant<int, BIT>{});
    low[e] = up ? got : low[e];
    high[e] = up ? high[e] : got;
  }
}

// 16 neighbouring outputs of row b from column a on (those inside the matrix):
// mask, accumulation, type.  Rows of `out` and of the mask may lie at any address.
// All lanes of a quad come here with the same a and with neighbouring rows.
//
// In fp32 a lane's 16 are four stores 16 bytes wide; they are traded within the
// quad first, so that neighbouring lanes write neighbouring pieces of a row (4096 x
// 4096 from 512 tokens 30 us, 32 with a mask; untraded 43).  bf16 has two stores a
// lane, where trading gains nothing (16.8 and 16.6 us, masked 19.1 and 19.6).
__device__ __forceinline__ void f8_store16(const NtArgs& g, int64_t a, int64_t b, const floatx4 (&v)[4]) {
  if (a >= g.na) return;
  const int cnt = (int)min<int64_t>(g.na - a, 16);
  const bool add = g.accumulate, row = b < g.nb;
  floatx4 o[4] = {v[0], v[1], v[2], v[3]};
  if (g.mask && row) {
    const uint8_t* m = g.mask + b * g.na + a;
    u32x4 w = u32x4{0u, 0u, 0u, 0u};
    if (cnt == 16) {
      w = *reinterpret_cast<const u32x4_bytes*>(m);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < cnt) w[i >> 2] |= (uint32_t)m[i] << (8 * (i & 3));
    }
    const float none = nt_pruned<EP_MASKED>(g);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((w[i >> 2] >> (8 * (i & 3))) & 255u) o[i >> 2][i & 3] = none;
  }
  if (g.out_dtype == SG_F32) {
    if (cnt == 16) {
      f8_trade<1>(o[0], o[1]);
      f8_trade<1>(o[2], o[3]);
      f8_trade<2>(o[0], o[2]);
      f8_trade<2>(o[1], o[3]);
      const int r = threadIdx.x & 3;
      const int64_t rows = g.nb - (b - r);
      if (rows <= 0) return;
      float* p = static_cast<float*>(g.out) + (b - r) * g.ldo + a + 4 * r;
      if (add) {  // (all loads ahead of the stores; rows past the last re-read it)
        u32x4 w[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) w[f] = *reinterpret_cast<const u32x4_any*>(p + min<int64_t>(f, rows - 1) * g.ldo);
#pragma unroll
        for (int f = 0; f < 4; ++f) o[f] += __builtin_bit_cast(floatx4, w[f]);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (f < rows) *reinterpret_cast<u32x4_any*>(p + f * g.ldo) = __builtin_bit_cast(u32x4, o[f]);
    } else if (row) {
      float* p = static_cast<float*>(g.out) + b * g.ldo + a;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < cnt) p[i] = add ? p[i] + o[i >> 2][i & 3] : o[i >> 2][i & 3];
    }
    return;
  }
  if (!row) return;
  uint16_t* p = static_cast<uint16_t*>(g.out) + b * g.ldo + a;
  if (cnt == 16) {
    if (add) {
      const u32x4 w[2] = {*reinterpret_cast<const u32x4_any*>(p), *reinterpret_cast<const u32x4_any*>(p + 8)};
#pragma unroll
      for (int k = 0; k < 16; ++k)
        o[k >> 2][k & 3] += __uint_as_float(k & 1 ? w[k >> 3][(k >> 1) & 3] & 0xffff0000u : w[k >> 3][(k >> 1) & 3] << 16);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = bf16_of(o[2 * h + (k >> 1)][2 * (k & 1)]) | (bf16_of(o[2 * h + (k >> 1)][2 * (k & 1) + 1]) << 16);
      *reinterpret_cast<u32x4_any*>(p + 8 * h) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < cnt) p[i] = (uint16_t)bf16_of(add ? bf16_to_f32(p[i]) + o[i >> 2][i & 3] : o[i >> 2][i & 3]);
  }
}

}  // namespace sg
