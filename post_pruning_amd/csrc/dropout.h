// Dropout whose numbers come from a counter.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC11): ten rounds turn a 128-bit counter and a 64-bit key into
// four 32-bit words.  Element (row, col) of a matrix takes word col % 4 of the
// counter (col / 4, row, offset) under the key `seed`, so that whoever meets the
// element again -- the gradient's epilogue, another form of the same
// activations -- makes the same number anew, whatever its pitch or tile.
#pragma once

#include "sg_internal.h"

namespace sg {

// What the kernels take of an sg_drop (sg_internal.h: DropArgs).
struct DropKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  uint64_t seed = d.seed, offset = d.offset;
  if (d.state) {  // (the same for every thread: scalar loads)
    seed += d.state[0];
    offset += d.state[1];
  }
  return DropKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)offset, (uint32_t)(offset >> 32)};
}

// a ^ b ^ c in one instruction (its truth table is 0x96).
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

__device__ __forceinline__ u32x4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                               uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = xor3((uint32_t)(b >> 32), c1, k0);
    c1 = (uint32_t)b;
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return u32x4{c0, c1, c2, c3};
}

// The words of elements (row, 4 quad) to (row, 4 quad + 3).
__device__ __forceinline__ u32x4 drop_words(const DropKey& k, uint32_t row, uint32_t quad) {
  return philox4x32_10(quad, row, k.o0, k.o1, k.k0, k.k1);
}

}  // namespace sg
