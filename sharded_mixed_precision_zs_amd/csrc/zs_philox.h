/*
 * zs_philox.h -- the random numbers of dropout (gfx950): Philox4x32 with
 * seven rounds, as published (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", 2011; seven is the fewest with which their
 * tests found nothing). A function of the seed (the key) and of a counter:
 * {column / 8, row, offset low, offset high} gives four words, sixteen bits
 * for each of eight neighbouring elements. So a mask is formed again where it
 * is needed and never stored, and is the same whatever the launch.
 *
 * A round is two 32 x 32 bit products; one vector of eight costs some 90
 * instruction slots, a third of what HBM leaves time for at 16 bits an
 * element in and out.
 */
#ifndef ZS_PHILOX_H
#define ZS_PHILOX_H

#include "zs_mx.h"

namespace zs {

struct DropArgs {
  const uint64_t *dev_offset;   /* optional, added to `offset` when the kernel runs */
  uint64_t offset;
  uint32_t key[2];
  uint32_t threshold;           /* of 65536 numbers, how many drop; 0: no dropout */
  float factor;                 /* 65536 / (65536 - threshold); 0 if nothing is kept */
  double factor64;
};

struct RandomWords {
  uint32_t w[4];
};

/* A counter's upper half: the same for a whole launch. */
__device__ __forceinline__ uint64_t drop_offset(const DropArgs &d) {
  return d.offset + (d.dev_offset ? *d.dev_offset : 0);
}

/* a ^ b ^ c in one instruction */
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return (uint32_t)__builtin_amdgcn_bitop3_b32((int)a, (int)b, (int)c, 0x96);
}

__device__ __forceinline__ RandomWords random_words(const DropArgs &d, uint64_t offset,
                                                    uint32_t block, uint32_t row) {
  uint32_t c0 = block, c1 = row, c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = d.key[0], k1 = d.key[1];
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = xor3((uint32_t)(b >> 32), c1, k0);
    c1 = (uint32_t)b;
    c2 = xor3((uint32_t)(a >> 32), c3, k1);
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return RandomWords{{c0, c1, c2, c3}};
}

/* Whether element j of the eight stays, where something may be dropped: its
 * bits are not below the threshold, compared as 16-bit numbers. */
__device__ __forceinline__ bool kept(const RandomWords &r, int j, uint32_t threshold) {
  const uint32_t w = r.w[j / 2];
  return (uint16_t)(j & 1 ? w >> 16 : w) > (uint16_t)(threshold - 1);
}

}  // namespace zs
#endif  // ZS_PHILOX_H
