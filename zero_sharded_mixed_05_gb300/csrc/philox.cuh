// philox.cuh -- the bits of a dropout: Philox 4x32 with ten rounds (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011), a
// function of a counter and a key that keeps nothing.  Eight numbers take one
// call's 128 bits, 16 each: half the integer work of 32 bits a number, and p to
// 1.5e-5.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "zero_block.h"

namespace zo {

// What a kernel needs of a dropout.
struct Drop {
  zero_rng rng;
  uint32_t cut;     // halves from here on are kept; 0: no dropout
  float factor;     // 65536 / (65536 - cut), or 0
};

inline Drop drop_of(const zero_rng& rng, double p) {
  Drop d;
  d.rng = rng;
  d.cut = (uint32_t)(65536.0 * p + 0.5);
  d.factor = d.cut < 65536 ? (float)(65536.0 / (65536.0 - d.cut)) : 0.0f;
  return d;
}

__device__ __forceinline__ uint32_t step_of(const Drop& d) {
  return d.rng.step_dev ? (uint32_t)__ldg(reinterpret_cast<const unsigned long long*>(d.rng.step_dev))
                        : (uint32_t)d.rng.step;
}

// Bit i is set where number i of the block of eight is kept.
__device__ __forceinline__ uint32_t kept(const Drop& d, uint32_t step, int64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = d.rng.call, c3 = step;
  uint32_t k0 = (uint32_t)d.rng.seed, k1 = (uint32_t)(d.rng.seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0xffffu) >= d.cut) bits |= 1u << 2 * i;
    if ((w[i] >> 16) >= d.cut) bits |= 2u << 2 * i;
  }
  return bits;
}

}  // namespace zo
