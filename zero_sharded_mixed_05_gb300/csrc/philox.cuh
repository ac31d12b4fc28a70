// philox.cuh -- the bits of a dropout: Philox 4x32 with ten rounds (Salmon,
// Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011), a
// function of a counter and a key that keeps nothing.  Eight numbers take one
// call's 128 bits, 16 each: half the integer work of 32 bits a number, and p to
// 1.5e-5.  A call is 20 wide products, 20 exclusive ors of three words and 16 instructions
// for the comparisons: 56, or 7 a number.  Dropout alone measures 10.8 integer
// instructions a number, its addresses and masks among them, which keep the integer pipe
// 69 % busy for the 47.6 us of 67 million numbers: 33 us, next to 40 us of memory traffic.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "zero_block.h"

namespace zo {

// What a kernel needs of a dropout.
struct Drop {
  uint32_t key[10][2];        // of the rounds
  const int64_t* step_dev;
  uint32_t call, step;
  uint32_t cut;               // halves from here on are kept; 0: no dropout
  uint32_t select;            // see kept()
  float factor;               // 65536 / (65536 - cut), or 0
};

inline Drop drop_of(const zero_rng& rng, double p) {
  Drop d;
  for (uint32_t i = 0; i < 10; ++i) {
    d.key[i][0] = (uint32_t)rng.seed + i * 0x9E3779B9u;
    d.key[i][1] = (uint32_t)(rng.seed >> 32) + i * 0xBB67AE85u;
  }
  d.step_dev = rng.step_dev;
  d.call = rng.call;
  d.step = (uint32_t)rng.step;
  d.cut = (uint32_t)(65536.0 * p + 0.5);
  d.select = d.cut < 65536 ? 0xBB99 : 0x4444;
  d.factor = d.cut < 65536 ? (float)(65536.0 / (65536.0 - d.cut)) : 0.0f;
  return d;
}

__device__ __forceinline__ uint32_t step_of(const Drop& d) {
  return d.step_dev ? (uint32_t)__ldg(reinterpret_cast<const unsigned long long*>(d.step_dev)) : d.step;
}

__device__ __forceinline__ uint32_t pick_bytes(uint32_t x, uint32_t selector) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(x), "r"(selector));
  return r;
}

// For a block of eight numbers, a half of all ones for each that is kept and of
// zeros for the others: what a pair of 16-bit numbers is masked by.
__device__ __forceinline__ uint4 kept(const Drop& d, uint32_t step, int64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = d.call, c3 = step;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[i][0];
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[i][1];
    c3 = (uint32_t)a;
  }
  // Both halves against the cut at once: 15 bits by a subtraction that borrows from
  // the bit above them, which is then compared itself; that bit's byte is spread
  // over its half (where nothing is kept, zeros are picked instead).
  const uint32_t cut = d.cut * 0x10001u;
  const auto halves = [&](uint32_t w) {
    const uint32_t low = (w | 0x80008000u) - (cut & 0x7fff7fffu);
    return pick_bytes((w & ~cut) | (~(w ^ cut) & low), d.select);
  };
  return make_uint4(halves(c0), halves(c1), halves(c2), halves(c3));
}

__device__ __forceinline__ uint32_t word_of(const uint4& m, int k) {
  return k == 0 ? m.x : k == 1 ? m.y : k == 2 ? m.z : m.w;
}

// Numbers that are not kept become zero, whatever they hold.
__device__ __forceinline__ float2 masked(float2 x, uint32_t m) {
  return make_float2(__uint_as_float(__float_as_uint(x.x) & pick_bytes(m, 0x1010)),
                     __uint_as_float(__float_as_uint(x.y) & pick_bytes(m, 0x3232)));
}
__device__ __forceinline__ void mask8(float2* x, const uint4& m) {
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = masked(x[k], word_of(m, k));
}

}  // namespace zo
