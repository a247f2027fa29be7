// Counter-based random numbers: Philox 4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  Each
// round multiplies two of the counter's words by fixed odd constants and mixes
// the products' halves with the other two words and the key, which advances by
// Weyl constants.  Nothing is kept between calls: the words for a counter can be
// made again anywhere, so a mask needs no memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// x ^ y ^ z in one instruction.
__device__ __forceinline__ uint32_t xor3(uint32_t x, uint32_t y, uint32_t z) {
  return __builtin_amdgcn_bitop3_b32(x, y, z, 0x96);
}

struct Philox {
  uint32_t w[4];
  // 16-bit half i (0..7): the low half of each word first
  __device__ __forceinline__ unsigned half(int i) const { return i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffffu; }
};

// The four words for counter {block, step} and key {seed} (low word first).
__device__ __forceinline__ Philox philox(uint64_t block, uint64_t step, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)step, c3 = (uint32_t)(step >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    const uint32_t n0 = xor3((uint32_t)(q >> 32), c1, k0), n2 = xor3((uint32_t)(p >> 32), c3, k1);
    c1 = (uint32_t)q;
    c3 = (uint32_t)p;
    c0 = n0;
    c2 = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Philox{{c0, c1, c2, c3}};
}

}  // namespace moe
