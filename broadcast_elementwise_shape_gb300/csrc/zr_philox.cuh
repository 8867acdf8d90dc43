// zr_philox.cuh — the counter-based generator Philox4x32-10 (J. K. Salmon,
// M. A. Moraes, R. O. Dror and D. E. Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", SC 2011).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace zr {

// The key's schedule (the paper's Weyl constants added from round to round) is
// the same for every element, so the host computes it.
inline void philox_keys(uint64_t seed, uint32_t* key) {
  uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
  for (int r = 0; r < 10; ++r, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    key[2 * r] = k0;
    key[2 * r + 1] = k1;
  }
}

// The four words of counter (c0, c1, c2, c3): ten rounds of two 32 x 32 -> 64
// multiplications.
__device__ __forceinline__ void philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                       const uint32_t* key, uint32_t* w) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
    c0 = uint32_t(b >> 32) ^ c1 ^ key[2 * r];
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ key[2 * r + 1];
    c3 = uint32_t(a);
  }
  w[0] = c0; w[1] = c1; w[2] = c2; w[3] = c3;
}

}  // namespace zr
