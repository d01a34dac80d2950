// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw
// ("Parallel random numbers: as easy as 1, 2, 3", 2011): four 32-bit words that are
// a function of a 128-bit counter and a 64-bit key alone.
#pragma once

#include <stdint.h>

namespace mok {

// Of N counters under one key, round by round: a round waits for its products, and
// the counters share its key.
template <int N>
__device__ __forceinline__ void philox4x32_10(uint4 (&c)[N], uint2 k) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t a = static_cast<uint64_t>(c[i].x) * 0xD2511F53u;
      const uint64_t b = static_cast<uint64_t>(c[i].z) * 0xCD9E8D57u;
      c[i] = make_uint4(static_cast<uint32_t>(b >> 32) ^ c[i].y ^ k.x, static_cast<uint32_t>(b),
                        static_cast<uint32_t>(a >> 32) ^ c[i].w ^ k.y, static_cast<uint32_t>(a));
    }
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
}

}  // namespace mok
