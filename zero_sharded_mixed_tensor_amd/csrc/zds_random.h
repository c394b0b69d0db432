// Random numbers from a counter: Philox4x32-10 (Salmon, Moraes, Dror, Shaw:
// "Parallel random numbers: as easy as 1, 2, 3", 2011). Ten rounds of two
// 32 x 32 -> 64 bit products on a 128-bit counter under a 64-bit key that is
// raised by a constant in each round. A call is 20 products and 20 three-way
// exclusive ors (one instruction each); the keys are the same on every lane and
// stay in scalar registers.
#pragma once

#include <cstdint>

#include "zds_scalar.h"

namespace zds {

// The counter's last word: which use of the generator the numbers are for.
constexpr uint32_t kStreamRounding = 1, kStreamDropout = 2;

struct RandomWords {
  uint32_t w[4];
};

ZDS_HD inline uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);
#else
  return a ^ b ^ c;
#endif
}

ZDS_HD inline RandomWords random_words(uint64_t seed, uint64_t call, uint32_t steps_seen, uint32_t stream) {
  uint32_t c0 = static_cast<uint32_t>(call), c1 = static_cast<uint32_t>(call >> 32), c2 = steps_seen, c3 = stream;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = xor3(static_cast<uint32_t>(p1 >> 32), c1, k0);
    c1 = static_cast<uint32_t>(p1);
    c2 = xor3(static_cast<uint32_t>(p0 >> 32), c3, k1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return RandomWords{{c0, c1, c2, c3}};
}

}  // namespace zds
