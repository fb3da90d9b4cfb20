// The Philox4x32-10 counter-based generator (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC'11).  The fourth counter
// word tells the library's users of one key apart: 0 for the low-bit
// messages' stochastic rounding, 1 for dropout.
#pragma once

#include "common.h"

namespace sag {

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
    return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);   // the truth table of a ^ b ^ c
}

// Philox4x32 with 10 rounds: c is the counter in and the block out.  Each
// round's two 32 x 32 -> 64-bit products are taken whole, so one
// instruction gives both halves of each, and each pair of exclusive ors is
// one.
__device__ __forceinline__ void philox4x32_10(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(kPhiloxM0) * c[0];
        const uint64_t p1 = static_cast<uint64_t>(kPhiloxM1) * c[2];
        const uint32_t n0 = xor3(static_cast<uint32_t>(p1 >> 32), c[1], k0);
        const uint32_t n2 = xor3(static_cast<uint32_t>(p0 >> 32), c[3], k1);
        c[0] = n0;
        c[1] = static_cast<uint32_t>(p1);
        c[2] = n2;
        c[3] = static_cast<uint32_t>(p0);
        k0 += kPhiloxW0;
        k1 += kPhiloxW1;
    }
}

}  // namespace sag
