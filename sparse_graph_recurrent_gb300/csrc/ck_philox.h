// The counter-based generator of dropout and of token sampling: Philox-4x32
// with 10 rounds, from its published definition (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011, section 3.3 and
// table 2).  A 128-bit counter and a 64-bit key give four 32-bit words; here
// the key is the caller's seed, the counter's low half the element's index
// divided by four and its high half the caller's step, so that every (seed,
// step) is a stream of its own and an element's word can be found again
// without anything stored.
#pragma once

#include <stdint.h>

namespace ck {

struct PhiloxKey {
    uint32_t k0, k1;    // seed, low and high word
    uint32_t c2, c3;    // step, low and high word
};

__device__ __forceinline__ uint4 philox(uint64_t block, const PhiloxKey &key) {
    uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = key.c2, d = key.c3;
    uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        const uint64_t x = (uint64_t)a * 0xD2511F53u, y = (uint64_t)c * 0xCD9E8D57u;
        const uint32_t na = (uint32_t)(y >> 32) ^ b ^ k0, nc = (uint32_t)(x >> 32) ^ d ^ k1;
        b = (uint32_t)y;
        d = (uint32_t)x;
        a = na;
        c = nc;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(a, b, c, d);
}

// The key of (seed, step); step_dev, when given, is a device word that holds
// the step in place of `step`.
__device__ __forceinline__ PhiloxKey philox_key(uint64_t seed, uint64_t step,
                                                const int64_t *step_dev) {
    if (step_dev) step = (uint64_t)*step_dev;
    return PhiloxKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step,
                     (uint32_t)(step >> 32)};
}

}  // namespace ck
