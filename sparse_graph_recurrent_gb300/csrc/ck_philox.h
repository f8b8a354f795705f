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

struct PhiloxKeys {
    uint32_t k[10][2];  // the keys of the ten rounds: the seed, moved on by two constants
    uint64_t step;
    const int64_t *step_dev;  // when given, a device word that holds the step
    static PhiloxKeys of(uint64_t seed, uint64_t step, const int64_t *step_dev) {
        PhiloxKeys p{};
        for (int i = 0; i < 10; ++i) {
            p.k[i][0] = (uint32_t)seed + (uint32_t)i * 0x9E3779B9u;
            p.k[i][1] = (uint32_t)(seed >> 32) + (uint32_t)i * 0xBB67AE85u;
        }
        p.step = step;
        p.step_dev = step_dev;
        return p;
    }
    __device__ __forceinline__ uint64_t at() const { return step_dev ? (uint64_t)*step_dev : step; }
};

// Rounds `from` to 9.  `keys` is a kernel's argument: its words then are operands
// from constant memory.
template <int from>
__device__ __forceinline__ uint4 philox_rounds(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                               const PhiloxKeys &keys) {
#pragma unroll
    for (int round = from; round < 10; ++round) {
        const uint64_t x = (uint64_t)a * 0xD2511F53u, y = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(y >> 32) ^ b ^ keys.k[round][0];
        c = (uint32_t)(x >> 32) ^ d ^ keys.k[round][1];
        b = (uint32_t)y;
        d = (uint32_t)x;
    }
    return make_uint4(a, b, c, d);
}

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t step, const PhiloxKeys &keys) {
    return philox_rounds<0>((uint32_t)block, (uint32_t)(block >> 32), (uint32_t)step, (uint32_t)(step >> 32),
                            keys);
}

// Blocks `block` and block + 1, `block` even, with 37 wide products for 40: they have
// the product of the step in the first round and that which follows from it in the
// second in common, and the two other products of the first round differ by the factor.
__device__ __forceinline__ void philox_two(uint64_t block, uint64_t step, const PhiloxKeys &keys, uint4 &r0,
                                           uint4 &r1) {
    const uint64_t x0 = (uint64_t)(uint32_t)block * 0xD2511F53u, x1 = x0 + 0xD2511F53u;
    const uint64_t y = (uint64_t)(uint32_t)step * 0xCD9E8D57u;
    const uint32_t a = (uint32_t)(y >> 32) ^ (uint32_t)(block >> 32) ^ keys.k[0][0], b = (uint32_t)y;
    const uint32_t dk = (uint32_t)(step >> 32) ^ keys.k[0][1];
    const uint64_t z = (uint64_t)a * 0xD2511F53u;
    const uint32_t bk = b ^ keys.k[1][0], zk = (uint32_t)(z >> 32) ^ keys.k[1][1];
    const uint64_t y0 = (uint64_t)((uint32_t)(x0 >> 32) ^ dk) * 0xCD9E8D57u,
                   y1 = (uint64_t)((uint32_t)(x1 >> 32) ^ dk) * 0xCD9E8D57u;
    r0 = philox_rounds<2>((uint32_t)(y0 >> 32) ^ bk, (uint32_t)y0, zk ^ (uint32_t)x0, (uint32_t)z, keys);
    r1 = philox_rounds<2>((uint32_t)(y1 >> 32) ^ bk, (uint32_t)y1, zk ^ (uint32_t)x1, (uint32_t)z, keys);
}

}  // namespace ck
