// The counter-based generator of the dropout mask: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011), one 128-bit block for 8 consecutive
// elements, 16 bits each.
//
// 16 bits an element instead of 32: a block's ten rounds (20 32x32->64 products) then serve one
// 16-byte word of a 16-bit tensor, half the integer work, and the dropout alone moves only 4 to 6
// bytes per such element.  The cost is that p is rounded to a multiple of 2^-16; the kept
// elements' factor uses the rounded p, so the expectation stays exact.
#pragma once

#include <stdint.h>

#include "dw_common.cuh"

namespace dwk {

struct DropoutRng {
    uint32_t k0, k1, o0, o1;  // key = seed, upper half of the counter = offset

    __device__ __forceinline__ void load(const unsigned long long *rng) {
        const unsigned long long seed = load_global(rng), offset = load_global(rng + 1);
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        o0 = static_cast<uint32_t>(offset);
        o1 = static_cast<uint32_t>(offset >> 32);
    }

    // The blocks g[0 .. NO-1]: block g has elements 8 g .. 8 g + 7, element 8 g + i in bits
    // 16 (i % 2) .. of word i / 2.
    template <int NO, typename G> __device__ __forceinline__ void blocks(const G (&g)[NO], uint4 (&w)[NO]) const {
        uint32_t a = k0, b = k1;
#pragma unroll
        for (int j = 0; j < NO; ++j) {
            const uint64_t gj = g[j];
            w[j] = make_uint4(static_cast<uint32_t>(gj), static_cast<uint32_t>(gj >> 32), o0, o1);
        }
#pragma unroll
        for (int r = 0; r < 10; ++r) {
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                const uint64_t p = static_cast<uint64_t>(w[j].x) * 0xD2511F53u;
                const uint64_t q = static_cast<uint64_t>(w[j].z) * 0xCD9E8D57u;
                w[j] = make_uint4(static_cast<uint32_t>(q >> 32) ^ w[j].y ^ a, static_cast<uint32_t>(q),
                                  static_cast<uint32_t>(p >> 32) ^ w[j].w ^ b, static_cast<uint32_t>(p));
            }
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
    }

    __device__ __forceinline__ uint4 block(uint64_t g) const {
        const uint64_t gs[1] = {g};
        uint4 w[1];
        blocks<1>(gs, w);
        return w[0];
    }

    // Whether one element is kept (a whole block per call: the slow, general form).
    __device__ __forceinline__ bool kept(uint64_t e, uint32_t thr) const {
        const uint4 w = block(e >> 3);
        const uint32_t i = static_cast<uint32_t>(e) & 7u;
        const uint32_t u = i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w);
        return ((i & 1u) ? (u >> 16) : (u & 0xffffu)) >= thr;
    }
};

}  // namespace dwk
