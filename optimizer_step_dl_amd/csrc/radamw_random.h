// radamw_random.h -- the counter-based generator of dropout, on the device.
//
// Philox 4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): a bijection of a 128-bit
// counter under a 64-bit key, so that any lane forms any element's number
// from its place alone and the backward pass forms the same ones again.
//
//   key     = seed
//   counter = (column / 8, first_row + row, offset's low word, its high word)
//
// A counter's four words are eight 16-bit numbers for eight columns: the low
// half of word 0, its high half, and so on.  A round is two products of 32 x
// 32 bits, which the vector units do at a quarter of their rate; with a 32-bit
// number per element the products alone would take longer than HBM needs to
// move 16-bit elements in and out, with 16 bits half as long.
#pragma once

#include "radamw_block.h"
#include "radamw_rows.h"

namespace radamw {

__device__ __forceinline__ u32x4 random_words(uint32_t column8, uint32_t row, const DropArgs &d) {
    uint32_t c0 = column8, c1 = d.first_row + row, c2 = d.off0, c3 = d.off1, k0 = d.key0, k1 = d.key1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// Whether column j of a counter's eight is kept.
__device__ __forceinline__ bool kept(u32x4 words, int j, uint32_t threshold) {
    const uint32_t w = words[j >> 1];
    return (j & 1 ? w >> 16 : w & 0xffffu) >= threshold;
}

}  // namespace radamw
