// The counter-based generator of the dropout masks: Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011). A mask element is a function
// of (seed, offset, row, column) alone, so forward and backward recompute it, nothing is
// stored, and a token's mask does not depend on the batch it sits in.
//
//   counter = (column / 8, row, offset low, offset high), key = (seed low, seed high)
//
// One call gives 128 bits: 16 for each of the 8 columns of a vector (element 2 i in the low
// half of word i). An element is kept when its 16 bits are at least the threshold
// floor(65536 p + 1/2); the kept values are scaled by 65536 / (65536 - threshold), the inverse
// of the exact probability to keep. 16 bits rather than 32 halve the integer work, which would
// otherwise be as long as the memory traffic of a bf16 tensor: about 10 multiply and logic
// instructions an element against 4 bytes.
#pragma once

#include <stdint.h>

namespace moe {
namespace {

struct Philox {
    uint32_t k0, k1, c2, c3;  // the key and the offset's two words
};

// rng: device int64[2], (seed, offset)
__device__ __forceinline__ Philox philox_load(const int64_t* rng)
{
    // one lane's copy for all: the key schedule then stays in uniform registers
    const uint64_t seed = __shfl_sync(0xffffffffu, (unsigned long long)rng[0], 0);
    const uint64_t off = __shfl_sync(0xffffffffu, (unsigned long long)rng[1], 0);
    return Philox{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

__device__ __forceinline__ void philox_round(uint32_t& c0, uint32_t& c1, uint32_t& c2,
                                             uint32_t& c3, uint32_t k0, uint32_t k1)
{
    const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
}

__device__ __forceinline__ void philox8(const Philox& g, uint32_t col8, uint32_t row,
                                        uint32_t (&w)[4])
{
    w[0] = col8;
    w[1] = row;
    w[2] = g.c2;
    w[3] = g.c3;
#pragma unroll
    for (uint32_t i = 0; i < 10; ++i)
        philox_round(w[0], w[1], w[2], w[3], g.k0 + i * 0x9E3779B9u, g.k1 + i * 0xBB67AE85u);
}

// N vectors at once: a round's keys are formed once for all of them, and their rounds interleave
template <int N>
__device__ __forceinline__ void philox8n(const Philox& g, const uint32_t (&col8)[N],
                                         const uint32_t (&row)[N], uint32_t (&w)[N][4])
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        w[n][0] = col8[n];
        w[n][1] = row[n];
        w[n][2] = g.c2;
        w[n][3] = g.c3;
    }
    uint32_t k0 = g.k0, k1 = g.k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
        for (int n = 0; n < N; ++n)
            philox_round(w[n][0], w[n][1], w[n][2], w[n][3], k0, k1);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// whether element e (0..7) of the vector is kept
__device__ __forceinline__ bool philox_keep(const uint32_t (&w)[4], int e, uint32_t threshold)
{
    const uint32_t u = (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
    return u >= threshold;
}

}  // namespace
}  // namespace moe
