// Quotients by a divisor fixed for a launch.
#pragma once

#include <stdint.h>

namespace moe {
namespace {

// 32-bit quotients by a fixed divisor: n / d = (n * m) >> (32 + s) for n < 2^31 (m = ceil(2^(32+s)
// / d) with 2^s >= d is below 2^33, its top bit added back)
struct FastDiv {
    uint32_t d, m, s;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0)
    {
        while ((1ull << s) < div) ++s;
        m = (uint32_t)(((1ull << 32) * ((1ull << s) - div)) / div + 1);
    }
    __device__ __forceinline__ uint32_t quot(uint32_t n) const
    {
        return (__umulhi(n, m) + n) >> s;
    }
};

__device__ __forceinline__ int64_t quotient(int64_t n, const FastDiv& f, bool narrow)
{
    return narrow ? (int64_t)f.quot((uint32_t)n) : n / f.d;
}

}  // namespace
}  // namespace moe
