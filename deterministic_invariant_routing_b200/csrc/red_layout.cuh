// Where a block's reductions keep their warps' sums in shared memory. Plain arithmetic, so that a
// host compiler takes it too.
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__
#else
#define MOE_HD
#endif

namespace moe {

constexpr int kRed = 32;  // warps of a block at most: floats per value and half

// Place of warp `warp`'s sum of value `k` in a call that uses half `half` of the buffer.
//
// Two calls in a row use different halves, and one barrier a call (between its writes and its
// reads) is enough when these do not overlap: a warp that writes call i + 1's sums may run beside
// a warp that still reads call i's, but call i + 2 writes only after the barrier of call i + 1,
// which every reader of call i has reached. So a half has room for the most values, `kmax`, that
// any call on the buffer sums, whatever the number that this call sums.
template <int kmax>
MOE_HD constexpr int red_place(int half, int k, int warp)
{
    return (half * kmax + k) * kRed + warp;
}

template <int kmax>
constexpr int kRedFloats = 2 * kmax * kRed;

}  // namespace moe
