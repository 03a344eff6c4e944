// The microscaled 4-bit format (OCP Microscaling Formats v1.0, MXFP4): e2m1 elements in blocks
// of 32 along a row under one e8m0 scale. Codes are packed two to a byte, the even column in
// the low nibble; a block's scale byte s stands for 2^(s - 127).
//
//   s = max(0, floor(log2(amax)) - 2 + 127)     the largest e2m1 exponent is 2
//   code = e2m1(x 2^(127 - s))                  to nearest even, saturated at +-6
//
// The products by powers of two are exact (or far below the smallest code), so every code is
// rounded once. A block with an infinity or a NaN gets the scale 255 (NaN) and codes 0: every
// product that meets it is NaN, as the format asks for, and its neighbours are untouched.
#pragma once

#include "vec8.cuh"

namespace moe {
namespace {

// scale byte of a block whose largest magnitude is amax (NaN and infinity have bits above or
// at 0x7f800000)
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// the factor 2^(127 - s) that brings a block to the e2m1 range (0 for a NaN block)
__device__ __forceinline__ float mx_inv_scale(uint32_t s)
{
    return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// 2^(s - 127): subnormal for s = 0, NaN for 255
__device__ __forceinline__ float mx_scale(uint32_t s)
{
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fffffffu : s << 23);
}

// 8 scaled values to 8 codes, element 0 in the lowest nibble
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// largest magnitude's bits of 8 values, as an unsigned maximum: NaN ranks above infinity
__device__ __forceinline__ uint32_t mx_amax8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
}

// codes of 8 values under scale byte s; a NaN block's values are replaced before the conversion
__device__ __forceinline__ uint32_t mx_encode8(const float (&v)[8], uint32_t s)
{
    if (s == 255u) return 0u;
    const float f = mx_inv_scale(s);
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = v[e] * f;
    return mx_codes8(w);
}

// 8 codes to the values they stand for (exact: e2m1 in fp16)
__device__ __forceinline__ void mx_decode8(uint32_t codes, float (&f)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 v = *reinterpret_cast<const __half2*>(&h[i]);
        f[2 * i] = __low2float(v);
        f[2 * i + 1] = __high2float(v);
    }
}

// Offset of the scale of (row, block) in the tensor core's tiles: 128 rows by 4 blocks of 32
// (128 columns) are 512 consecutive bytes, row r at 16 (r % 32) + 4 (r / 32), its 4 blocks in
// order; tiles follow along the row first. `row` counts over all matrices of a batch (each a
// multiple of 128 rows); `blocks` is the blocks of a row, rounded up to 4.
__host__ __device__ __forceinline__ int64_t mx_tiled_scale(int64_t row, int block, int blocks)
{
    const int r = (int)(row & 127);
    return ((row >> 7) * (blocks >> 2) + (block >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 +
           (block & 3);
}

}  // namespace
}  // namespace moe
