// Vectors of 8 consecutive elements of a bf16, fp16 or fp32 tensor: 16- or 32-byte loads and
// stores, widened to fp32 and rounded once to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

// Two fp32 values in one 64-bit register pair: the packed add, multiply and fma of sm_100
// (each half rounded to nearest as its scalar form) halve the instructions of row kernels whose
// arithmetic would otherwise take longer than their memory traffic.
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void unpack(F2 a, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 a)
{
    float lo, hi;
    unpack(a, lo, hi);
    return lo + hi;
}

template <int DT>
struct Vec8;

template <>
struct Vec8<MOE_BF16> {
    uint4 q;
    __device__ __forceinline__ void load(const void* p, int64_t vec)
    {
        q = static_cast<const uint4*>(p)[vec];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        q = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store(void* p, int64_t vec) const
    {
        static_cast<uint4*>(p)[vec] = q;
    }
};

template <>
struct Vec8<MOE_F16> {
    uint4 q;
    __device__ __forceinline__ void load(const void* p, int64_t vec)
    {
        q = static_cast<const uint4*>(p)[vec];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = *reinterpret_cast<const __half2*>(&u[i]);
            f[2 * i] = __low2float(h);
            f[2 * i + 1] = __high2float(h);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        q = make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store(void* p, int64_t vec) const
    {
        static_cast<uint4*>(p)[vec] = q;
    }
};

template <>
struct Vec8<MOE_F32> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t vec)
    {
        const float4* s = static_cast<const float4*>(p) + 2 * vec;
        a = s[0];
        b = s[1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void store(void* p, int64_t vec) const
    {
        float4* d = static_cast<float4*>(p) + 2 * vec;
        d[0] = a;
        d[1] = b;
    }
};

// the 8 elements as four pairs
template <int DT>
__device__ __forceinline__ void get2(const Vec8<DT>& q, F2 (&f)[4])
{
    float s[8];
    q.get(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(s[2 * i], s[2 * i + 1]);
}
template <int DT>
__device__ __forceinline__ void set2(Vec8<DT>& q, const F2 (&f)[4])
{
    float s[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack(f[i], s[2 * i], s[2 * i + 1]);
    q.set(s);
}

// 8 parameters starting at 8 * vec: fp32, or the activations' type
template <int DT>
__device__ __forceinline__ void load_param8(const void* p, bool f32, int64_t vec, float (&f)[8])
{
    if (DT == MOE_F32 || f32) {
        Vec8<MOE_F32> v;
        v.load(p, vec);
        v.get(f);
    } else {
        Vec8<DT> v;
        v.load(p, vec);
        v.get(f);
    }
}

template <int DT>
__device__ __forceinline__ void load_param2(const void* p, bool f32, int64_t vec, F2 (&f)[4])
{
    float s[8];
    load_param8<DT>(p, f32, vec, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(s[2 * i], s[2 * i + 1]);
}

template <int DT>
__device__ __forceinline__ float load_param(const void* p, bool f32, int64_t i)
{
    if (DT == MOE_F32 || f32) return static_cast<const float*>(p)[i];
    if (DT == MOE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}

}  // namespace
}  // namespace moe
