// Quantisation to the microscaled 4-bit format and back (mx_format.cuh). Bound by memory:
// 2 or 4 bytes read and 17/32 written per element, no reuse. A lane takes 8 consecutive
// elements, four lanes a block of 32: two shuffles give the block's largest magnitude.
#include "mx_format.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;
constexpr int kQVec = 4;  // vectors of 8 per thread, a block's width apart

// the block maximum over the four lanes that share it
__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Scales in tiles: lane 0 of the 16 that share 128 columns stores the word of their 4 blocks.
// `s` is the lane's block scale; `word` counts 128 columns.
__device__ __forceinline__ uint32_t quad_word(uint32_t s)
{
    const int lane = threadIdx.x & 31;
    const uint32_t b1 = __shfl_down_sync(0xffffffffu, s, 4), b2 = __shfl_down_sync(0xffffffffu, s, 8),
                   b3 = __shfl_down_sync(0xffffffffu, s, 12);
    return (lane & 15) == 0 ? s | b1 << 8 | b2 << 16 | b3 << 24 : 0u;
}

// x [rows, 8 nvec], row-major scales: one run of vectors (a block never spans two rows)
template <int DT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(const void* x, int64_t total,
                                                                uint32_t* codes, uint8_t* scales)
{
    pdl_wait();
    const int64_t base = (int64_t)blockIdx.x * (kQThreads * kQVec) + threadIdx.x;
    Vec8<DT> q[kQVec];
#pragma unroll
    for (int i = 0; i < kQVec; ++i)
        if (base + kQThreads * i < total) q[i].load(x, base + kQThreads * i);
#pragma unroll
    for (int i = 0; i < kQVec; ++i) {
        const int64_t v = base + kQThreads * i;
        float f[8] = {};
        if (v < total) q[i].get(f);
        const uint32_t s = mx_scale_byte(quad_max(mx_amax8(f)));  // quads are whole: 4 | total
        if (v < total) {
            codes[v] = mx_encode8(f, s);
            if ((threadIdx.x & 3) == 0) scales[v >> 2] = (uint8_t)s;
        }
    }
}

// The same with the scales in tiles, over rows padded to 128 and vectors padded to 16 (`nvecp`):
// the padding's scales are written as 0, so that every byte of the tiles is defined.
template <int DT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_tiled_kernel(const void* x, int64_t rows,
                                                                      int32_t nvec, int32_t nvecp,
                                                                      int64_t total,
                                                                      uint32_t* codes,
                                                                      uint8_t* scales)
{
    pdl_wait();
    const int64_t base = (int64_t)blockIdx.x * (kQThreads * kQVec) + threadIdx.x;
    Vec8<DT> q[kQVec];
    int64_t row[kQVec];
    int32_t col[kQVec];
#pragma unroll
    for (int i = 0; i < kQVec; ++i) {
        const int64_t v = base + kQThreads * i;
        row[i] = total <= 0xffffffffll ? (int64_t)((uint32_t)v / (uint32_t)nvecp) : v / nvecp;
        col[i] = (int32_t)(v - row[i] * nvecp);
        if (row[i] < rows && col[i] < nvec) q[i].load(x, row[i] * nvec + col[i]);
    }
#pragma unroll
    for (int i = 0; i < kQVec; ++i) {
        const bool in = row[i] < rows && col[i] < nvec;
        float f[8] = {};
        if (in) q[i].get(f);
        const uint32_t s = mx_scale_byte(quad_max(mx_amax8(f)));
        const uint32_t word = quad_word(s);
        if (in) codes[row[i] * nvec + col[i]] = mx_encode8(f, s);
        if ((threadIdx.x & 15) == 0 && base + kQThreads * i < total)
            *reinterpret_cast<uint32_t*>(scales + mx_tiled_scale(row[i], col[i] >> 2, nvecp >> 2)) =
                word;
    }
}

// The dispatch of a layer whose experts take 4-bit rows: token t is quantised once and its
// codes and scales are written to row dest_row[t, j] for every j (and, token-major, to t when
// the shared expert needs them). One thread per vector of a token.
__global__ void __launch_bounds__(kQThreads) mx_scatter_kernel(
    const void* x, int64_t total, int32_t nvec, const int32_t* dest_row, int K, int64_t rows,
    uint32_t* codes, uint8_t* scales, uint32_t* tok_codes, uint8_t* tok_scales, int32_t* status)
{
    pdl_wait();
    const int64_t v = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
    Vec8<MOE_BF16> q;
    float f[8] = {};
    if (v < total) {
        q.load(x, v);
        q.get(f);
    }
    const uint32_t s = mx_scale_byte(quad_max(mx_amax8(f)));
    const uint32_t word = quad_word(s);  // H is a multiple of 128: 16 lanes share a row
    if (v >= total) return;
    const int64_t t = total <= 0xffffffffll ? (int64_t)((uint32_t)v / (uint32_t)nvec) : v / nvec;
    const int32_t c = (int32_t)(v - t * nvec);
    const uint32_t w = mx_encode8(f, s);
    for (int j = 0; j < K; ++j) {
        const int32_t r = dest_row[t * K + j];
        if (r < 0) continue;
        if (r >= rows) {
            if (c == 0) status_add(status, MOE_ST_BAD_ROWS, 1);
            continue;
        }
        codes[(int64_t)r * nvec + c] = w;
        if ((c & 15) == 0)
            *reinterpret_cast<uint32_t*>(scales + mx_tiled_scale(r, c >> 2, nvec >> 2)) = word;
    }
    if (tok_codes != nullptr) {
        tok_codes[v] = w;
        if ((c & 15) == 0)
            *reinterpret_cast<uint32_t*>(tok_scales + mx_tiled_scale(t, c >> 2, nvec >> 2)) = word;
    }
}

template <int DT, bool TILED>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(const uint32_t* codes,
                                                                  const uint8_t* scales,
                                                                  int64_t total, int32_t nvec,
                                                                  void* out)
{
    pdl_wait();
    const int64_t base = (int64_t)blockIdx.x * (kQThreads * kQVec) + threadIdx.x;
    uint32_t c[kQVec], s[kQVec];
#pragma unroll
    for (int i = 0; i < kQVec; ++i) {
        const int64_t v = base + kQThreads * i;
        if (v < total) {
            c[i] = codes[v];
            int64_t at = v >> 2;
            if (TILED) {
                const int64_t row = total <= 0xffffffffll
                                        ? (int64_t)((uint32_t)v / (uint32_t)nvec)
                                        : v / nvec;
                at = mx_tiled_scale(row, (int)(v - row * nvec) >> 2, (nvec + 15) / 16 * 4);
            }
            s[i] = scales[at];
        }
    }
#pragma unroll
    for (int i = 0; i < kQVec; ++i) {
        const int64_t v = base + kQThreads * i;
        if (v < total) {
            const float k = mx_scale(s[i]);
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t n = (c[i] >> (4 * e)) & 15u, m = n & 7u;
                // 0, 1/2, then (1 + fraction / 2) 2^(exponent - 1)
                const float a = m < 2u ? 0.5f * (float)m
                                       : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
                f[e] = (n & 8u ? -a : a) * k;
            }
            Vec8<DT> o;
            o.set(f);
            o.store(out, v);
        }
    }
}

unsigned blocks_of(int64_t total)
{
    return (unsigned)((total + kQThreads * kQVec - 1) / (kQThreads * kQVec));
}

template <int DT>
cudaError_t quantize(const void* x, int64_t rows, int32_t nvec, bool tiled, uint8_t* codes,
                     uint8_t* scales, cudaStream_t st)
{
    uint32_t* c = reinterpret_cast<uint32_t*>(codes);
    if (!tiled) {
        const int64_t total = rows * nvec;
        return launch_pdl(mx_quantize_kernel<DT>, dim3(blocks_of(total)), dim3(kQThreads), 0, st,
                          x, total, c, scales);
    }
    const int32_t nvecp = (nvec + 15) / 16 * 16;
    const int64_t total = (rows + 127) / 128 * 128 * nvecp;
    return launch_pdl(mx_quantize_tiled_kernel<DT>, dim3(blocks_of(total)), dim3(kQThreads), 0, st,
                      x, rows, nvec, nvecp, total, c, scales);
}

template <int DT>
cudaError_t dequantize(int64_t rows, int32_t nvec, bool tiled, const uint8_t* codes,
                       const uint8_t* scales, void* out, cudaStream_t st)
{
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    const int64_t total = rows * nvec;
    return launch_pdl(tiled ? mx_dequantize_kernel<DT, true> : mx_dequantize_kernel<DT, false>,
                      dim3(blocks_of(total)), dim3(kQThreads), 0, st, c, scales, total, nvec, out);
}

}  // namespace

cudaError_t launch_mx_quantize(int64_t rows, int32_t K, int dtype, bool tiled, const void* x,
                               uint8_t* codes, uint8_t* scales, cudaStream_t st)
{
    switch (dtype) {
        case MOE_BF16: return quantize<MOE_BF16>(x, rows, K / 8, tiled, codes, scales, st);
        case MOE_F16: return quantize<MOE_F16>(x, rows, K / 8, tiled, codes, scales, st);
        default: return quantize<MOE_F32>(x, rows, K / 8, tiled, codes, scales, st);
    }
}

cudaError_t launch_mx_scatter(const moe_cfg& c, const uint16_t* x, const int32_t* dest_row,
                              uint8_t* codes, uint8_t* scales, uint8_t* tok_codes,
                              uint8_t* tok_scales, int32_t* status, cudaStream_t st)
{
    const int32_t nvec = c.H / 8;
    const int64_t total = (int64_t)c.T * nvec;
    return launch_pdl(mx_scatter_kernel, dim3((unsigned)((total + kQThreads - 1) / kQThreads)),
                      dim3(kQThreads), 0, st, x, total, nvec, dest_row, c.K,
                      (int64_t)c.T * c.K, reinterpret_cast<uint32_t*>(codes), scales,
                      reinterpret_cast<uint32_t*>(tok_codes), tok_scales, status);
}

cudaError_t launch_mx_dequantize(int64_t rows, int32_t K, int dtype, bool tiled,
                                 const uint8_t* codes, const uint8_t* scales, void* out,
                                 cudaStream_t st)
{
    switch (dtype) {
        case MOE_BF16: return dequantize<MOE_BF16>(rows, K / 8, tiled, codes, scales, out, st);
        case MOE_F16: return dequantize<MOE_F16>(rows, K / 8, tiled, codes, scales, out, st);
        default: return dequantize<MOE_F32>(rows, K / 8, tiled, codes, scales, out, st);
    }
}

}  // namespace moe
