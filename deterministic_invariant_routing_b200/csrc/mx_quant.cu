// Quantisation to the microscaled 4-bit format and back (mx_format.cuh). Bound by memory:
// 2 or 4 bytes read and 17/32 written per element, no reuse, so what matters is the work per
// element. Quantising, a thread takes a whole block of 32: its largest magnitude needs no
// shuffles, its codes are one 16-byte store, and the index arithmetic is paid once for 32
// elements (with 8 a thread the dispatch below was bound by instructions: 63 us for 16384
// tokens of 2048 to 8 rows each; 38 us now, 209 MB). Back, a thread writes 8 elements, so that
// stores are whole. 49152 x 2048 bf16 weights: 41 us to codes (254 MB, 6.2 TB/s) and 41 us back.
#include "fast_div.cuh"
#include "mx_format.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;

// quantise the block of 32 elements at block index b of x: its scale byte and codes
template <int DT>
__device__ __forceinline__ uint32_t quantize_block(const Vec8<DT> (&q)[4], uint4& codes)
{
    float f[4][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i].get(f[i]);
        m = max(m, mx_amax8(f[i]));
    }
    const uint32_t s = mx_scale_byte(m);
    codes = make_uint4(mx_encode8(f[0], s), mx_encode8(f[1], s), mx_encode8(f[2], s),
                       mx_encode8(f[3], s));
    return s;
}

// the word of 4 neighbouring lanes' scale bytes, in the first of them
__device__ __forceinline__ uint32_t quad_word(uint32_t s)
{
    s |= __shfl_down_sync(0xffffffffu, s, 1) << 8;
    return s | __shfl_down_sync(0xffffffffu, s, 2) << 16;
}

// x as one run of `total` blocks (rows are whole blocks), row-major scales
template <int DT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(const void* x, int64_t total,
                                                                uint4* codes, uint8_t* scales)
{
    pdl_wait();
    const int64_t b = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
    if (b >= total) return;
    Vec8<DT> q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i].load(x, 4 * b + i);
    uint4 c;
    const uint32_t s = quantize_block<DT>(q, c);
    codes[b] = c;
    scales[b] = (uint8_t)s;
}

// The same with the scales in tiles, over rows padded to 128 and blocks padded to 4 (`nbp` a
// row): the padding's scales are written as 0, so that every byte of the tiles is defined.
template <int DT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_tiled_kernel(const void* x, int64_t rows,
                                                                      int32_t nb, int32_t nbp,
                                                                      FastDiv div, int64_t total,
                                                                      uint4* codes,
                                                                      uint8_t* scales)
{
    pdl_wait();
    const int64_t v = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
    // (threads past the last block stay below 2^31 too)
    const int64_t row = quotient(v, div, total <= 0x7fffffffll - kQThreads);
    const int32_t col = (int32_t)(v - row * nbp);
    uint32_t s = 0;
    if (row < rows && col < nb) {
        const int64_t b = row * nb + col;
        Vec8<DT> q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i].load(x, 4 * b + i);
        uint4 c;
        s = quantize_block<DT>(q, c);
        codes[b] = c;
    }
    const uint32_t word = quad_word(s);
    if ((threadIdx.x & 3) == 0 && v < total)
        *reinterpret_cast<uint32_t*>(scales + mx_tiled_scale(row, col, nbp)) = word;
}

// The dispatch of a layer whose experts take 4-bit rows: token t is quantised once and its
// codes and scales are written to row dest_row[t, j] for every j (and, token-major, to t when
// the shared expert needs them). One thread per block of a token (nb blocks a row, a multiple
// of 4).
__global__ void __launch_bounds__(kQThreads) mx_scatter_kernel(
    const void* x, int64_t total, int32_t nb, FastDiv div, const int32_t* dest_row, int K,
    int64_t rows, uint4* codes, uint8_t* scales, uint4* tok_codes, uint8_t* tok_scales,
    int32_t* status)
{
    pdl_wait();
    const int64_t b = (int64_t)blockIdx.x * kQThreads + threadIdx.x;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    uint32_t s = 0;
    if (b < total) {
        Vec8<MOE_BF16> q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i].load(x, 4 * b + i);
        s = quantize_block<MOE_BF16>(q, w);
    }
    const uint32_t word = quad_word(s);
    if (b >= total) return;
    const int64_t t = quotient(b, div, total <= 0x7fffffffll);
    const int32_t c = (int32_t)(b - t * nb);
    const bool first = (c & 3) == 0;
    for (int j = 0; j < K; ++j) {
        const int32_t r = dest_row[t * K + j];
        if (r < 0) continue;
        if (r >= rows) {
            if (c == 0) status_add(status, MOE_ST_BAD_ROWS, 1);
            continue;
        }
        codes[(int64_t)r * nb + c] = w;
        if (first)
            *reinterpret_cast<uint32_t*>(scales + mx_tiled_scale(r, c, nb)) = word;
    }
    if (tok_codes != nullptr) {
        tok_codes[b] = w;
        if (first)
            *reinterpret_cast<uint32_t*>(tok_scales + mx_tiled_scale(t, c, nb)) = word;
    }
}

constexpr int kDVec = 4;  // vectors of 8 per thread, a block's width apart

template <int DT, bool TILED>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(const uint32_t* codes,
                                                                  const uint8_t* scales,
                                                                  int64_t total, int32_t nvec,
                                                                  FastDiv div, void* out)
{
    pdl_wait();
    const int64_t base = (int64_t)blockIdx.x * (kQThreads * kDVec) + threadIdx.x;
    uint32_t c[kDVec], s[kDVec];
#pragma unroll
    for (int i = 0; i < kDVec; ++i) {
        const int64_t v = base + kQThreads * i;
        if (v < total) {
            c[i] = codes[v];
            int64_t at = v >> 2;
            if (TILED) {
                const int64_t row = quotient(v, div, total <= 0x7fffffffll);
                at = mx_tiled_scale(row, (int)(v - row * nvec) >> 2, (nvec + 15) / 16 * 4);
            }
            s[i] = scales[at];
        }
    }
#pragma unroll
    for (int i = 0; i < kDVec; ++i) {
        const int64_t v = base + kQThreads * i;
        if (v < total) {
            const float k = mx_scale(s[i]);
            float f[8];
            mx_decode8(c[i], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= k;
            Vec8<DT> o;
            o.set(f);
            o.store(out, v);
        }
    }
}

unsigned blocks_of(int64_t total, int per) { return (unsigned)((total + per - 1) / per); }

template <int DT>
cudaError_t quantize(const void* x, int64_t rows, int32_t nb, bool tiled, uint8_t* codes,
                     uint8_t* scales, cudaStream_t st)
{
    uint4* c = reinterpret_cast<uint4*>(codes);
    if (!tiled) {
        const int64_t total = rows * nb;
        return launch_pdl(mx_quantize_kernel<DT>, dim3(blocks_of(total, kQThreads)),
                          dim3(kQThreads), 0, st, x, total, c, scales);
    }
    const int32_t nbp = (nb + 3) / 4 * 4;
    const int64_t total = (rows + 127) / 128 * 128 * nbp;
    return launch_pdl(mx_quantize_tiled_kernel<DT>, dim3(blocks_of(total, kQThreads)),
                      dim3(kQThreads), 0, st, x, rows, nb, nbp, FastDiv((uint32_t)nbp), total, c,
                      scales);
}

template <int DT>
cudaError_t dequantize(int64_t rows, int32_t nvec, bool tiled, const uint8_t* codes,
                       const uint8_t* scales, void* out, cudaStream_t st)
{
    const int64_t total = rows * nvec;
    return launch_pdl(tiled ? mx_dequantize_kernel<DT, true> : mx_dequantize_kernel<DT, false>,
                      dim3(blocks_of(total, kQThreads * kDVec)), dim3(kQThreads), 0, st,
                      reinterpret_cast<const uint32_t*>(codes), scales, total, nvec,
                      FastDiv((uint32_t)nvec), out);
}

}  // namespace

cudaError_t launch_mx_quantize(int64_t rows, int32_t K, int dtype, bool tiled, const void* x,
                               uint8_t* codes, uint8_t* scales, cudaStream_t st)
{
    switch (dtype) {
        case MOE_BF16: return quantize<MOE_BF16>(x, rows, K / 32, tiled, codes, scales, st);
        case MOE_F16: return quantize<MOE_F16>(x, rows, K / 32, tiled, codes, scales, st);
        default: return quantize<MOE_F32>(x, rows, K / 32, tiled, codes, scales, st);
    }
}

cudaError_t launch_mx_scatter(const moe_cfg& c, const uint16_t* x, const int32_t* dest_row,
                              uint8_t* codes, uint8_t* scales, uint8_t* tok_codes,
                              uint8_t* tok_scales, int32_t* status, cudaStream_t st)
{
    const int32_t nb = c.H / 32;
    const int64_t total = (int64_t)c.T * nb;
    return launch_pdl(mx_scatter_kernel, dim3(blocks_of(total, kQThreads)), dim3(kQThreads), 0, st,
                      x, total, nb, FastDiv((uint32_t)nb), dest_row, c.K, (int64_t)c.T * c.K,
                      reinterpret_cast<uint4*>(codes), scales, reinterpret_cast<uint4*>(tok_codes),
                      tok_scales, status);
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
