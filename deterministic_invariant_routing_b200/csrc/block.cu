// What joins two blocks of the residual stream, and its gradients: the norm after a block, its
// gate, dropout and residual scale, the residual sum and the next block's norm, in one pass.
//
//   z = drop(rms(y) w_post),  rms(v) = v / sqrt(mean(v^2) + eps)
//   r = round(residual_scale x + branch_scale gate z),  n = round(rms(r) w_next)
//
// n is taken from the rounded r, so the fused call gives the bits of the two calls it replaces.
// Every sum is fp32 in an order that depends on H alone (a thread's own vectors, a shuffle
// tree in each warp, the warps in order): a token's row never depends on T or on its neighbours.
//
// By its bytes it is bound by memory: 4 row passes forward (x, y in; r, n out), 6 backward (y,
// r, dr, dn in; dx, dy out). A row stays in the registers of one block (one warp up to H = 512),
// so nothing is read twice, and the backward recomputes both norms' statistics and the dropout
// mask from what it reads anyway: nothing but r and y is kept from the forward. The backward does
// not reach that bound, nor another: at 16-bit types it has 57 instructions an element, the mask
// alone 8, and issues at 0.57 of the rate (memory at the copy's rate would take 0.88 of it) with 16
// warps an SM, all that the sums of the parameter gradients allow; latency is left, around a row's
// two barriers. Instructions are what there was to take out: hence the packed fp32 arithmetic
// (F2), the kernels without branches for calls with both norms, and the shuffles that add two values
// at once. Measured on B200:
//   forward, 16384 x 2048 bf16, channel gate, dropout: 45 us (268 MB; 41 us at the copy's rate)
//   forward, the same without w_post, gate and dropout, bf16 weights: 47.5 us
//   backward, 8192 x 4096 bf16, channel gate, dropout: 97 us (403 MB; 61 us)
//   backward, 16384 x 2048 bf16, both norms, fp32 weights: 68 us, with bf16 weights (kAny): 129;
//     without w_post, bf16 weights (kAny): 100 us (403 MB each; 61 us)
//
// Parameter gradients are column sums over tokens: block b of a grid whose size is a function
// of (T, H, type) adds rows b, b + blocks, ... into its registers and writes one partial row; a
// second kernel sums the partials in order. No atomics: the bits repeat, on any device.
#include "fast_div.cuh"
#include "philox.cuh"
#include "red_layout.cuh"
#include "vec8.cuh"

namespace moe {
namespace {

struct NormArgs {
    const void *x, *y, *w_post, *gate, *w_next, *dr, *dn;
    void *r, *n, *dx, *dy, *dgate;
    float* part;  // [blocks, slots, H]
    const int64_t* rng;
    const int32_t* row_ids;
    int64_t T;
    int32_t H;
    int32_t nvec;  // H / 8
    uint32_t first_row, threshold;
    int32_t gate_mode, param_f32;
    int32_t slot_next, slot_post, slot_gate, slots;  // partial rows of a block, -1: none
    float eps, inv_h, residual_scale, branch_scale, inv_keep;  // inv_h: 1 / H
};

// Sums K <= 4 values over a warp: each of the first shuffles adds two values at once (a lane keeps
// one of them and gives the other away), so four values take 6 shuffles instead of 20. Value k's
// total ends up in lane owner(k), and with ALL_LANES in every lane (a shuffle more per value).
// The order of a value's sum is fixed.
__device__ __forceinline__ int owner(int k) { return (k & 1) * 16 + (k >> 1) * 8; }

template <int K, bool ALL_LANES>
__device__ __forceinline__ void warp_sum(float (&v)[K])
{
    constexpr uint32_t all = 0xffffffffu;
    if (K == 1) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v[0] += __shfl_xor_sync(all, v[0], off);
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16;
    const float a = v[0], b = v[K > 1 ? 1 : 0];
    float p = (hi ? b : a) + __shfl_xor_sync(all, hi ? a : b, 16);  // sums of v0 | v1
    if (K > 2) {
        const float c = v[K > 2 ? 2 : 0], d = K > 3 ? v[K > 3 ? 3 : 0] : 0.0f;
        const float q = (hi ? d : c) + __shfl_xor_sync(all, hi ? c : d, 16);  // v2 | v3
        const bool odd = lane & 8;
        p = (odd ? q : p) + __shfl_xor_sync(all, odd ? p : q, 8);
    } else {
        p += __shfl_xor_sync(all, p, 8);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) p += __shfl_xor_sync(all, p, off);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = ALL_LANES ? __shfl_sync(all, p, owner(k)) : p;
}

// Sums K values over a row's threads: within each warp, then over the warps' sums in shared
// memory -- up to 8 of them (MAXT <= 256) added by every thread from two 16-byte reads a value,
// which the whole warp makes at one address; more by the shuffles again. `red` (cleared by
// red_init()) alternates between two halves that hold KMAX values each, the most that a kernel
// sums at once, so that calls of different K do not meet and one barrier a call is enough
// (red_place has the argument).
template <int K, int KMAX, int MAXT>
__device__ __forceinline__ void row_sum(float (&v)[K], float (&red)[kRedFloats<KMAX>], int& half)
{
    static_assert(K <= KMAX, "a half of the buffer holds KMAX values");
    warp_sum<K, MAXT == 32>(v);
    if (MAXT == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = half;
    half ^= 1;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (lane == owner(k)) red[red_place<KMAX>(h, k, warp)] = v[k];
    __syncthreads();
    if (MAXT <= 256) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float4 p = *reinterpret_cast<const float4*>(red + red_place<KMAX>(h, k, 0));
            const float4 q = *reinterpret_cast<const float4*>(red + red_place<KMAX>(h, k, 4));
            v[k] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = red[red_place<KMAX>(h, k, lane)];
        warp_sum<K, true>(v);
    }
}

// zeros for the warps that a block does not have (visible after row_sum's first barrier)
template <int FLOATS>
__device__ __forceinline__ void red_init(float (&red)[FLOATS])
{
    const int warps = blockDim.x >> 5;
    for (int i = threadIdx.x; i < FLOATS; i += blockDim.x)
        if ((i & (kRed - 1)) >= warps) red[i] = 0.0f;
}

__device__ __forceinline__ float inv_rms(float ss, const NormArgs& a)
{
    return rsqrtf(ss * a.inv_h + a.eps);
}

__device__ __forceinline__ uint32_t row_id(const NormArgs& a, int64_t t)
{
    return a.row_ids != nullptr ? (uint32_t)a.row_ids[t] : a.first_row + (uint32_t)t;
}

// the kept elements of a vector, 0 elsewhere (a select: dropped infinities and NaNs give 0)
__device__ __forceinline__ void drop2(const uint32_t (&w)[4], uint32_t threshold, F2 (&f)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpack(f[i], lo, hi);
        f[i] = f2(philox_keep(w, 2 * i, threshold) ? lo : 0.0f,
                  philox_keep(w, 2 * i + 1, threshold) ? hi : 0.0f);
    }
}

// What a call has: kAny looks as it goes; kAll and kAllDrop are calls with both norms (backward: dr
// and room for the ring too) and fp32 parameters, without and with dropout. In the kernel of a block
// a row they also mean rows that fill their threads, elsewhere FULL says so. Looking costs the
// backward: a fifth of its instructions were branches and their constants (16384 x 1000 bf16 90 us
// with it, 62 without). A block without w_post, or with weights of the rows' type, takes kAny.
enum { kAny = 0, kAll = 1, kAllDrop = 2 };

constexpr int kRowsAhead = 2;  // rows on their way in residual_norm_rows_kernel

// one row per block of blockDim.x <= MAXT threads, or (MAXT = 32) one per warp, threadIdx.y the row
template <int DT, int V, int MAXT, int MODE>
__global__ void __launch_bounds__(MAXT == 32 ? 128 : MAXT)
    residual_norm_kernel(const __grid_constant__ NormArgs a)
{
    constexpr bool ONEWARP = MAXT == 32, ALL = MODE != kAny;
    const bool post = ALL || a.w_post != nullptr, next = ALL || a.w_next != nullptr;
    const bool branch = ALL || a.y != nullptr, param_f32 = ALL || a.param_f32;
    const bool drop = MODE == kAllDrop || (MODE == kAny && a.threshold != 0);
    __shared__ __align__(16) float red[kRedFloats<1>];
    int half = 0;
    red_init(red);
    pdl_wait();
    const int64_t t = ONEWARP ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (t >= a.T) return;  // whole warps (ONEWARP); never otherwise
    const int tid = threadIdx.x, step = blockDim.x;
    const int64_t row = t * a.nvec;
    Vec8<DT> x[V], y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (ALL || v < a.nvec) {
            x[i].load(a.x, row + v);
            if (branch) y[i].load(a.y, row + v);
        }
    }
    if (branch) {
        float scale = a.branch_scale * (drop ? a.inv_keep : 1.0f);
        if (post) {
            F2 acc = f2(0.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (ALL || tid + i * step < a.nvec) {
                    F2 q[4];
                    get2(y[i], q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = fma2(q[e], q[e], acc);
                }
            }
            float ss[1] = {sum2(acc)};
            row_sum<1, 1, MAXT>(ss, red, half);
            scale *= inv_rms(ss[0], a);
        }
        if (a.gate_mode == MOE_GATE_TOKEN) scale *= load_param<DT>(a.gate, param_f32, t);
        uint32_t mask[V][4];
        if (drop) {
            const uint32_t rid = row_id(a, t);
            uint32_t col[V], rows[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                col[i] = (uint32_t)(tid + i * step);
                rows[i] = rid;
            }
            philox8n<V>(philox_load(a.rng), col, rows, mask);
        }
        const F2 sc = f2(scale), rs = f2(a.residual_scale);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (ALL || v < a.nvec) {
                F2 z[4], q[4];
                get2(y[i], z);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = mul2(z[e], sc);
                if (post) {
                    load_param2<DT>(a.w_post, param_f32, v, q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = mul2(z[e], q[e]);
                }
                if (drop) drop2(mask[i], a.threshold, z);
                if (a.gate_mode >= MOE_GATE_CHANNEL && a.gate_mode != MOE_GATE_TOKEN) {
                    if (a.gate_mode == MOE_GATE_CHANNEL) {
                        load_param2<DT>(a.gate, param_f32, v, q);
                    } else {
                        Vec8<DT> g;
                        g.load(a.gate, row + v);
                        get2(g, q);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = mul2(z[e], q[e]);
                }
                get2(x[i], q);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = fma2(rs, q[e], z[e]);
                set2(x[i], q);
                x[i].store(a.r, row + v);
            }
        }
    }
    if (!next) return;
    F2 acc = f2(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (ALL || tid + i * step < a.nvec) {
            F2 q[4];
            get2(x[i], q);  // the rounded r
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = fma2(q[e], q[e], acc);
        }
    }
    float ss[1] = {sum2(acc)};
    row_sum<1, 1, MAXT>(ss, red, half);
    const F2 inv = f2(inv_rms(ss[0], a));
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (ALL || v < a.nvec) {
            F2 q[4], w[4];
            get2(x[i], q);
            load_param2<DT>(a.w_next, param_f32, v, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = mul2(mul2(q[e], inv), w[e]);
            set2(x[i], q);
            x[i].store(a.n, row + v);
        }
    }
}

// The same over many rows: a block takes one row after the other, with the weights in registers
// and the next rows on their way to shared memory (cp.async; a warp copies its own vectors, so
// no barrier). The arithmetic is the kernel's above, value for value; a place past the row's end
// holds zeros, which add nothing, and only its stores are left out. 16 warps an SM with 128
// registers each and no look at the weights again: 16384 x 2048 bf16 44.8 us, against 55 for the
// kernel above at 32 warps (8192 x 4096: 46.8 against 59). FULL: rows fill their threads (with
// the looks at the row's end the first takes 46.5).
template <int DT, int MAXT, int MODE, bool FULL>
__global__ void __launch_bounds__(MAXT, 512 / MAXT)
    residual_norm_rows_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int V = 2, W16 = DT == MOE_F32 ? 2 : 1;  // vectors a thread, their 16-byte words
    constexpr bool ALL = MODE != kAny;
    const bool post = ALL || a.w_post != nullptr, next = ALL || a.w_next != nullptr;
    const bool branch = ALL || a.y != nullptr, param_f32 = ALL || a.param_f32;
    const bool drop = MODE == kAllDrop || (MODE == kAny && a.threshold != 0);
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[kRedFloats<1>];
    int half = 0;
    red_init(red);
    pdl_wait();
    const int tid = threadIdx.x, step = blockDim.x, nvec = a.nvec, gate_mode = a.gate_mode;
    const bool last_in = FULL || tid + step < nvec;  // the first vector always is
    F2 wp[V][4], wn[V][4], wg[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) wp[i][e] = wn[i][e] = wg[i][e] = f2(0.0f);
        if (i == 0 || last_in) {
            const int v = tid + i * step;
            if (post) load_param2<DT>(a.w_post, param_f32, v, wp[i]);
            if (next) load_param2<DT>(a.w_next, param_f32, v, wn[i]);
            if (gate_mode == MOE_GATE_CHANNEL) load_param2<DT>(a.gate, param_f32, v, wg[i]);
        }
    }
    Philox ph;
    if (drop) ph = philox_load(a.rng);
    // A stage: x and y, V vectors a thread each. A warp's 32 vectors are W16 x 32 words in a row;
    // lane l copies words l (and 32 + l), so that a copy's bytes are consecutive, and reads words
    // W16 l and up, its own vector.
    const int lane = tid & 31, first = tid - lane;
    const uint32_t array16 = (uint32_t)(W16 * step) * 16u, stage_bytes = 2 * V * array16;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring) + (uint32_t)first * (W16 * 16u);
    const uint32_t end = base + kRowsAhead * stage_bytes;
    if (!FULL) {  // the places past a row's end stay zero
        for (int k = tid; k < (int)(kRowsAhead * stage_bytes / 16u); k += step)
            ring[k] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
    }
    auto fetch = [&](uint32_t at, int64_t t) {
        if (t < a.T) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int h = 0; h < W16; ++h) {
                        const int word = (first + i * step) * W16 + 32 * h + lane;
                        if ((FULL || word < nvec * W16) && (k == 0 || branch))
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             at + (uint32_t)(k * V + i) * array16 +
                                             (uint32_t)(32 * h + lane) * 16u),
                                         "l"(static_cast<const uint4*>(k ? a.y : a.x) +
                                             t * nvec * W16 + word)
                                         : "memory");
                    }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t at = base;
    auto get = [&](int k, int i, F2 (&f)[4]) {
        uint4 w[W16];
#pragma unroll
        for (int h = 0; h < W16; ++h)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[h].x), "=r"(w[h].y), "=r"(w[h].z), "=r"(w[h].w)
                         : "r"(at + (uint32_t)(k * V + i) * array16 +
                               (uint32_t)(W16 * lane + h) * 16u)
                         : "memory");
        Vec8<DT> q;
        q.load(w, 0);
        get2(q, f);
    };
    for (int s = 0; s < kRowsAhead; ++s)
        fetch(base + (uint32_t)s * stage_bytes, blockIdx.x + (int64_t)s * gridDim.x);
    const F2 rs = f2(a.residual_scale);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRowsAhead - 1) : "memory");
        if (W16 > 1) __syncwarp();
        const int64_t row = t * nvec;
        Vec8<DT> o[V];
        F2 acc = f2(0.0f);
        float ss[1];
        if (branch) {
            F2 z[V][4];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                get(1, i, z[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = fma2(z[i][e], z[i][e], acc);
            }
            uint32_t mask[V][4];
            if (drop) {
                const uint32_t rid = row_id(a, t);
                uint32_t col[V], rows[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    col[i] = (uint32_t)(tid + i * step);
                    rows[i] = rid;
                }
                philox8n<V>(ph, col, rows, mask);
            }
            float scale = a.branch_scale * (drop ? a.inv_keep : 1.0f);
            if (post) {
                ss[0] = sum2(acc);
                row_sum<1, 1, MAXT>(ss, red, half);
                scale *= inv_rms(ss[0], a);
            }
            if (gate_mode == MOE_GATE_TOKEN) scale *= load_param<DT>(a.gate, param_f32, t);
            const F2 sc = f2(scale);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                F2 q[4];
                const int64_t v = row + tid + i * step;
#pragma unroll
                for (int e = 0; e < 4; ++e) z[i][e] = mul2(z[i][e], sc);
                if (post) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[i][e] = mul2(z[i][e], wp[i][e]);
                }
                if (drop) drop2(mask[i], a.threshold, z[i]);
                if (gate_mode == MOE_GATE_CHANNEL) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[i][e] = mul2(z[i][e], wg[i][e]);
                } else if (gate_mode == MOE_GATE_FULL && (i == 0 || last_in)) {
                    o[i].load(a.gate, v);
                    get2(o[i], q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[i][e] = mul2(z[i][e], q[e]);
                }
                get(0, i, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = fma2(rs, q[e], z[i][e]);
                set2(o[i], q);
                if (i == 0 || last_in) o[i].store(a.r, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                F2 q[4];
                get(0, i, q);
                set2(o[i], q);
            }
        }
        acc = f2(0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            F2 q[4];
            get2(o[i], q);  // the rounded r (past the row's end 0 times a NaN scale may be NaN)
            if (i == 0 || last_in) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc = fma2(q[e], q[e], acc);
            }
        }
        if (W16 > 1) __syncwarp();  // the warp has read the stage
        fetch(at, t + (int64_t)kRowsAhead * gridDim.x);
        at += stage_bytes;
        if (at == end) at = base;
        if (!next) continue;
        ss[0] = sum2(acc);
        row_sum<1, 1, MAXT>(ss, red, half);
        const F2 inv = f2(inv_rms(ss[0], a));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            F2 q[4];
            get2(o[i], q);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = mul2(mul2(q[e], inv), wn[i][e]);
            set2(o[i], q);
            if (i == 0 || last_in) o[i].store(a.n, row + tid + i * step);
        }
    }
}

// Backward of one row after the other:
//   d  = dr + s w_next dn - r s^3 mean(w_next dn r)      s = 1 / sqrt(mean(r^2) + eps)
//   dx = residual_scale d,  b = branch_scale d
//   dgate = b z (summed over tokens, over columns, or kept),  c = drop'(b gate)
//   dy = u w_post c - y u^3 mean(w_post c y)             u = 1 / sqrt(mean(y^2) + eps)
//   dw_next = sum_t dn r s,  dw_post = sum_t c y u
//
// A thread's three accumulators for each of its columns take most of its registers, so few
// warps fit on an SM and loads have to be in flight without them: each warp copies its own
// vectors of the next rows to a ring in shared memory (cp.async, no barrier) and reads them back,
// twice, when their row comes. Consecutive lanes copy consecutive words: of fp32, where a vector is
// two words, a lane copies one of its own and one of another's (8192 x 2048: 76 us, 112 with
// every lane copying its own two). The ring has as many stages, up to 4, as fit in shared memory;
// rows of which not even one fits are read from memory (fp32 with r, dn, dr and y above H = 14336,
// with a full gate besides above 11264).
//
// Above H = 8192 a block has more than 512 threads, 64 registers each, and the sums spill (496 to
// 656 bytes of stores a thread): 4096 x 12288 bf16 261 us, 16384 341; 2048 x 12288 fp32 212, 16384
// 360; against 92, 123, 92 and 123 us at the copy's rate.
struct BwdRing {
    int32_t stages, arrays;               // stages 0: no ring
    int32_t i_r, i_dn, i_dr, i_y, i_gate; // place of each array in a stage, -1: absent
};

template <int DT, int V, int MAXT, int MODE, bool FULL>
__global__ void __launch_bounds__(MAXT == 32 ? 128 : MAXT, MAXT == 32    ? 4
                                                           : MAXT == 256 ? 2
                                                                         : 1)
    residual_norm_bwd_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ BwdRing g)
{
    constexpr bool ONEWARP = MAXT == 32, ALL = MODE != kAny;
    constexpr int W16 = DT == MOE_F32 ? 2 : 1;  // 16-byte words of a vector
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[kRedFloats<3>];
    int half = 0;
    red_init(red);
    pdl_wait();
    const int tid = threadIdx.x, step = blockDim.x;
    const int lin = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const int64_t rows = ONEWARP ? (int64_t)gridDim.x * blockDim.y : gridDim.x;
    const int64_t first = ONEWARP ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    const bool post = ALL || a.w_post != nullptr, next = ALL || a.w_next != nullptr;
    const bool branch = ALL || a.y != nullptr, has_dr = ALL || a.dr != nullptr;
    const bool drop = MODE == kAllDrop || (MODE == kAny && a.threshold != 0);
    const bool has_ring = ALL || g.stages > 0, param_f32 = ALL || a.param_f32;
    const int nvec = a.nvec, gate_mode = a.gate_mode;
    const uint32_t threshold = a.threshold;
    // places of the arrays in a stage
    const int at_r = ALL ? 0 : g.i_r, at_dn = ALL ? 1 : g.i_dn, at_dr = ALL ? 2 : g.i_dr,
              at_y = ALL ? 3 : g.i_y;
    F2 gn[V][4], gp[V][4], gg[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) gn[i][e] = gp[i][e] = gg[i][e] = f2(0.0f);
    // with one vector a thread its weights and channel gate stay in registers
    constexpr bool KEEP = ALL && V == 1;
    F2 kn[4], kp[4], kg[4];
    if (KEEP && (FULL || tid < nvec)) {
        load_param2<DT>(a.w_next, true, tid, kn);
        load_param2<DT>(a.w_post, true, tid, kp);
        if (gate_mode == MOE_GATE_CHANNEL) load_param2<DT>(a.gate, true, tid, kg);
    }
    // (this thread's place in the ring: 16 bytes per thread, arrays and vectors `lane16` apart)
    // with two, in its own slots of shared memory behind the ring (read from memory they come
    // from L2: beside the ring, L1 holds less than a row's weights)
    constexpr bool SLOTS = ALL && V == 2 && MAXT != 1024;
    const uint32_t lane16 = (uint32_t)threads * 16u;
    const int lane = tid & 31;
    // from a lane's own place to its vector's first word (fp32: words 2 l and 2 l + 1 of 64)
    const uint32_t own = W16 == 1 ? 0u
                                  : (lane < 16 ? 0u : lane16) + 16u * (uint32_t)(2 * lane & 31) -
                                        16u * (uint32_t)lane;
    const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(ring) + (uint32_t)lin * 16u;
    const uint32_t stage_bytes = (uint32_t)(g.arrays * V * W16) * lane16;
    const uint32_t slots0 = ring0 + (uint32_t)g.stages * stage_bytes;
    auto param_slot = [&](int which, int i, int h) {
        return slots0 + (uint32_t)((which * V + i) * 2 + h) * lane16;
    };
    if (SLOTS) {
        auto stage_in = [&](int which, const void* p) {
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (FULL || tid + i * step < nvec)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                                         param_slot(which, i, h)),
                                     "l"(static_cast<const uint4*>(p) + 2 * (tid + i * step) + h)
                                     : "memory");
        };
        stage_in(0, a.w_next);
        stage_in(1, a.w_post);
        if (gate_mode == MOE_GATE_CHANNEL) stage_in(2, a.gate);
        asm volatile("cp.async.commit_group;" ::: "memory");  // older than every row's group
    }
    auto param = [&](const void* p, const F2 (&kept)[4], int which, int i, F2 (&w)[4]) {
        if (KEEP) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = kept[e];
        } else if (SLOTS) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                             : "=l"(w[2 * h].v), "=l"(w[2 * h + 1].v)
                             : "r"(param_slot(which, i, h))
                             : "memory");
        } else {
            load_param2<DT>(p, param_f32, tid + i * step, w);
        }
    };
    Philox ph;
    if (drop) ph = philox_load(a.rng);

    auto fetch = [&](uint32_t at, int64_t t) {
        auto one = [&](int array, const void* p) {
            if (array < 0) return;
            const uint4* src = static_cast<const uint4*>(p) + t * nvec * W16;
#pragma unroll
            for (int i = 0; i < V; ++i) {
#pragma unroll
                for (int h = 0; h < W16; ++h) {
                    const int word = (tid - lane + i * step) * W16 + 32 * h + lane;
                    if (FULL || word < nvec * W16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         at + (uint32_t)((array * V + i) * W16 + h) * lane16),
                                     "l"(src + word)
                                     : "memory");
                }
            }
        };
        if (t < a.T) {
            one(at_r, a.r);
            one(at_dn, a.dn);
            one(at_dr, a.dr);
            one(at_y, a.y);
            one(g.i_gate, a.gate);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto row_ready = [&]() {  // at most stages - 1 newer rows still in flight
        switch (g.stages) {
            case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
            case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
            case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
            default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        }
    };
    uint32_t at = ring0;  // the current row's stage
    auto get = [&](int array, const void* p, int64_t row, int i, F2 (&f)[4]) {
        Vec8<DT> q;
        if (has_ring) {
            uint4 w[W16];
#pragma unroll
            for (int h = 0; h < W16; ++h)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[h].x), "=r"(w[h].y), "=r"(w[h].z), "=r"(w[h].w)
                             : "r"(at + (uint32_t)((array * V + i) * W16) * lane16 + own +
                                   16u * (uint32_t)h)
                             : "memory");
            q.load(w, 0);
        } else {
            q.load(p, row + tid + i * step);
        }
        get2(q, f);
    };
    for (int s = 0; s < g.stages; ++s) fetch(ring0 + (uint32_t)s * stage_bytes, first + s * rows);

    const F2 rscale = f2(a.residual_scale);
    const F2 bscale = f2(a.branch_scale * (drop ? a.inv_keep : 1.0f));  // with 1 / P(keep)
    for (int64_t t = first; t < a.T; t += rows) {
        const int64_t row = t * nvec;
        if (has_ring) {
            row_ready();
            if (W16 > 1) __syncwarp();
        }
        F2 rr = f2(0.0f), wr = f2(0.0f), yy = f2(0.0f);  // r^2, w_next dn r, y^2
        F2 kr[4], kd[4];  // KEEP: r and dn between the passes
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (FULL || v < nvec) {
                F2 p[4], q[4], w[4];
                if (next) {
                    get(at_r, a.r, row, i, p);
                    get(at_dn, a.dn, row, i, q);
                    param(a.w_next, kn, 0, i, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        rr = fma2(p[e], p[e], rr);
                        wr = fma2(mul2(q[e], w[e]), p[e], wr);
                        if (KEEP) {
                            kr[e] = p[e];
                            kd[e] = q[e];
                        }
                    }
                }
                if (post) {
                    get(at_y, a.y, row, i, p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) yy = fma2(p[e], p[e], yy);
                }
            }
        }
        float s3[3] = {sum2(rr), sum2(wr), sum2(yy)};
        if (next || post) row_sum<3, 3, MAXT>(s3, red, half);
        const float s = next ? inv_rms(s3[0], a) : 0.0f;
        // (from the sum outwards: s^3 by itself is subnormal for rows of 1e13 and infinite for
        // rows of zeros with an eps below 1e-25)
        const F2 s2x = f2(s), mean_n = f2(next ? -(s * (s * (s * (s3[1] * a.inv_h)))) : 0.0f);
        const float u = post ? inv_rms(s3[2], a) : 1.0f;
        const F2 u2x = f2(u);
        const F2 tg = f2(gate_mode == MOE_GATE_TOKEN ? load_param<DT>(a.gate, param_f32, t)
                                                       : 1.0f);
        const uint32_t rid = drop ? row_id(a, t) : 0u;
        F2 cy = f2(0.0f), bz = f2(0.0f);  // w_post c y, b z
        F2 c[V][4];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (FULL || v < nvec) {
                F2 d[4], q[4];
                if (has_dr) {
                    get(at_dr, a.dr, row, i, d);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = f2(0.0f);
                }
                if (next) {
                    F2 p[4], w[4];
                    if (KEEP) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[e] = kr[e];
                            q[e] = kd[e];
                        }
                    } else {
                        get(at_r, a.r, row, i, p);
                        get(at_dn, a.dn, row, i, q);
                    }
                    param(a.w_next, kn, 0, i, w);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const F2 k = mul2(q[e], s2x);
                        d[e] = fma2(k, w[e], d[e]);
                        d[e] = fma2(p[e], mean_n, d[e]);
                        gn[i][e] = fma2(k, p[e], gn[i][e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) q[e] = mul2(rscale, d[e]);
                Vec8<DT> o;
                set2(o, q);
                o.store(a.dx, row + v);
                if (branch) {
                    F2 yu[4], w[4];
                    uint32_t bitsw[4] = {0u, 0u, 0u, 0u};
                    if (drop) philox8(ph, (uint32_t)v, rid, bitsw);
                    get(at_y, a.y, row, i, yu);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        d[e] = mul2(d[e], bscale);
                        yu[e] = mul2(yu[e], u2x);
                    }
                    if (post) param(a.w_post, kp, 1, i, w);
                    if (drop) drop2(bitsw, threshold, d);
                    if (gate_mode != MOE_GATE_NONE) {
                        // b z: the factor 1 / P(keep) of z is already in d, dropped ones are 0
                        F2 z[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[e] = post ? mul2(yu[e], w[e]) : yu[e];
                        if (drop) drop2(bitsw, threshold, z);
                        if (gate_mode == MOE_GATE_FULL) {
                            get(g.i_gate, a.gate, row, i, q);
#pragma unroll
                            for (int e = 0; e < 4; ++e) z[e] = mul2(z[e], d[e]);
                            set2(o, z);
                            o.store(a.dgate, row + v);
                        } else if (gate_mode == MOE_GATE_CHANNEL) {
                            param(a.gate, kg, 2, i, q);
#pragma unroll
                            for (int e = 0; e < 4; ++e) gg[i][e] = fma2(d[e], z[e], gg[i][e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                bz = fma2(d[e], z[e], bz);
                                q[e] = tg;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[e] = mul2(d[e], q[e]);
                    }
                    if (post) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            gp[i][e] = fma2(d[e], yu[e], gp[i][e]);
                            c[i][e] = mul2(d[e], w[e]);
                            cy = fma2(c[i][e], yu[e], cy);
                        }
                    } else {
                        set2(o, d);
                        o.store(a.dy, row + v);
                    }
                }
            }
        }
        float s2[2] = {sum2(cy), sum2(bz)};
        if (post || gate_mode == MOE_GATE_TOKEN) row_sum<2, 3, MAXT>(s2, red, half);
        if (gate_mode == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(a.dgate)[t] = s2[1];
        if (post) {
            // dy = u c - y u^2 mean(c y u): the sum above already holds one factor u
            const F2 mean_p = f2(-(u * (u * (s2[0] * a.inv_h))));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + i * step;
                if (FULL || v < nvec) {
                    F2 y[4];
                    get(at_y, a.y, row, i, y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = fma2(y[e], mean_p, mul2(c[i][e], u2x));
                    Vec8<DT> o;
                    set2(o, y);
                    o.store(a.dy, row + v);
                }
            }
        }
        if (has_ring) {
            if (W16 > 1) __syncwarp();  // the warp has read the stage
            fetch(at, t + g.stages * rows);
            at += stage_bytes;
            if (at == ring0 + (uint32_t)g.stages * stage_bytes) at = ring0;
        }
    }

    // this row group's partial sums
    float* part = a.part + first * a.slots * (int64_t)a.H;
    auto put = [&](int where, const F2 (&p)[V][4]) {
        if (where < 0) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (v < a.nvec) {
                float4* d = reinterpret_cast<float4*>(part + (int64_t)where * a.H) + 2 * v;
                Vec8<MOE_F32> f;
                set2(f, p[i]);
                d[0] = f.a;
                d[1] = f.b;
            }
        }
    };
    put(a.slot_next, gn);
    put(a.slot_post, gp);
    put(a.slot_gate, gg);
}

// out[slot][column] = sum over the partial rows in order: a warp takes 32 columns of a slice of
// the rows, the slices of a block are added in order. Bound by the latency of the loads, hence
// 20 rows of a slice at once (all 19 of them at the 296 partials of 4096 columns; the 592 of
// narrower rows take two rounds) and blocks that are all resident together: 6 us for 296 x 3 x 4096
// right behind the backward, with the partials in L2 (9.2 from memory); two more with 32 slices of
// 8 loads at a time.
struct ReduceArgs {
    const float* part;
    int32_t parts, slots, H;
    float* out[3];
};

constexpr int kSlices = 16;
constexpr int kBatch = 20;  // rows in flight a thread

__global__ void __launch_bounds__(32 * kSlices) param_grad_kernel(ReduceArgs a)
{
    __shared__ float red[kSlices][33];
    pdl_wait();
    const int lane = threadIdx.x, slice = threadIdx.y;
    const int col = blockIdx.x * 32 + lane, slot = blockIdx.y;
    const int per = (a.parts + kSlices - 1) / kSlices;
    const int beg = slice * per, end = beg + per < a.parts ? beg + per : a.parts;
    float s = 0.0f;
    if (col < a.H) {
        const float* p = a.part + (int64_t)slot * a.H + col;
        const int64_t stride = (int64_t)a.slots * a.H;
        for (int i = beg; i < end; i += kBatch) {
            float f[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) f[j] = i + j < end ? p[(i + j) * stride] : 0.0f;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) s += f[j];
        }
    }
    red[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && col < a.H) {
        s = red[0][lane];
#pragma unroll
        for (int i = 1; i < kSlices; ++i) s += red[i][lane];
        a.out[slot][col] = s;
    }
}

// out = keep ? x / probability : 0, each thread kVec vectors of 8, a block's width apart. A bf16
// tensor moves 4 bytes an element and takes 15 instructions for it, 5 of them Philox's products
// and xors (27.7 us for 16384 x 2048, 4.8 TB/s, 0.74 of the copy's rate; 34 us with the keys formed
// per vector and a division per vector). No unit is full: the SM is at 0.53 of its throughput, with
// 43 % of its warps resident; latency is left, of the loads or of Philox's dependent rounds.
constexpr int kVec = 4;

template <int DT>
__global__ void __launch_bounds__(256) dropout_kernel(const void* x, void* out, int64_t total,
                                                      FastDiv nvec, uint32_t threshold,
                                                      float inv_keep, const int64_t* rng,
                                                      uint32_t first_row, const int32_t* row_ids)
{
    pdl_wait();
    const Philox ph = philox_load(rng);
    const int64_t base = (int64_t)blockIdx.x * (256 * kVec) + threadIdx.x;
    Vec8<DT> q[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (base + 256 * i < total) q[i].load(x, base + 256 * i);
    uint32_t col[kVec], row[kVec], w[kVec][4];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int64_t g = base + 256 * i < total ? base + 256 * i : 0;
        const int64_t t = quotient(g, nvec, total <= 0x7fffffffll);
        col[i] = (uint32_t)(g - t * nvec.d);
        row[i] = row_ids != nullptr ? (uint32_t)row_ids[t] : first_row + (uint32_t)t;
    }
    philox8n<kVec>(ph, col, row, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (base + 256 * i < total) {
            float f[8];
            q[i].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = philox_keep(w[i], e, threshold) ? f[e] * inv_keep : 0.0f;
            q[i].set(f);
            q[i].store(out, base + 256 * i);
        }
    }
}

// threads and vectors per thread of a row of nvec vectors: one warp up to 64 vectors (H = 512),
// beyond that a block with two vectors a thread
struct RowShape {
    bool one_warp;
    int V, threads;
};

RowShape row_shape(int nvec)
{
    if (nvec <= 32) return {true, 1, 32};
    if (nvec <= 64) return {true, 2, 32};
    return {false, 2, ((nvec + 1) / 2 + 31) / 32 * 32};
}

constexpr int kWarpRows = 4;  // rows of a block in the one-warp form

// The backward: one vector a thread (its 24 sums and 24 weights in registers) up to H = 512, or in
// fp32, where the ring leaves no room for weights in shared memory, up to H = 2048; two beyond
// that. 16384 x 2048 with dropout and a channel gate, one vector against two: bf16 112 and 104
// us, fp32 140 and 213.
RowShape bwd_shape(int nvec, int dtype)
{
    if (nvec <= 32) return {true, 1, 32};
    if (nvec <= (dtype == MOE_F32 ? 256 : 64)) return {false, 1, (nvec + 31) / 32 * 32};
    return {false, 2, ((nvec + 1) / 2 + 31) / 32 * 32};
}

// row groups of the backward: a function of T, H and the type alone, so that the order of the
// parameter sums does not depend on the device (about 512 threads for each of a B200's 148 SMs,
// at least two rows a group)
int64_t bwd_groups(int64_t T, int32_t H, int dtype)
{
    const RowShape s = bwd_shape(H / 8, dtype);
    int64_t per_sm = 512 / s.threads;
    if (per_sm < 1) per_sm = 1;
    int64_t g = 148 * per_sm;
    if (g > (T + 1) / 2) g = (T + 1) / 2;
    if (s.one_warp) g = (g + kWarpRows - 1) / kWarpRows * kWarpRows;
    return g;
}

NormArgs base_args(const moe_norm_cfg& c)
{
    NormArgs a{};
    a.T = c.T;
    a.H = c.H;
    a.nvec = c.H / 8;
    a.first_row = (uint32_t)c.first_row;
    a.threshold = dropout_threshold(c.p);
    a.inv_keep = dropout_scale(a.threshold);
    a.gate_mode = c.gate;
    a.param_f32 = c.param_dtype == MOE_F32;
    a.eps = c.eps;
    a.inv_h = 1.0f / (float)c.H;
    a.residual_scale = c.residual_scale;
    a.branch_scale = c.branch_scale;
    return a;
}

template <int DT, int V, int MAXT>
cudaError_t norm_fwd_variant(const NormArgs& a, dim3 grid, dim3 block, cudaStream_t st)
{
    const bool all = a.w_post != nullptr && a.w_next != nullptr && a.param_f32 &&
                     a.nvec == V * (int)block.x;
    auto kernel = !all               ? residual_norm_kernel<DT, V, MAXT, kAny>
                  : a.threshold == 0 ? residual_norm_kernel<DT, V, MAXT, kAll>
                                     : residual_norm_kernel<DT, V, MAXT, kAllDrop>;
    return launch_pdl(kernel, grid, block, 0, st, a);
}

template <int DT, int MAXT>
cudaError_t norm_rows(const NormArgs& a, unsigned blocks, dim3 block, cudaStream_t st)
{
    const bool all = a.y != nullptr && a.w_post != nullptr && a.w_next != nullptr && a.param_f32;
    const bool drop = a.threshold != 0, full = a.nvec == 2 * (int)block.x;
    const int which = !all ? 0 : 1 + 2 * full + drop;
    auto kernel = !all   ? residual_norm_rows_kernel<DT, MAXT, kAny, false>
                  : full ? (drop ? residual_norm_rows_kernel<DT, MAXT, kAllDrop, true>
                                 : residual_norm_rows_kernel<DT, MAXT, kAll, true>)
                         : (drop ? residual_norm_rows_kernel<DT, MAXT, kAllDrop, false>
                                 : residual_norm_rows_kernel<DT, MAXT, kAll, false>);
    const size_t smem = (size_t)kRowsAhead * 4 * (DT == MOE_F32 ? 32 : 16) * block.x;
    if (smem > 48000) {  // fp32 above 187 threads, others above 375
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess) return err;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        static bool attr_set[5][64] = {};
        if (!attr_set[which][dev]) {
            err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kRowsAhead * 4 * 32 * MAXT);
            if (err != cudaSuccess) return err;
            attr_set[which][dev] = true;
        }
    }
    return launch_pdl(kernel, dim3(blocks), block, smem, st, a);
}

template <int DT>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st)
{
    const RowShape s = row_shape(a.nvec);
    if (s.one_warp) {
        const dim3 grid((unsigned)((a.T + kWarpRows - 1) / kWarpRows)), block(32, kWarpRows);
        return s.V == 1 ? norm_fwd_variant<DT, 1, 32>(a, grid, block, st)
                        : norm_fwd_variant<DT, 2, 32>(a, grid, block, st);
    }
    const dim3 grid((unsigned)a.T), block(s.threads);
    // With two rows or more for every block that fits, rows one after the other: of 2048 bf16, 600
    // rows (592 blocks) take 3.9 us by blocks of their own and 4.1 so, 1200 6.5 and 5.7, 4800 17.6
    // and 15.7, 16384 55 and 45.
    const int64_t blocks = 148 * (512 / s.threads);  // 0 above 512 threads
    if (blocks > 0 && a.T >= 2 * blocks)
        return s.threads <= 256 ? norm_rows<DT, 256>(a, (unsigned)blocks, block, st)
                                : norm_rows<DT, 512>(a, (unsigned)blocks, block, st);
    if (s.threads <= 256) return norm_fwd_variant<DT, 2, 256>(a, grid, block, st);
    if (s.threads <= 512) return norm_fwd_variant<DT, 2, 512>(a, grid, block, st);
    return norm_fwd_variant<DT, 2, 1024>(a, grid, block, st);
}

template <int DT, int V, int MAXT, int MODE, bool FULL>
cudaError_t norm_bwd_launch(const NormArgs& a, const BwdRing& g, dim3 grid, dim3 block, size_t smem,
                            cudaStream_t st)
{
    auto kernel = residual_norm_bwd_kernel<DT, V, MAXT, MODE, FULL>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool attr_set[64] = {};
    if (!attr_set[dev]) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   233472 - 1024 - 768);
        if (err != cudaSuccess) return err;
        attr_set[dev] = true;
    }
    return launch_pdl(kernel, grid, block, smem, st, a, g);
}

template <int DT, int V, int MAXT>
cudaError_t norm_bwd_variant(const NormArgs& a, BwdRing g, dim3 grid, dim3 block, cudaStream_t st)
{
    const int threads = (int)(block.x * block.y);
    const int per_sm = threads <= 512 ? 512 / threads : 1;
    const size_t stage = (size_t)g.arrays * V * (DT == MOE_F32 ? 32 : 16) * threads;
    // an SM's 228 KB, less a block's kilobyte and its static part, for per_sm blocks
    const size_t room = 233472 / per_sm - 1024 - 768;
    // the weights' slots of kAll and kAllDrop (V = 2)
    const size_t slots = V == 2 && MAXT != 1024
                             ? (size_t)(a.gate_mode == MOE_GATE_CHANNEL ? 3 : 2) * V * 32 * threads
                             : 0;
    auto stages_in = [&](size_t bytes) {
        const size_t n = stage > 0 ? bytes / stage : 0;
        return (int32_t)(n > 4 ? 4 : n);
    };
    g.stages = room > slots ? stages_in(room - slots) : 0;
    const bool all = a.w_post != nullptr && a.w_next != nullptr && a.dr != nullptr && a.param_f32 &&
                     g.stages > 0;
    if (!all) g.stages = stages_in(room);
    const size_t smem = g.stages * stage + (all ? slots : 0);
    if (!all) return norm_bwd_launch<DT, V, MAXT, kAny, false>(a, g, grid, block, smem, st);
    if (a.nvec == V * (int)block.x)
        return a.threshold != 0
                   ? norm_bwd_launch<DT, V, MAXT, kAllDrop, true>(a, g, grid, block, smem, st)
                   : norm_bwd_launch<DT, V, MAXT, kAll, true>(a, g, grid, block, smem, st);
    return a.threshold != 0
               ? norm_bwd_launch<DT, V, MAXT, kAllDrop, false>(a, g, grid, block, smem, st)
               : norm_bwd_launch<DT, V, MAXT, kAll, false>(a, g, grid, block, smem, st);
}

template <int DT>
cudaError_t norm_bwd(const NormArgs& a, int64_t groups, cudaStream_t st)
{
    BwdRing g{};
    auto take = [&](bool on) { return on ? g.arrays++ : -1; };
    g.i_r = take(a.w_next != nullptr);
    g.i_dn = take(a.w_next != nullptr);
    g.i_dr = take(a.dr != nullptr);
    g.i_y = take(a.y != nullptr);
    g.i_gate = take(a.gate_mode == MOE_GATE_FULL);
    const RowShape s = bwd_shape(a.nvec, DT);
    if (s.one_warp)
        return norm_bwd_variant<DT, 1, 32>(a, g, dim3((unsigned)(groups / kWarpRows)),
                                           dim3(32, kWarpRows), st);
    const dim3 grid((unsigned)groups), block(s.threads);
    if (s.V == 1) return norm_bwd_variant<DT, 1, 256>(a, g, grid, block, st);
    if (s.threads <= 256) return norm_bwd_variant<DT, 2, 256>(a, g, grid, block, st);
    if (s.threads <= 512) return norm_bwd_variant<DT, 2, 512>(a, g, grid, block, st);
    return norm_bwd_variant<DT, 2, 1024>(a, g, grid, block, st);
}

int bwd_slots(const moe_norm_cfg& c, bool post, bool next)
{
    return (post ? 1 : 0) + (next ? 1 : 0) + (c.gate == MOE_GATE_CHANNEL ? 1 : 0);
}

}  // namespace

uint32_t dropout_threshold(double p) { return (uint32_t)(p * 65536.0 + 0.5); }

float dropout_scale(uint32_t threshold)
{
    return threshold >= 65536u ? 0.0f : (float)(65536.0 / (65536.0 - (double)threshold));
}

size_t residual_norm_bwd_ws_bytes(const moe_norm_cfg& c)
{
    return (size_t)bwd_groups(c.T, c.H, c.dtype) * 3 * (size_t)c.H * sizeof(float);
}

cudaError_t launch_residual_norm(const moe_norm_cfg& c, const void* x, const void* y,
                                 const void* w_post, const void* gate, const void* w_next,
                                 const int64_t* rng, const int32_t* row_ids, void* r, void* n,
                                 cudaStream_t st)
{
    NormArgs a = base_args(c);
    a.x = x;
    a.y = y;
    a.w_post = w_post;
    a.gate = gate;
    a.w_next = w_next;
    a.rng = rng;
    a.row_ids = row_ids;
    a.r = r;
    a.n = n;
    switch (c.dtype) {
        case MOE_BF16: return norm_fwd<MOE_BF16>(a, st);
        case MOE_F16: return norm_fwd<MOE_F16>(a, st);
        default: return norm_fwd<MOE_F32>(a, st);
    }
}

cudaError_t launch_residual_norm_bwd(const moe_norm_cfg& c, const void* r, const void* y,
                                     const void* w_post, const void* gate, const void* w_next,
                                     const int64_t* rng, const int32_t* row_ids, const void* dr,
                                     const void* dn, void* dx, void* dy, float* dw_post,
                                     void* dgate, float* dw_next, void* ws, cudaStream_t st)
{
    const int64_t groups = bwd_groups(c.T, c.H, c.dtype);
    NormArgs a = base_args(c);
    a.r = const_cast<void*>(r);
    a.y = y;
    a.w_post = w_post;
    a.gate = gate;
    a.w_next = w_next;
    a.rng = rng;
    a.row_ids = row_ids;
    a.dr = dr;
    a.dn = dn;
    a.dx = dx;
    a.dy = dy;
    a.dgate = dgate;
    a.part = static_cast<float*>(ws);
    ReduceArgs ra{};
    int slot = 0;
    auto take = [&](bool on, float* out) {
        if (!on) return -1;
        ra.out[slot] = out;
        return slot++;
    };
    a.slot_next = take(w_next != nullptr, dw_next);
    a.slot_post = take(w_post != nullptr, dw_post);
    a.slot_gate = take(c.gate == MOE_GATE_CHANNEL, static_cast<float*>(dgate));
    a.slots = bwd_slots(c, w_post != nullptr, w_next != nullptr);
    cudaError_t e;
    switch (c.dtype) {
        case MOE_BF16: e = norm_bwd<MOE_BF16>(a, groups, st); break;
        case MOE_F16: e = norm_bwd<MOE_F16>(a, groups, st); break;
        default: e = norm_bwd<MOE_F32>(a, groups, st); break;
    }
    if (e != cudaSuccess || slot == 0) return e;
    ra.part = a.part;
    ra.parts = (int32_t)groups;
    ra.slots = slot;
    ra.H = c.H;
    return launch_pdl(param_grad_kernel, dim3((unsigned)((c.H + 31) / 32), (unsigned)slot),
                      dim3(32, kSlices), 0, st, ra);
}

cudaError_t launch_dropout(int64_t T, int32_t H, int dtype, double p, const void* x,
                           const int64_t* rng, int64_t first_row, const int32_t* row_ids,
                           void* out, cudaStream_t st)
{
    const int32_t nvec = H / 8;
    const int64_t total = T * nvec;
    const uint32_t th = dropout_threshold(p);
    const float inv = dropout_scale(th);
    const dim3 grid((unsigned)((total + 256 * kVec - 1) / (256 * kVec)));
    const uint32_t fr = (uint32_t)first_row;
    switch (dtype) {
        case MOE_BF16:
            return launch_pdl(dropout_kernel<MOE_BF16>, grid, dim3(256), 0, st, x, out, total,
                              FastDiv((uint32_t)nvec), th, inv, rng, fr, row_ids);
        case MOE_F16:
            return launch_pdl(dropout_kernel<MOE_F16>, grid, dim3(256), 0, st, x, out, total,
                              FastDiv((uint32_t)nvec), th, inv, rng, fr, row_ids);
        default:
            return launch_pdl(dropout_kernel<MOE_F32>, grid, dim3(256), 0, st, x, out, total,
                              FastDiv((uint32_t)nvec), th, inv, rng, fr, row_ids);
    }
}

}  // namespace moe
