// What joins two blocks of the residual stream, and its gradients: the norm after a block, its
// gate, dropout and residual scale, the residual sum and the next block's norm, in one pass.
//
//   z = drop(rms(y) w_post),  rms(v) = v / sqrt(mean(v^2) + eps)
//   r = round(residual_scale x + branch_scale gate z),  n = round(rms(r) w_next)
//
// n is taken from the rounded r, so the fused call gives the bits of the two calls it replaces.
// Every sum is fp32 in an order that depends on H alone (a thread's own vectors, a shuffle
// tree in each warp, the same tree over the warps): a token's row never depends on T or on its neighbours.
//
// All of it is bound by memory: 4 row passes forward (x, y in; r, n out), 6 backward (y, r, dr,
// dn in; dx, dy out). A row stays in the registers of one block (one warp up to H = 512), so
// nothing is read twice. The backward recomputes both norms' statistics and the dropout mask
// from what it reads anyway: nothing but r and y is kept from the forward.
//
// Parameter gradients are column sums over tokens: block b of a grid whose size is a function
// of (T, H) adds rows b, b + blocks, ... into its registers and writes one partial row; a second
// kernel sums the partials in order. No atomics: the bits repeat, on any device.
#include "philox.cuh"
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

// Sums K values over a row's threads: a shuffle tree within each warp, then the same tree over
// the warps' sums, read from shared memory by every warp. `red` alternates between two halves,
// so one barrier a call is enough (a warp that writes a half again has passed the barrier of
// the call in between, which every reader of that half had reached).
template <int K>
__device__ __forceinline__ void warp_sum(float (&v)[K])
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
}

template <int K, bool ONEWARP>
__device__ __forceinline__ void row_sum(float (&v)[K], float* red, int& half)
{
    warp_sum<K>(v);
    if (ONEWARP) return;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* b = red + half * 32 * K;
    half ^= 1;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) b[k * 32 + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lane < warps ? b[k * 32 + lane] : 0.0f;
    warp_sum<K>(v);
}

__device__ __forceinline__ float inv_rms(float ss, const NormArgs& a)
{
    return rsqrtf(ss * a.inv_h + a.eps);
}

__device__ __forceinline__ uint32_t row_id(const NormArgs& a, int64_t t)
{
    return a.row_ids != nullptr ? (uint32_t)a.row_ids[t] : a.first_row + (uint32_t)t;
}

// a gate's 8 values for one vector of row t
template <int DT>
__device__ __forceinline__ void gate8(const NormArgs& a, int64_t t, int v, float token_gate,
                                      float (&g)[8])
{
    if (a.gate_mode == MOE_GATE_CHANNEL) {
        load_param8<DT>(a.gate, a.param_f32, v, g);
    } else if (a.gate_mode == MOE_GATE_FULL) {
        Vec8<DT> q;
        q.load(a.gate, t * a.nvec + v);
        q.get(g);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = token_gate;
    }
}

// one row per block of blockDim.x <= MAXT threads, or (MAXT = 32) one per warp, threadIdx.y the row
template <int DT, int V, int MAXT>
__global__ void __launch_bounds__(MAXT == 32 ? 128 : MAXT) residual_norm_kernel(NormArgs a)
{
    constexpr bool ONEWARP = MAXT == 32;
    __shared__ float red[2 * 32];
    int half = 0;
    pdl_wait();
    const int64_t t = ONEWARP ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (t >= a.T) return;  // whole warps (ONEWARP); never otherwise
    const int tid = threadIdx.x, step = blockDim.x;
    const int64_t row = t * a.nvec;
    Vec8<DT> x[V], y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v < a.nvec) {
            x[i].load(a.x, row + v);
            if (a.y != nullptr) y[i].load(a.y, row + v);
        }
    }
    float f[V][8];
    if (a.y != nullptr) {
        float inv = 1.0f;
        if (a.w_post != nullptr) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (tid + i * step < a.nvec) {
                    float q[8];
                    y[i].get(q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss[0] = fmaf(q[e], q[e], ss[0]);
                }
            }
            row_sum<1, ONEWARP>(ss, red, half);
            inv = inv_rms(ss[0], a);
        }
        const float tg = a.gate_mode == MOE_GATE_TOKEN ? load_param<DT>(a.gate, a.param_f32, t)
                                                       : 1.0f;
        Philox ph;
        if (a.threshold) ph = philox_load(a.rng);
        const uint32_t rid = row_id(a, t);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (v < a.nvec) {
                float z[8], q[8];
                y[i].get(z);
                if (a.w_post != nullptr) {
                    load_param8<DT>(a.w_post, a.param_f32, v, q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = z[e] * inv * q[e];
                }
                if (a.threshold) {
                    uint32_t w[4];
                    philox8(ph, (uint32_t)v, rid, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = philox_keep(w, e, a.threshold) ? z[e] * a.inv_keep : 0.0f;
                }
                if (a.gate_mode != MOE_GATE_NONE) {
                    gate8<DT>(a, t, v, tg, q);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] *= q[e];
                }
                x[i].get(q);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    q[e] = a.residual_scale * q[e] + a.branch_scale * z[e];
                x[i].set(q);
                x[i].store(a.r, row + v);
            }
        }
    }
    if (a.w_next == nullptr) return;
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (tid + i * step < a.nvec) {
            x[i].get(f[i]);  // the rounded r
#pragma unroll
            for (int e = 0; e < 8; ++e) ss[0] = fmaf(f[i][e], f[i][e], ss[0]);
        }
    }
    row_sum<1, ONEWARP>(ss, red, half);
    const float inv = inv_rms(ss[0], a);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = tid + i * step;
        if (v < a.nvec) {
            float q[8];
            load_param8<DT>(a.w_next, a.param_f32, v, q);
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = f[i][e] * inv * q[e];
            Vec8<DT> o;
            o.set(q);
            o.store(a.n, row + v);
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
// warps fit on an SM and loads have to be in flight without them: each thread copies its own
// vectors of the next rows to its own slots of a ring in shared memory (cp.async; nobody else
// reads them, so no barrier) and reads them back, twice, when their row comes. Rows too wide
// for a stage of the ring (fp32 above H = 8192) are read from memory instead.
struct BwdRing {
    int32_t stages, arrays;               // stages 0: no ring
    int32_t i_r, i_dn, i_dr, i_y, i_gate; // place of each array in a stage, -1: absent
};

template <int DT, int V, int MAXT>
__global__ void __launch_bounds__(MAXT == 32 ? 128 : MAXT, MAXT == 32 || MAXT == 128 ? 4
                                                           : MAXT == 256              ? 2
                                                                                      : 1)
    residual_norm_bwd_kernel(NormArgs a, BwdRing g)
{
    constexpr bool ONEWARP = MAXT == 32;
    constexpr int W16 = DT == MOE_F32 ? 2 : 1;  // 16-byte words of a vector
    extern __shared__ uint4 ring[];
    __shared__ float red[2 * 32 * 3];
    int half = 0;
    pdl_wait();
    const int tid = threadIdx.x, step = blockDim.x;
    const int lin = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const int64_t rows = ONEWARP ? (int64_t)gridDim.x * blockDim.y : gridDim.x;
    const int64_t first = ONEWARP ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    const bool post = a.w_post != nullptr, next = a.w_next != nullptr, branch = a.y != nullptr;
    const bool drop = a.threshold != 0;
    float gn[V][8], gp[V][8], gg[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) gn[i][e] = gp[i][e] = gg[i][e] = 0.0f;
    Philox ph;
    if (drop) ph = philox_load(a.rng);

    auto slot = [&](int stage, int array, int i) {
        return ring + ((int64_t)(stage * g.arrays + array) * (V * W16) + i * W16) * threads + lin;
    };
    auto fetch = [&](int stage, int64_t t) {
        auto one = [&](int array, const void* p) {
            if (array < 0) return;
            const uint4* src = static_cast<const uint4*>(p) + t * a.nvec * W16;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + i * step;
                if (v < a.nvec) {
                    uint4* dst = slot(stage, array, i);
#pragma unroll
                    for (int h = 0; h < W16; ++h)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                         (uint32_t)__cvta_generic_to_shared(dst + h * threads)),
                                     "l"(src + v * W16 + h)
                                     : "memory");
                }
            }
        };
        if (t < a.T) {
            one(g.i_r, a.r);
            one(g.i_dn, a.dn);
            one(g.i_dr, a.dr);
            one(g.i_y, a.y);
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
    int stage = 0;
    auto get = [&](int array, const void* p, int64_t row, int i, float (&f)[8]) {
        Vec8<DT> q;
        if (g.stages > 0) {
            const uint4* src = slot(stage, array, i);
            uint4 w[W16];
#pragma unroll
            for (int h = 0; h < W16; ++h) w[h] = src[h * threads];
            q.load(w, 0);
        } else {
            q.load(p, row + tid + i * step);
        }
        q.get(f);
    };
    for (int s = 0; s < g.stages; ++s) fetch(s, first + s * rows);

    for (int64_t t = first; t < a.T; t += rows) {
        const int64_t row = t * a.nvec;
        if (g.stages > 0) row_ready();
        float s3[3] = {0.0f, 0.0f, 0.0f};  // r^2, w_next dn r, y^2
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (v < a.nvec) {
                if (next) {
                    float p[8], q[8], w[8];
                    get(g.i_r, a.r, row, i, p);
                    get(g.i_dn, a.dn, row, i, q);
                    load_param8<DT>(a.w_next, a.param_f32, v, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s3[0] = fmaf(p[e], p[e], s3[0]);
                        s3[1] = fmaf(q[e] * w[e], p[e], s3[1]);
                    }
                }
                if (post) {
                    float p[8];
                    get(g.i_y, a.y, row, i, p);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s3[2] = fmaf(p[e], p[e], s3[2]);
                }
            }
        }
        if (next || post) row_sum<3, ONEWARP>(s3, red, half);
        const float s = next ? inv_rms(s3[0], a) : 0.0f;
        const float mean_n = next ? s * s * (s3[1] * a.inv_h) : 0.0f;
        const float u = post ? inv_rms(s3[2], a) : 1.0f;
        const float tg = a.gate_mode == MOE_GATE_TOKEN ? load_param<DT>(a.gate, a.param_f32, t)
                                                       : 1.0f;
        const uint32_t rid = drop ? row_id(a, t) : 0u;
        float s2[2] = {0.0f, 0.0f};  // w_post c y, b z
        float c[V][8];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (v < a.nvec) {
                float d[8], q[8];
                if (a.dr != nullptr) {
                    get(g.i_dr, a.dr, row, i, d);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] = 0.0f;
                }
                if (next) {
                    float p[8], w[8];
                    get(g.i_r, a.r, row, i, p);
                    get(g.i_dn, a.dn, row, i, q);
                    load_param8<DT>(a.w_next, a.param_f32, v, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        d[e] += s * (q[e] * w[e] - p[e] * mean_n);
                        gn[i][e] = fmaf(q[e], p[e] * s, gn[i][e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = a.residual_scale * d[e];
                Vec8<DT> o;
                o.set(q);
                o.store(a.dx, row + v);
                if (branch) {
                    float y[8], w[8];
                    uint32_t bitsw[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
                    if (drop) philox8(ph, (uint32_t)v, rid, bitsw);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] *= a.branch_scale;
                    get(g.i_y, a.y, row, i, y);
                    if (post) load_param8<DT>(a.w_post, a.param_f32, v, w);
                    if (a.gate_mode != MOE_GATE_NONE) {
                        float z[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] = post ? y[e] * u * w[e] : y[e];
                        if (drop) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                z[e] = philox_keep(bitsw, e, a.threshold) ? z[e] * a.inv_keep : 0.0f;
                        }
                        if (a.gate_mode == MOE_GATE_FULL) {
                            get(g.i_gate, a.gate, row, i, q);
#pragma unroll
                            for (int e = 0; e < 8; ++e) z[e] *= d[e];
                            o.set(z);
                            o.store(a.dgate, row + v);
                        } else if (a.gate_mode == MOE_GATE_CHANNEL) {
                            load_param8<DT>(a.gate, a.param_f32, v, q);
#pragma unroll
                            for (int e = 0; e < 8; ++e) gg[i][e] = fmaf(d[e], z[e], gg[i][e]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                s2[1] = fmaf(d[e], z[e], s2[1]);
                                q[e] = tg;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e] *= q[e];
                    }
                    if (drop) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[e] = philox_keep(bitsw, e, a.threshold) ? d[e] * a.inv_keep : 0.0f;
                    }
                    if (post) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            gp[i][e] = fmaf(d[e], y[e] * u, gp[i][e]);
                            c[i][e] = d[e] * w[e];
                            s2[0] = fmaf(c[i][e], y[e], s2[0]);
                        }
                    } else {
                        o.set(d);
                        o.store(a.dy, row + v);
                    }
                }
            }
        }
        if (post || a.gate_mode == MOE_GATE_TOKEN) row_sum<2, ONEWARP>(s2, red, half);
        if (a.gate_mode == MOE_GATE_TOKEN && tid == 0) static_cast<float*>(a.dgate)[t] = s2[1];
        if (post) {
            const float mean_p = u * u * (s2[0] * a.inv_h);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = tid + i * step;
                if (v < a.nvec) {
                    float y[8];
                    get(g.i_y, a.y, row, i, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = u * (c[i][e] - y[e] * mean_p);
                    Vec8<DT> o;
                    o.set(y);
                    o.store(a.dy, row + v);
                }
            }
        }
        if (g.stages > 0) {
            fetch(stage, t + g.stages * rows);
            if (++stage == g.stages) stage = 0;
        }
    }

    // this row group's partial sums
    float* part = a.part + first * a.slots * (int64_t)a.H;
    auto put = [&](int where, const float (&f)[V][8]) {
        if (where < 0) return;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = tid + i * step;
            if (v < a.nvec) {
                float4* d = reinterpret_cast<float4*>(part + (int64_t)where * a.H) + 2 * v;
                d[0] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
                d[1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
            }
        }
    };
    put(a.slot_next, gn);
    put(a.slot_post, gp);
    put(a.slot_gate, gg);
}

// out[slot][column] = sum over the partial rows in order: a warp takes 32 columns of a slice of
// the rows, the slices of a block are added in order. Bound by the latency of a slice's loads,
// hence many short slices.
struct ReduceArgs {
    const float* part;
    int32_t parts, slots, H;
    float* out[3];
};

constexpr int kSlices = 32;

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
#pragma unroll 8
        for (int i = beg; i < end; ++i) s += p[i * stride];
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

// out = keep ? x / probability : 0, each thread kVec vectors of 8, a block's width apart
constexpr int kVec = 4;

template <int DT>
__global__ void __launch_bounds__(256) dropout_kernel(const void* x, void* out, int64_t T,
                                                      int32_t nvec, uint32_t threshold,
                                                      float inv_keep, const int64_t* rng,
                                                      uint32_t first_row, const int32_t* row_ids)
{
    pdl_wait();
    const Philox ph = philox_load(rng);
    const int64_t total = T * nvec;
    const int64_t base = (int64_t)blockIdx.x * (256 * kVec) + threadIdx.x;
    Vec8<DT> q[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (base + 256 * i < total) q[i].load(x, base + 256 * i);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int64_t g = base + 256 * i;
        if (g < total) {
            const int64_t t = total <= 0xffffffffll ? (int64_t)((uint32_t)g / (uint32_t)nvec)
                                                    : g / nvec;
            const uint32_t v = (uint32_t)(g - t * nvec);
            uint32_t w[4];
            philox8(ph, v, row_ids != nullptr ? (uint32_t)row_ids[t] : first_row + (uint32_t)t, w);
            float f[8];
            q[i].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = philox_keep(w, e, threshold) ? f[e] * inv_keep : 0.0f;
            q[i].set(f);
            q[i].store(out, g);
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

// the backward keeps 24 sums per vector in registers: one vector a thread up to H = 4096
RowShape bwd_shape(int nvec)
{
    if (nvec <= 32) return {true, 1, 32};
    if (nvec <= 512) return {false, 1, (nvec + 31) / 32 * 32};
    return {false, 2, ((nvec + 1) / 2 + 31) / 32 * 32};
}

// row groups of the backward: a function of (T, H) alone, so that the order of the parameter
// sums does not depend on the device (about 512 threads for each of a B200's 148 SMs, at least
// two rows a group)
int64_t bwd_groups(int64_t T, int32_t H)
{
    const RowShape s = bwd_shape(H / 8);
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

template <int DT>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st)
{
    const RowShape s = row_shape(a.nvec);
    if (s.one_warp) {
        const dim3 grid((unsigned)((a.T + kWarpRows - 1) / kWarpRows)), block(32, kWarpRows);
        return s.V == 1 ? launch_pdl(residual_norm_kernel<DT, 1, 32>, grid, block, 0, st, a)
                        : launch_pdl(residual_norm_kernel<DT, 2, 32>, grid, block, 0, st, a);
    }
    auto kernel = s.threads <= 256   ? residual_norm_kernel<DT, 2, 256>
                  : s.threads <= 512 ? residual_norm_kernel<DT, 2, 512>
                                     : residual_norm_kernel<DT, 2, 1024>;
    return launch_pdl(kernel, dim3((unsigned)a.T), dim3(s.threads), 0, st, a);
}

template <int DT, int V, int MAXT>
cudaError_t norm_bwd_variant(const NormArgs& a, BwdRing g, dim3 grid, dim3 block, cudaStream_t st)
{
    auto kernel = residual_norm_bwd_kernel<DT, V, MAXT>;
    const int threads = (int)(block.x * block.y);
    const int per_sm = threads <= 512 ? 512 / threads : 1;
    const size_t stage = (size_t)g.arrays * V * (DT == MOE_F32 ? 32 : 16) * threads;
    g.stages = (int32_t)(225000 / per_sm / (stage > 0 ? stage : 1));
    if (g.stages > 4) g.stages = 4;
    const size_t smem = g.stages * stage;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool attr_set[64] = {};
    if (!attr_set[dev]) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226000);
        if (err != cudaSuccess) return err;
        attr_set[dev] = true;
    }
    return launch_pdl(kernel, grid, block, smem, st, a, g);
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
    const RowShape s = bwd_shape(a.nvec);
    if (s.one_warp)
        return norm_bwd_variant<DT, 1, 32>(a, g, dim3((unsigned)(groups / kWarpRows)),
                                           dim3(32, kWarpRows), st);
    const dim3 grid((unsigned)groups), block(s.threads);
    if (s.V == 1) {
        if (s.threads <= 128) return norm_bwd_variant<DT, 1, 128>(a, g, grid, block, st);
        if (s.threads <= 256) return norm_bwd_variant<DT, 1, 256>(a, g, grid, block, st);
        return norm_bwd_variant<DT, 1, 512>(a, g, grid, block, st);
    }
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
    return (size_t)bwd_groups(c.T, c.H) * 3 * (size_t)c.H * sizeof(float);
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
    const int64_t groups = bwd_groups(c.T, c.H);
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
            return launch_pdl(dropout_kernel<MOE_BF16>, grid, dim3(256), 0, st, x, out, T, nvec,
                              th, inv, rng, fr, row_ids);
        case MOE_F16:
            return launch_pdl(dropout_kernel<MOE_F16>, grid, dim3(256), 0, st, x, out, T, nvec,
                              th, inv, rng, fr, row_ids);
        default:
            return launch_pdl(dropout_kernel<MOE_F32>, grid, dim3(256), 0, st, x, out, T, nvec,
                              th, inv, rng, fr, row_ids);
    }
}

}  // namespace moe
