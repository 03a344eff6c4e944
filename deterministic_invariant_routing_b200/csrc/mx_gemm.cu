// The expert products with both operands in the microscaled 4-bit format: rows of A grouped by
// expert, A and B as e2m1 codes under e8m0 scales (mx_format.cuh),
//
//   out[r, c] = sum over k of (A[r, k] 2^(sa[r, k / 32] - 127)) (B_g[c, k] 2^(sb[c, k / 32] - 127))
//
// on the tensor cores with tcgen05.mma kind::mxf4 (K = 64 an instruction, the scales applied
// by the tensor core, fp32 accumulation in TMEM). The structure is the bf16 pair kernel's: a
// cluster of two CTAs computes 256 rows by 256 columns, each CTA holding its 128 rows of A and
// half of B's columns, so that a k-block (256 columns of K: 128 bytes a row) takes 32 KiB a CTA
// for the 512 cycles its four instructions need. Where groups have few rows, single CTAs compute
// tiles of 128 rows by the same 256 columns instead (launch_mx_gemm has the rule).
//
// Scales: an instruction reads them from TMEM, 4 bytes (4 blocks of 32) per row in a 32-bit
// column for every 32 rows. Both operands keep them in tiles of 128 rows by 4 blocks (512 bytes,
// mx_tiled_scale), which TMA brings in beside the operands and tcgen05.cp (32x128b.warpx4) copies
// to 4 columns, issued in order before the instructions that read them. Each CTA needs the
// scales of its 128 rows and of all 256 columns. A tile of rows therefore starts on a multiple of
// 128 of the row index: an expert's first tile may begin with rows of the expert before it,
// which are computed and not stored. (Rows started at the expert's first row, with a warp
// reading row-major scales four k-blocks ahead and writing the tile itself, measured 2060
// cycles a k-block against 512: the fence between its writes and the copy waits for its reads.)
//
// TMEM: two accumulators of 256 columns and 24 columns of scales do not fit in 512, so the
// accumulators share 32 columns ([0, 256) and [224, 480)): a tile's epilogue reads those first
// and lets the next tile's instructions start after them.
//
// Arithmetic per row: k-blocks in increasing order, four K = 64 steps each (two in a last block
// of 128 columns), one accumulator; nothing depends on where the row sits, on its expert's
// other rows or on T. Rows outside the group are computed and never stored.
//
// Every wait is bounded (MOE_ST_PIPE_TIMEOUT); offsets outside [0, rows] or below the largest
// before them are clamped and counted in MOE_ST_BAD_ROWS, so no tile reaches past the buffers and
// no row is in two groups.
//
// Measured on B200 (kernel alone, 1.9 GHz): 65536 x 4096 x 4096 in one group 375-385 us = 5.7-5.9
// PFLOP/s (the same kernel issuing its instructions on stale operands: 315 us, 7.0); the 30B-A3B
// layer at 16384 tokens, 128 experts: gate_up 177 us (825 GFLOP; 133 us at that rate with the
// rounding up to tiles), down 142 us (412 GFLOP, 537 MB of output: 82 us of writing); 24594 rows
// over 256 experts of 2048 x 4096 (1.14 GB of weights, 174 us of reading) 222 us; 512 rows over 128
// experts of 2048 x 768 (107 MB, 16 us) 19.4 us. What is left is the gap between two tiles of a
// cluster, about 1000 cycles from the last instruction of one, through its epilogue's first reads,
// to the first of the next (the price of the shared columns), and for down the stores.
#include "mx_format.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr int XH = 128;                 // rows per CTA
constexpr int XN = 256;                 // columns per tile (SwiGLU: 128 gate, 128 up)
constexpr int XK = 256;                 // columns of K per stage
constexpr uint32_t kXA = XH * XK / 2;   // 16 KiB
constexpr uint32_t kXSA = 1024;         // scales of 128 rows, two tiles of 4 blocks
constexpr uint32_t kXSB = 2048;         // scales of 256 columns
constexpr uint32_t kXBox = 32 * XK / 2; // a 32-row box of A
constexpr int kXEpiWarps = 8;
constexpr int kXThreads = 32 * (2 + kXEpiWarps);
constexpr uint32_t kXCols = 512;        // TMEM columns
constexpr uint32_t kXAcc1 = 224;        // the second accumulator; the first is at 0
constexpr uint32_t kXTmemSA = 480, kXTmemSB = 488;
constexpr uint16_t kXPair = 0x3;

// Shared memory is split between operand stages and store tiles (32 rows x 64 columns of bf16 per
// epilogue warp). Quantised outputs need no store tiles.
template <bool PAIR, int S, int BUFS>
struct MxSmem {
    static constexpr int kRows = PAIR ? 2 * XH : XH;                // rows per tile
    static constexpr uint32_t kB = (PAIR ? 128u : 256u) * XK / 2;  // a CTA's columns of B
    static constexpr uint32_t kStage = kXA + kB + kXSA + kXSB;
    static constexpr uint32_t kEpi = (uint32_t)BUFS * kXEpiWarps * 4096u;
    static constexpr int kBars = 2 * S + 6;
    static size_t bytes(int groups)
    {
        return 1024 + (size_t)S * kStage + kEpi + kBars * 8 + 16 +
               ((size_t)2 * (groups + 1) + kXThreads / 32) * sizeof(int32_t);
    }
};

enum MxEpilogue { MX_BF16 = 0, MX_SWIGLU = 1, MX_SWIGLU_QUANT = 2 };

struct MxArgs {
    int k, k_blocks, n, n_tiles, groups;
    int64_t rows;
    const int32_t* offsets;  // [groups + 1], or NULL: one group of all rows
    int sb_tiles;            // 128-row scale tiles per group of B
    int half;                // SwiGLU: n, the first up row; 0 otherwise
    uint16_t* out;           // [rows, n] bf16
    uint8_t* out_codes;      // MX_SWIGLU_QUANT: [rows, n / 2], and scales in tiles
    uint8_t* out_scales;
    int32_t* status;
};

struct MxTile {
    int g, n;
    int64_t row0, row_beg, row_end;  // the tile's first row, the group's rows
};

// rows of a group that starts at `beg`, tiled from the multiple of 128 below it
__device__ __forceinline__ int mx_row_tiles(int beg, int end, int rows)
{
    return end > beg ? (end - (beg & ~127) + rows - 1) / rows : 0;
}

// which of CTA `rank`'s four 32-row boxes hold rows of the group
__device__ __forceinline__ uint32_t mx_boxes(const MxTile& t, uint32_t rank)
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t r = t.row0 + (int64_t)rank * XH + 32 * j;
        if (r < t.row_end && r + 32 > t.row_beg) m |= 1u << j;
    }
    return m;
}

// kind::mxf4 with e2m1 operands (format 1), e8m0 scales (bit 23), both K-major;
// the scale bytes of a 32-bit column that the instruction reads start at byte `id` (0 or 2)
constexpr uint32_t mx_idesc(int m, int n, uint32_t id)
{
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
           ((uint32_t)(m >> 4) << 24) | (id << 29);
}

template <bool PAIR>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                         uint32_t sa, uint32_t sb, uint32_t accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n\t}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n\t}\n" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// 512 bytes of shared memory (32 rows of 16; of both CTAs of a pair) to 4 TMEM columns, a
// multiple of 4, in all lane quarters
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc)
{
    if (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
}

// arrive on `bar` (of both CTAs of a pair) once the tcgen05 work issued so far has completed
template <bool PAIR>
__device__ __forceinline__ void mx_commit(uint32_t bar)
{
    if (PAIR) mma_commit_pair_mc(bar, kXPair);
    else mma_commit(bar);
}

// a TMA load whose bytes are counted on `bar`, the leader's of a pair
template <bool PAIR>
__device__ __forceinline__ void mx_load(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint32_t bar)
{
    if (PAIR) tma_load_2d_pair(dst, map, x, y, bar);
    else tma_load_2d(dst, map, x, y, bar);
}

// True in one lane of a converged warp. The loading and issuing roles run as whole warps whose
// loop state is the same in every lane, and only the instructions themselves are one lane's: the
// compiler then keeps descriptors and addresses in uniform registers, which is where tcgen05 and
// TMA instructions take them from. As loops of a single thread (`lane == 0`) every operand was
// moved there per instruction, and issuing a k-block took 1400 cycles instead of 512.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(p));
    return p != 0;
}

// bring a tensor map (a kernel parameter) into the cache that TMA reads it through
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// a value that every lane of the warp holds, known to be the same in all of them
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// descriptor of such a 512-byte tile: no swizzle, groups of 8 rows 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3fffu) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}

// 64 consecutive fp32 columns of this thread's TMEM lane, waited for as in tmem_ld32
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, "
        "%35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, "
        "%52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63},  "
        "[%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]),
          "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
          "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]),
          "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]),
          "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}

// silu(g) * u with the hardware's base-2 exponential and reciprocal (a few ulp of fp32, far below
// the bf16 rounding that follows): six instructions. The epilogue has 16384 of these per CTA and
// tile beside a main loop a quarter as long as the bf16 kernel's; with the IEEE reciprocal and
// the denormal-safe exponential it took about 11000 cycles a tile and bound the product.
// g -> -inf gives -0; an overflowed exponential gives a zero reciprocal.
__device__ __forceinline__ float swiglu_fast(float g, float u)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

// PAIR: a cluster of two CTAs a tile of 256 rows; else one CTA a tile of 128, with all of B's
// columns of the tile in its stages
template <int MODE, bool PAIR, int kXS, int BUFS>
__global__ void __launch_bounds__(kXThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                   const __grid_constant__ CUtensorMap tmA32,
                   const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA,
                   const __grid_constant__ CUtensorMap tmSB,
                   const __grid_constant__ CUtensorMap tmO, MxArgs args)
{
    constexpr bool kGlu = MODE != MX_BF16;
    using M = MxSmem<PAIR, kXS, BUFS>;
    constexpr uint32_t kXB = M::kB, kXStage = M::kStage;
    constexpr int XM = M::kRows, kCtas = PAIR ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_u32(smem_raw);
    uint8_t* base = smem_raw + ((1024u - (raw_s & 1023u)) & 1023u);
    const uint32_t sA0 = smem_u32(base);
    const uint32_t sB0 = sA0 + kXS * kXA;
    const uint32_t sSA0 = sB0 + kXS * kXB;
    const uint32_t sSB0 = sSA0 + kXS * kXSA;
    const uint32_t sE0 = sA0 + kXS * kXStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(base + kXS * kXStage + M::kEpi);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(kXS + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kXS + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (uint32_t)(2 * kXS + 2 + a); };
    const uint32_t tover = bar0 + 8u * (uint32_t)(2 * kXS + 4);  // the shared columns are read
    const uint32_t drain = tover + 8u;
    uint32_t* misc = reinterpret_cast<uint32_t*>(bars + M::kBars);  // [0] tmem, [1] abort
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    int32_t* prefix = reinterpret_cast<int32_t*>(misc + 4);  // [groups + 1] row tiles before g
    int32_t* offs = prefix + (args.groups + 1);              // [groups + 1]
    int32_t* totals = offs + (args.groups + 1);              // [warps] row tiles of a warp's groups

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int G = args.groups;
    const uint32_t rank = PAIR ? blockIdx.x & 1 : 0;  // clusters are pairs of consecutive blocks
    const bool leader = rank == 0;
    const int cluster = blockIdx.x / kCtas, nclusters = gridDim.x / kCtas;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kXS; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), kCtas * kXEpiWarps);  // a warp each
        }
        mbar_init(tover, kCtas * kXEpiWarps / 2);  // half of each CTA's epilogue warps
        mbar_init(drain, 1);
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0 && elect_one()) {
        prefetch_map(&tmA);
        prefetch_map(&tmA32);
        prefetch_map(&tmB);
        prefetch_map(&tmSA);
        prefetch_map(&tmSB);
        prefetch_map(&tmO);
    }
    if (warp == 1) {
        if (PAIR) tmem_alloc_pair(smem_u32(misc), kXCols);
        else tmem_alloc(smem_u32(misc), kXCols);
    }
    // (the barriers above are ready for the other CTA: fenced, and waited for below)
    if (PAIR) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    pdl_wait();
    // The groups' offsets, clamped, and the row tiles before each group: a group a thread, scanned
    // within a warp and then over the warps' totals. (Offsets by all threads and then four groups
    // a lane of one warp took 1600 cycles at 128 groups, of the 20 000 of a decode product.)
    int carry = 0, falling = 0;  // falling: some offset is below its predecessor
    for (int g0 = 0; g0 < G; g0 += kXThreads) {
        const int g = g0 + (int)threadIdx.x;
        int n = 0, falls = 0;
        if (g < G) {
            const int rows = (int)args.rows;
            const int raw0 = args.offsets != nullptr ? args.offsets[g] : 0;
            const int raw1 = args.offsets != nullptr ? args.offsets[g + 1] : rows;
            const int beg = min(max(raw0, 0), rows), end = min(max(raw1, 0), rows);
            n = mx_row_tiles(beg, end, XM);
            falls = end < beg;
            offs[g] = beg;
            if (g == G - 1) offs[G] = end;
            if (blockIdx.x == 0) {
                const int bad = (end < beg) + (raw1 != end) + (g == 0 && raw0 != beg);
                if (bad) status_add(args.status, MOE_ST_BAD_ROWS, bad);
            }
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (g0 != 0) __syncthreads();  // the totals of the 320 groups before are read
        if (lane == 31) totals[warp] = incl;
        falling |= __syncthreads_or(falls);
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kXThreads / 32; ++w) {
            const int v = totals[w];
            before += w < warp ? v : 0;
            all += v;
        }
        if (g < G) prefix[g] = carry + before + incl - n;
        carry += all;
    }
    if (falling) {
        // every offset is raised to the largest before it, so that no row is in two groups (two
        // tiles would store it in no order); counted above, and not in a hurry
        __syncthreads();
        if (threadIdx.x == 0) {
            int top = offs[0], tiles = 0;
            for (int g = 0; g < G; ++g) {
                const int end = max(offs[g + 1], top);
                offs[g] = top;
                prefix[g] = tiles;
                tiles += mx_row_tiles(top, end, XM);
                top = end;
            }
            offs[G] = top;
            totals[0] = tiles;
        }
        __syncthreads();
        carry = totals[0];
    }
    if (threadIdx.x == 0) prefix[G] = carry;
    tc_fence_before();
    __syncthreads();
    if (PAIR) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem_base = (uint32_t)uniform((int)misc[0]);
    const int total = uniform(carry * args.n_tiles);
    // a bounded wait of a whole warp: true when every lane's completed
    auto wait_warp = [&](uint32_t bar, uint32_t parity, bool honour_abort = true) -> bool {
        return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, args.status,
                                                    honour_abort));
    };
    auto aborted = [&]() -> bool { return __any_sync(0xffffffffu, *abort_flag != 0); };
    auto decode = [&](int t) -> MxTile {
        MxTile ti;
        const int mt = t / args.n_tiles;
        ti.n = t - mt * args.n_tiles;
        // the last group with prefix[g] <= mt (empty groups have no tile), the warp's 32 lanes
        // looking at as many places of [lo, lo + span) at a time
        int lo = 0;
        for (int span = G; span > 1;) {
            const int step = (span + 31) / 32;
            const int g = lo + lane * step;
            const uint32_t m = __ballot_sync(0xffffffffu, lane * step < span && prefix[g] <= mt);
            const int last = 31 - __clz(m);  // lane 0's place always qualifies
            span = min(step, span - last * step);
            lo += last * step;
        }
        ti.g = lo;
        ti.row_beg = offs[lo];
        ti.row0 = (ti.row_beg & ~(int64_t)127) + (int64_t)(mt - prefix[lo]) * XM;
        ti.row_end = offs[lo + 1];
        return ti;
    };

    if (warp == 0) {
        // -------------------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_phase = 0;
        const uint32_t fb0 =
            PAIR ? (uint32_t)uniform((int)mapa_shared(full_bar(0), 0)) : full_bar(0);
        const int kc = args.k / 128;  // scale tiles along K
        for (int t = cluster; t < total && !aborted(); t += nclusters) {
            const MxTile ti = decode(t);
            const int arow = uniform((int)ti.row0) + (int)rank * XH;
            const int b0 = uniform(ti.g) * args.sb_tiles + uniform(kGlu ? ti.n : 2 * ti.n);
            const int b1 = kGlu ? b0 + args.half / 128 : b0 + 1;  // 128-row tiles of B
            const int brow = (leader ? b0 : b1) * 128;
            // a whole tile's rows come in one box; of a partial one only the 32-row boxes with
            // rows of the group are read (decode-sized groups read few rows), the others come
            // from past the tensor's end, as zeros: 24594 rows over 256 experts, most of a
            // tile's rows padding, take 324 us in a loop at the power cap with zeros there and
            // 334 with whatever the stage held
            const uint32_t mine = (uint32_t)uniform((int)mx_boxes(ti, rank));
            const int past = (int)args.rows;
            const int sa = (arow >> 7) * kc, sb0 = b0 * kc, sb1 = b1 * kc;
            bool ok = true;
            for (int kb = 0; kb < args.k_blocks; ++kb) {
                if (!wait_warp(empty_bar(stage), phase ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = fb0 + 8u * (uint32_t)stage, ss = (uint32_t)stage;
                if (elect_one()) {
                    if (leader) mbar_expect_tx(full_bar(stage), kCtas * kXStage);
                    if (mine == 15u) {
                        mx_load<PAIR>(sA0 + ss * kXA, &tmA, kb * (XK / 2), arow, fb);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mx_load<PAIR>(sA0 + ss * kXA + j * kXBox, &tmA32, kb * (XK / 2),
                                          mine >> j & 1u ? arow + 32 * j : past, fb);
                    }
                    if (PAIR) {
                        mx_load<PAIR>(sB0 + ss * kXB, &tmB, kb * (XK / 2), brow, fb);
                    } else {
                        mx_load<PAIR>(sB0 + ss * kXB, &tmB, kb * (XK / 2), b0 * 128, fb);
                        mx_load<PAIR>(sB0 + ss * kXB + kXB / 2, &tmB, kb * (XK / 2), b1 * 128, fb);
                    }
                    mx_load<PAIR>(sSA0 + ss * kXSA, &tmSA, 0, sa + 2 * kb, fb);
                    mx_load<PAIR>(sSB0 + ss * kXSB, &tmSB, 0, sb0 + 2 * kb, fb);
                    mx_load<PAIR>(sSB0 + ss * kXSB + 1024u, &tmSB, 0, sb1 + 2 * kb, fb);
                }
                __syncwarp();
                armed |= 1u << stage;
                armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == kXS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
        }
        pdl_trigger();
        if (aborted() && leader) {
            for (int s = 0; s < kXS; ++s)
                if (armed & (1u << s)) wait_warp(full_bar(s), (armed_phase >> s) & 1u, false);
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------------------------------------------------- MMA issuer
            const uint64_t ad0 = sw128_desc(sA0), bd0 = sw128_desc(sB0);
            const uint64_t sad0 = scale_desc(sSA0), sbd0 = scale_desc(sSB0);
            const uint32_t tsa = tmem_base + kXTmemSA, tsb = tmem_base + kXTmemSB;
            int stage = 0;
            uint32_t phase = 0;
            int i = 0;
            for (int t = cluster; t < total && !aborted(); t += nclusters, ++i) {
                const int acc = i & 1;
                const uint32_t d = tmem_base + (acc ? kXAcc1 : 0u);
                bool ok = true;
                for (int kb = 0; kb < args.k_blocks; ++kb) {
                    if (!wait_warp(full_bar(stage), phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t st = (uint64_t)(uint32_t)stage;
                    const uint64_t ad = ad0 + st * (kXA >> 4), bd = bd0 + st * (kXB >> 4);
                    const uint64_t sad = sad0 + st * (kXSA >> 4), sbd = sbd0 + st * (kXSB >> 4);
                    const bool both = args.k - kb * XK >= XK;  // two chunks of 128 columns
                    const bool issuer = elect_one();
                    if (issuer) {
                        auto copy = [&](uint32_t c) {
                            tmem_cp_scales<PAIR>(tsa + 4u * c, sad + (uint64_t)(c * (512 >> 4)));
                            tmem_cp_scales<PAIR>(tsb + 8u * c, sbd + (uint64_t)(c * (512 >> 4)));
                            tmem_cp_scales<PAIR>(tsb + 8u * c + 4u,
                                                 sbd + (uint64_t)((1024 + c * 512) >> 4));
                        };
                        copy(0);
                        if (both) copy(1);
                    }
                    __syncwarp();
                    // a tile's first scales are copied while its accumulator is being read
                    if (kb == 0) {
                        ok = wait_warp(tempty_bar(acc), (((uint32_t)i >> 1) & 1u) ^ 1u) &&
                             (i == 0 || wait_warp(tover, ((uint32_t)i - 1u) & 1u));
                        if (!ok) break;
                        tc_fence_after();
                    }
                    if (issuer) {
                        auto mma = [&](uint32_t c, uint32_t accumulate) {
                            mma_mxf4<PAIR>(d, ad + 4u * c, bd + 4u * c, mx_idesc(XM, XN, 0),
                                           tsa + 4u * c, tsb + 8u * c, accumulate);
                            mma_mxf4<PAIR>(d, ad + 4u * c + 2u, bd + 4u * c + 2u,
                                           mx_idesc(XM, XN, 2), tsa + 4u * c, tsb + 8u * c, 1u);
                        };
                        mma(0, kb != 0 ? 1u : 0u);
                        if (both) mma(1, 1u);
                        mx_commit<PAIR>(empty_bar(stage));
                        if (kb == args.k_blocks - 1) mx_commit<PAIR>(tfull_bar(acc));
                    }
                    __syncwarp();
                    if (++stage == kXS) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
            }
            if (elect_one()) {
                if (PAIR) mma_commit_pair(drain);
                else mma_commit(drain);
            }
            __syncwarp();
            wait_warp(drain, 0u, false);
        }
    } else {
        // -------------------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lanes 32 q .. 32 q + 31
        const int row = q * 32 + lane;
        const int half = (warp - 2) >> 2;  // two warps a lane quarter: the first and last chunks
        const uint32_t tempty_leader0 = PAIR ? mapa_shared(tempty_bar(0), 0) : tempty_bar(0);
        const uint32_t tempty_leader1 = PAIR ? mapa_shared(tempty_bar(1), 0) : tempty_bar(1);
        const uint32_t tover_leader = PAIR ? mapa_shared(tover, 0) : tover;
        auto arrive = [](uint32_t bar) {
            if (PAIR) mbar_arrive_cluster(bar);
            else mbar_arrive(bar);
        };
        // Output: 32 rows x 64 columns of bf16 (128 bytes a row, 128-byte swizzle) through shared
        // memory and one TMA store where all 32 rows belong to the group, else row by row.
        const uint32_t ebuf0 = sE0 + (uint32_t)(warp - 2) * (BUFS * 4096u);
        const uint32_t eswz = (uint32_t)lane & 7u;
        uint32_t ebuf = ebuf0;
        auto tile_free = [&]() {  // the store that used this tile last has read it
            if (lane == 0) bulk_wait_read<(BUFS > 1 ? BUFS - 1 : 0)>();
            __syncwarp();
        };
        // 32 packed columns to the lower (0) or upper (1) half of this lane's row
        auto put32 = [&](const uint32_t* pk, int upper) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 ebuf + (uint32_t)lane * 128u +
                                 (((uint32_t)(4 * upper + v) ^ eswz) << 4)),
                             "r"(pk[4 * v]), "r"(pk[4 * v + 1]), "r"(pk[4 * v + 2]),
                             "r"(pk[4 * v + 3])
                             : "memory");
        };
        auto put_row = [&](const uint32_t* pk, uint16_t* dst_row) {
            uint4* dst = reinterpret_cast<uint4*>(dst_row);
#pragma unroll
            for (int v = 0; v < 4; ++v)
                dst[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
        };
        auto store_tile = [&](int row_blk, int col) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&tmO, ebuf, col, row_blk);
                bulk_commit();
            }
            if (BUFS > 1) ebuf = ebuf == ebuf0 ? ebuf0 + 4096u : ebuf0;
        };
        int i = 0;
        for (int t = cluster; t < total && !aborted(); t += nclusters, ++i) {
            const MxTile ti = decode(t);
            const int acc = i & 1;
            if (!wait_warp(tfull_bar(acc), ((uint32_t)i >> 1) & 1u)) break;
            tc_fence_after();
            const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (acc ? kXAcc1 : 0u);
            // the shared columns are the first accumulator's last chunk and the second's first:
            // each half starts at its outer end, and the half that meets them says so
            const bool over = half == (acc ? 0 : 1);
            auto release_shared = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(tover_leader);
            };
            const int64_t grow = ti.row0 + (int64_t)rank * XH + row;
            const bool valid = grow >= ti.row_beg && grow < ti.row_end;
            const int row_blk = (int)(ti.row0 + (int64_t)rank * XH + q * 32);
            // (without store tiles every row goes by itself)
            const bool full_blk =
                BUFS > 0 && row_blk >= ti.row_beg && (int64_t)row_blk + 31 < ti.row_end;
            if (!__any_sync(0xffffffffu, valid)) {
                // no row of the group: decode-sized groups leave the exponentials of one quarter
                if (over) release_shared();
            } else if (kGlu) {
                // this warp's 64 columns of h, 32 at a time
                const int col = ti.n * (XN / 2) + 64 * half;
                uint32_t codes[8], scales = 0;
                if (MODE == MX_SWIGLU && full_blk) tile_free();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int up = k ^ half;  // half 1 starts with its upper 32 columns
                    const uint32_t c = (uint32_t)(64 * half + 32 * up);
                    uint32_t g[32], u[32];
                    if (half) {  // the shared columns first: ups in this half, gates in the other
                        tmem_ld32(tbase + (uint32_t)(XN / 2) + c, u);
                        if (k == 0 && over) release_shared();
                        tmem_ld32(tbase + c, g);
                    } else {
                        tmem_ld32(tbase + c, g);
                        if (k == 0 && over) release_shared();
                        tmem_ld32(tbase + (uint32_t)(XN / 2) + c, u);
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        pk[j] = bf16x2_rne(swiglu_fast(__uint_as_float(g[2 * j]),
                                                       __uint_as_float(u[2 * j])),
                                           swiglu_fast(__uint_as_float(g[2 * j + 1]),
                                                       __uint_as_float(u[2 * j + 1])));
                    if (MODE == MX_SWIGLU) {
                        if (full_blk) put32(pk, up);
                        else if (valid) put_row(pk, args.out + grow * args.n + col + 32 * up);
                    } else {
                        // 32 columns of a row are one block: quantised from the bf16 values, so
                        // the fused product gives the codes of the two calls it replaces
                        uint32_t m = 0;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            m = max(m, max(pk[j] << 16 & 0x7fffffffu, pk[j] & 0x7fff0000u));
                        const uint32_t s = mx_scale_byte(m);
                        scales |= s << (8 * up);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                f[2 * e] = __uint_as_float(pk[4 * v + e] << 16);
                                f[2 * e + 1] = __uint_as_float(pk[4 * v + e] & 0xffff0000u);
                            }
                            const uint32_t w = mx_encode8(f, s);
                            if (up) codes[4 + v] = w;
                            else codes[v] = w;
                        }
                    }
                }
                if (MODE == MX_SWIGLU) {
                    if (full_blk) store_tile(row_blk, col);
                } else if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(args.out_codes + grow * (args.n / 2) +
                                                          col / 2);
                    dst[0] = make_uint4(codes[0], codes[1], codes[2], codes[3]);
                    dst[1] = make_uint4(codes[4], codes[5], codes[6], codes[7]);
                    *reinterpret_cast<uint16_t*>(
                        args.out_scales + mx_tiled_scale(grow, col / 32, args.n / 32)) =
                        (uint16_t)scales;
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    // each half from its outer end, where the shared columns are
                    const int c = half ? 192 - 64 * k : 64 * k;
                    const int col = ti.n * XN + c;
                    uint32_t r[64];
                    tmem_ld64(tbase + (uint32_t)c, r);
                    if (k == 0 && over) release_shared();
                    if (col >= args.n) continue;  // past the last column (n a multiple of 128)
                    uint32_t pk[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        pk[j] = bf16x2_rne(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                    if (full_blk) {
                        tile_free();
                        put32(pk, 0);
                        put32(pk + 16, 1);
                        store_tile(row_blk, col);
                    } else if (valid) {
                        put_row(pk, args.out + grow * args.n + col);
                        put_row(pk + 16, args.out + grow * args.n + col + 32);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive(acc ? tempty_leader1 : tempty_leader0);
        }
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    if (PAIR) cluster_sync();  // (with a release and an acquire: about 900 cycles)
    else __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, kXCols);
        else tmem_dealloc(tmem_base, kXCols);
    }
}

// codes [rows, k / 2] bytes: boxes of 128 bytes by box_rows rows, 128-byte swizzle
bool make_codes_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t k, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)(k / 2), (cuuint64_t)(rows > 0 ? rows : 1)};
    cuuint64_t strides[1] = {(cuuint64_t)(k / 2)};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// scale tiles of 512 bytes, two (256 columns of K) a box
bool make_scale_map(CUtensorMap* m, const void* ptr, int64_t tiles)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {256, (cuuint64_t)tiles};
    cuuint64_t strides[1] = {512};
    cuuint32_t box[2] = {256, 2};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [rows, n] as store tiles of 32 rows by 64 columns, 128-byte swizzle
bool make_out_map(CUtensorMap* m, void* ptr, int64_t rows, int64_t n)
{
    EncodeTiledFn fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)n, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)n * 2};
    cuuint32_t box[2] = {64, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int column_tiles(const MxProblem& p)
{
    return p.swiglu ? p.n / (XN / 2) : (p.n + XN - 1) / XN;
}

// tiles at most: two partial row tiles per group that has rows, and the full ones
int64_t most_tiles(const MxProblem& p, int rows)
{
    const int64_t partial = p.rows < p.groups ? p.rows : p.groups;
    return (p.rows / rows + 2 * partial) * column_tiles(p);
}

template <int MODE, bool PAIR, int S, int BUFS>
cudaError_t launch_mode(const MxProblem& p, cudaStream_t st)
{
    auto kernel = mx_gemm_kernel<MODE, PAIR, S, BUFS>;
    using M = MxSmem<PAIR, S, BUFS>;
    constexpr int kCtas = PAIR ? 2 : 1;
    const size_t smem = M::bytes(p.groups);
    if (smem > 232448) return cudaErrorInvalidValue;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool attr_set[64] = {};
    if (!attr_set[dev]) {
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
        if (err != cudaSuccess) return err;
        attr_set[dev] = true;
    }
    const bool glu = MODE != MX_BF16;
    const int b_rows = glu ? 2 * p.n : p.n;
    // (encoding a map takes half a microsecond of the call; those that this many rows cannot
    // use are stand-ins: a row in each of four 32-row boxes takes 66 rows, a store tile 32)
    CUtensorMap ma, ma32, mb, msa, ms, mo;
    if (!make_codes_map(&ma32, p.a, p.rows, p.k, 32)) return cudaErrorInvalidValue;
    if (!make_codes_map(&mb, p.b, (int64_t)p.groups * b_rows, p.k, XH)) return cudaErrorInvalidValue;
    if (!make_scale_map(&msa, p.a_scales, (p.rows + 127) / 128 * (p.k / 128)))
        return cudaErrorInvalidValue;
    if (!make_scale_map(&ms, p.b_scales, (int64_t)p.groups * (b_rows / 128) * (p.k / 128)))
        return cudaErrorInvalidValue;
    ma = ma32;
    if (p.rows >= 66 && !make_codes_map(&ma, p.a, p.rows, p.k, XH)) return cudaErrorInvalidValue;
    mo = ma32;  // without store tiles outputs are stored from registers
    if (BUFS > 0 && p.rows >= 32 && !make_out_map(&mo, p.out, p.rows, p.n))
        return cudaErrorInvalidValue;
    MxArgs a{};
    a.k = p.k;
    a.k_blocks = (p.k + XK - 1) / XK;
    a.n = p.n;
    a.n_tiles = column_tiles(p);
    a.groups = p.groups;
    a.rows = p.rows;
    a.offsets = p.offsets;
    a.sb_tiles = b_rows / 128;
    a.half = glu ? p.n : 0;
    a.out = p.out;
    a.out_codes = p.out_codes;
    a.out_scales = p.out_scales;
    a.status = p.status;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(148, 1, 1);
    cfg.blockDim = dim3(kXThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    static int max_clusters[64] = {};
    if (max_clusters[dev] == 0) {  // co-resident clusters (one CTA an SM at any group count)
        cfg.numAttrs = 1;          // the cluster shape only
        int n = 0;
        err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (err != cudaSuccess) return err;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        max_clusters[dev] = n;
    }
    int64_t clusters = most_tiles(p, M::kRows);
    if (clusters > max_clusters[dev]) clusters = max_clusters[dev];
    cfg.gridDim = dim3((unsigned)(kCtas * clusters), 1, 1);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, ma, ma32, mb, msa, ms, mo, a);
}

}  // namespace

cudaError_t launch_mx_gemm(const MxProblem& p, cudaStream_t st)
{
    if (p.k % 128 != 0 || p.n % 128 != 0) return cudaErrorInvalidValue;
    // At few rows a group most of a pair's 256 rows are padding, and one CTA a tile has twice as
    // many tiles in flight, each done in half the instructions. Measured, pairs against single
    // CTAs, in us: 512 rows over 128 experts, 2048 x 768, 27.3 against 21.0; 64 over 64, 1536 x
    // 2048 with SwiGLU, 22.7 / 16.7; 8192 over 256, 2048 x 4096 with SwiGLU, 221 / 198; at 64 rows
    // a group 37.0 / 37.3 and 51.3 / 48.8; at 128 42.7 / 51.4 and 59.1 / 61.9. Both give the same
    // bits: the row tile of an instruction is no part of a row's arithmetic.
    if (p.rows <= 64 * (int64_t)p.groups) {
        if (!p.swiglu) return launch_mode<MX_BF16, false, 4, 0>(p, st);
        return p.out_codes != nullptr ? launch_mode<MX_SWIGLU_QUANT, false, 4, 0>(p, st)
                                      : launch_mode<MX_SWIGLU, false, 4, 0>(p, st);
    }
    // (four stages and two store tiles a warp instead of five and one measured within 2 % either
    // way for plain products of K = 256 .. 4096)
    if (!p.swiglu) return launch_mode<MX_BF16, true, 5, 1>(p, st);
    return p.out_codes != nullptr ? launch_mode<MX_SWIGLU_QUANT, true, 6, 0>(p, st)
                                  : launch_mode<MX_SWIGLU, true, 5, 1>(p, st);
}

}  // namespace moe
