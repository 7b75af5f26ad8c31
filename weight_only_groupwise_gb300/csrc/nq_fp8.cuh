// nq_fp8.cuh -- products of e4m3 codes with a scale for each block of 128 along K (and along N for weights), on the
// fifth-generation tensor cores:
//
//   Y[i, n] = sum_b sx[i, b] sw[n / 128, b] sum_{k in block b} cx[i, k] cw[n, k]
//
// for groups of rows, each with its expert's weight (a dense product is one group). The inner sums are
// tcgen05.mma.kind::f8f6f4 into a fresh accumulator in TMEM for each block of K (products of codes are exact, the sums
// fp32); the epilogue warps load it and add it, times its scales, to fp32 sums in registers: the scales are any
// fp32 numbers, which the tensor cores' own block scales (powers of two) cannot hold.
//
// Two kernels share this file's tiles, rings and roles:
//   * fp8_rows_kernel, for many rows a group: rows of x are the MMA's M. A thread of the epilogue has a row, so that
//     its scale is one register for 128 columns.
//   * fp8_cols_kernel, for few rows a group: weights are the MMA's M, rows of x its N = 16..128, and what is
//     read of x, computed and loaded from TMEM shrinks with them: bound by the weights' bytes.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_fp8.h"
#include "nq_step.h"
#include "nq_tc.cuh"

namespace nq {

constexpr int kF8Epilogue = 8;                   // epilogue warps: 0..7, quarter = warp % 4, half = warp / 4
constexpr int kF8Producer = 8, kF8Mma = 9, kF8Scales = 10;
constexpr int kF8Threads = 12 * 32;              // (warp 11 only gives its registers away)
// Registers a thread: a block begins with 168; warps 8..11 hand theirs to the epilogue's 128 sums and 64 loads:
// 256 x 216 + 128 x 72 = 384 x 168.
constexpr int kF8EpilogueRegs = 216, kF8OtherRegs = 72;
static_assert(256 * kF8EpilogueRegs + 128 * kF8OtherRegs == kF8Threads * 168, "registers of a block");
constexpr int kF8MaxStages = 16;
constexpr int kF8Row = 128;                      // bytes (codes) of a stage's row: one block of K, one swizzled row
constexpr int kF8Tile = 128;                     // rows of a block's MMA operand A

// What both kernels read of the call.
struct Fp8Call {
    const float* xs;
    const int* rows;                             // NULL: row i of x
    const int* offsets;                          // NULL: one group of M rows
    const float* ws[2];                          // gate (or the only one), up
    long long xs_stride, ws_row[2], ws_expert[2];
    uint8_t* y;
    float* ys;
    long long y_stride, ys_stride;               // elements
    int x_rows, E, M, K, N;
    int x_past;                                  // a row number outside xmap
    int dtype;
    bool wide;                                   // results' rows aligned to 32 bytes
    bool quads;                                  // rows of xs aligned to 16 bytes
    int* err;                                    // the error word of bounded waits
    unsigned long long wait_ns;
};

struct alignas(64) Fp8Args {
    CUtensorMap xmap;                            // {K, rows of x}: boxes of 128 codes x rows, or x 1 for gathers
    CUtensorMap wmap[2];                         // {K, N, E}
    Fp8Call c;
};

// ---------------------------------------------------------------- instructions

template <int n>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void regs_fewer() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}

__device__ __forceinline__ void f8_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate, bool issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"((uint32_t)issue)
        : "memory");
}

// Instruction descriptor: D fp32, A and B e4m3, both K-major.
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Four rows of a 2-D map (box one row high) by their numbers; one outside the tensor reads as zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int c0, const int (&r)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}

#define NQ_O4(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3])
// n consecutive columns (8, 16 or 32) of the thread's TMEM lane.
template <int n>
__device__ __forceinline__ void f8_ld(uint32_t taddr, uint32_t* v) {
    static_assert(n == 8 || n == 16 || n == 32, "columns of a load");
    if constexpr (n == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : NQ_O4(v, 0), NQ_O4(v, 4)
                     : "r"(taddr)
                     : "memory");
    else if constexpr (n == 16)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : NQ_O4(v, 0), NQ_O4(v, 4), NQ_O4(v, 8), NQ_O4(v, 12)
                     : "r"(taddr)
                     : "memory");
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
            "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : NQ_O4(v, 0), NQ_O4(v, 4), NQ_O4(v, 8), NQ_O4(v, 12), NQ_O4(v, 16), NQ_O4(v, 20), NQ_O4(v, 24), NQ_O4(v, 28)
            : "r"(taddr)
            : "memory");
}
#undef NQ_O4
// Waits for the loads; names their registers, so that nothing that uses them is moved ahead of it.
#define NQ_I4(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3])
template <int n>
__device__ __forceinline__ void f8_wait_ld(uint32_t* v) {
    if constexpr (n == 8)
        asm volatile("tcgen05.wait::ld.sync.aligned;" : NQ_I4(v, 0), NQ_I4(v, 4)::"memory");
    else if constexpr (n == 16)
        asm volatile("tcgen05.wait::ld.sync.aligned;" : NQ_I4(v, 0), NQ_I4(v, 4), NQ_I4(v, 8), NQ_I4(v, 12)::"memory");
    else
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : NQ_I4(v, 0), NQ_I4(v, 4), NQ_I4(v, 8), NQ_I4(v, 12), NQ_I4(v, 16), NQ_I4(v, 20), NQ_I4(v, 24), NQ_I4(v, 28)::"memory");
}
#undef NQ_I4

__device__ __forceinline__ uint64_t f2_pack(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float2 f2_unpack(uint64_t v) {
    uint32_t lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
// acc += v * s, two fp32 numbers at once (sm_100 on; each rounded as a single fma).
__device__ __forceinline__ void f2_fma(uint64_t& acc, uint64_t v, uint64_t s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}

__device__ __forceinline__ uint32_t pack_16(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void store_32(void* p, const uint32_t (&u)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// Larger of two magnitudes by their bits: NaN is the largest of all.
__device__ __forceinline__ uint32_t bits_max(uint32_t m, float v) { return max(m, __float_as_uint(v) & 0x7FFFFFFFu); }

// ---------------------------------------------------------------- tiles

// Groups of rows and the tiles before each, in shared memory. A tile is `high` rows (at most) of a group by a
// column tile; a group's tiles run over its rows first, in bands of kF8Band, so that blocks that run together share
// both operands in L2.
constexpr int kF8Band = 16;

struct Fp8Groups {
    int* before;                                 // [E + 1] tiles before a group
    int* start;                                  // [E] its rows
    int* end;
};
constexpr int f8_group_bytes(int E) { return (3 * E + 1) * 4; }

struct Fp8Tile {
    int e, row0, rows, col;                      // expert, first row, rows of the tile, column tile
};

// All threads of a block: `sums` has room for a number of each warp. Returns the call's tiles.
__device__ __forceinline__ int fp8_groups(const Fp8Call& c, const Fp8Groups& g, int high, int cols, int* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    int total = 0;
    for (int e0 = 0; e0 < c.E; e0 += threads) {
        const int e = e0 + tid;
        int r0 = 0, r1 = 0;
        if (e < c.E) {
            r0 = c.offsets ? min(max(__ldg(c.offsets + e), 0), c.M) : 0;
            r1 = c.offsets ? max(min(__ldg(c.offsets + e + 1), c.M), r0) : c.M;
        }
        const int mine = (r1 - r0 + high - 1) / high * cols;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += u;
        }
        __syncthreads();                         // the sums of the round before have been read
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int base = total;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) base += sums[w];
            total += sums[w];
        }
        if (e < c.E) {
            g.before[e] = base + upto - mine;
            g.start[e] = r0;
            g.end[e] = r1;
        }
    }
    if (tid == 0) g.before[c.E] = total;
    return total;
}

// Tile number t, at group e or behind. even: a group's rows are shared out evenly over its tiles, in multiples of 16;
// else all but the last tile have `high` rows.
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Call& c, const Fp8Groups& g, int t, int from, int high, int cols, bool even) {
    int lo = from, hi = c.E - 1;                 // the last group with before <= t and tiles
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.before[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    Fp8Tile o;
    o.e = lo;
    const int r0 = g.start[lo], r1 = g.end[lo], n = (r1 - r0 + high - 1) / high;
    int i = t - g.before[lo];
    const int band = i / (kF8Band * cols), in_band = min(kF8Band, n - band * kF8Band);
    i -= band * kF8Band * cols;
    o.col = i / in_band;
    const int r = band * kF8Band + i - o.col * in_band;
    const int each = even ? ((r1 - r0 + n - 1) / n + 15) / 16 * 16 : high;
    o.row0 = r0 + r * each;
    o.rows = min(each, r1 - o.row0);             // (at least one: each <= high, and (n - 1) high < r1 - r0)
    return o;
}

// A producer lane's four rows of x, and how many lanes have rows of the tile (0: x is not gathered). A row that x has
// not is past the last, which reads as zeros; the last lane's rows behind the tile's repeat one that is there (a
// gather of rows outside takes several times as long: 128 rows of which one is in the tile, 2.9 us a block of K).
__device__ __forceinline__ int f8_gather_rows(const Fp8Call& c, const Fp8Tile& tile, int (&at)[4]) {
    if (!c.rows) return 0;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = __ldg(c.rows + tile.row0 + min(4 * lane + i, tile.rows - 1));
        at[i] = s >= 0 && s < c.x_rows ? s : c.x_past;
    }
    return (tile.rows + 3) / 4;
}

// ---------------------------------------------------------------- many rows a group

template <bool GLU>
struct Fp8RowsGeo {
    static constexpr int kCols = 256;            // of D: a tile's columns, or 128 of gate and 128 of up
    static constexpr int kOut = GLU ? 128 : 256; // columns of the result
    static constexpr int kStageBytes = (kF8Tile + kCols) * kF8Row;
    static constexpr int kStages = 4;
    static constexpr int kTurnBytes = GLU ? kF8Epilogue * 32 * 34 * 2 : kF8Epilogue * 32 * 34 * 2;  // a warp's 32 x 32 results
    static constexpr int kCtrlBytes = 512 + 1024 + kTurnBytes;
    static int smem(int E) { return 1024 + kStages * kStageBytes + kCtrlBytes + f8_group_bytes(E); }
};

template <bool GLU>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_rows_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8RowsGeo<GLU>;
    constexpr int kStages = Geo::kStages;
    const Fp8Call& c = a.c;
    extern __shared__ uint8_t f8_smem[];
    uint8_t* const ring = f8_smem + ((1024u - (smem_u32(f8_smem) & 1023u)) & 1023u);
    uint8_t* const ctrl = ring + kStages * Geo::kStageBytes;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
    // bars: full[16], empty[16], tfull[2], tempty[2], done
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kF8MaxStages, tfull0 = empty0 + 8 * kF8MaxStages;
    const uint32_t tempty0 = tfull0 + 16, done = tempty0 + 16;
    volatile int* const flags = reinterpret_cast<volatile int*>(ctrl + 320);     // [0] abort, [3] TMEM base
    int* const sums = reinterpret_cast<int*>(ctrl + 384);
    uint32_t* const largest = reinterpret_cast<uint32_t*>(ctrl + 512);           // [2 halves][128 rows]
    uint16_t* const turn = reinterpret_cast<uint16_t*>(ctrl + 512 + 1024);
    Fp8Groups groups;
    groups.before = reinterpret_cast<int*>(ctrl + Geo::kCtrlBytes);
    groups.start = groups.before + c.E + 1;
    groups.end = groups.start + c.E;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t wait_ns = c.wait_ns;
    int* const err = c.err;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, kF8Epilogue);
        }
        mbar_init(done, 1);
        flags[0] = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(const_cast<int*>(flags) + 3), 512);
    grid_launch_dependents();
    grid_dependency_wait();
    const int cols = (c.N + Geo::kOut - 1) / Geo::kOut, KB = (c.K + kFp8Block - 1) / kFp8Block;
    const int total = fp8_groups(c, groups, kF8Tile, cols, sums);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];

    // (each branch begins with its own count: where the paths met again, everything would have to fit the smaller)
    if (warp >= kF8Epilogue) {
        regs_fewer<kF8OtherRegs>();
    if (warp == kF8Producer) {
        // ------------------------------------------------------------ copies
        int seq = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, kF8Tile, cols, false);
            e = tile.e;
            int at[4];
            const int fours = f8_gather_rows(c, tile, at);
            for (int kb = 0; kb < KB && ok; ++kb, ++seq) {
                const int st = seq % kStages;
                if (seq >= kStages) ok = mbar_wait(empty0 + 8 * st, ((seq / kStages) - 1) & 1, flags, err, wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t xa = smem_u32(ring + st * Geo::kStageBytes), wa = xa + kF8Tile * kF8Row, bar = full0 + 8 * st;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)(Geo::kCols * kF8Row + (c.rows ? fours * 4 : kF8Tile) * kF8Row));
                    if (GLU) {
                        tma_load_3d(wa, &a.wmap[0], kb * kFp8Block, tile.col * 128, tile.e, bar);
                        tma_load_3d(wa + 128 * kF8Row, &a.wmap[1], kb * kFp8Block, tile.col * 128, tile.e, bar);
                    } else {
                        tma_load_3d(wa, &a.wmap[0], kb * kFp8Block, tile.col * 256, tile.e, bar);
                    }
                    if (!c.rows) tma_load_2d(xa, &a.xmap, kb * kFp8Block, tile.row0, bar);
                }
                __syncwarp();
                if (lane < fours) tma_gather4(xa + 4 * lane * kF8Row, &a.xmap, kb * kFp8Block, at, bar);
            }
        }
        if (!ok)
            for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)
                mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
    } else if (warp == kF8Mma) {
        // ------------------------------------------------------------ MMA issuer
        const bool leader = elect_one();
        int seq = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, kF8Tile, cols, false);
            e = tile.e;
            const int n = GLU ? Geo::kCols : min(Geo::kCols, (c.N - tile.col * Geo::kOut + 15) / 16 * 16);
            const uint32_t idesc = f8_idesc(kF8Tile, n);
            for (int kb = 0; kb < KB && ok; ++kb, ++seq) {
                const int st = seq % kStages, buf = seq & 1;
                ok = mbar_wait(full0 + 8 * st, (seq / kStages) & 1, flags, err, wait_ns);
                if (seq >= 2) ok = ok && mbar_wait(tempty0 + 8 * buf, ((seq >> 1) - 1) & 1, flags, err, wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t xa = smem_u32(ring + st * Geo::kStageBytes), wa = xa + kF8Tile * kF8Row;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    f8_mma(tmem + 256 * buf, smem_desc_sw128(xa + 32 * j), smem_desc_sw128(wa + 32 * j), idesc, j > 0 ? 1u : 0u, leader);
                tc_commit(empty0 + 8 * st, leader);
                tc_commit(tfull0 + 8 * buf, leader);
            }
        }
        tc_commit(done, leader);                 // every MMA has completed before TMEM can be freed
        mbar_wait_drain(done, 0, kDrainNs);
    }
    } else {
        // ------------------------------------------------------------ epilogue
        regs_more<kF8EpilogueRegs>();
        // Thread: a row and 128 columns of D (GLU: 64 of gate and the same 64 of up). The row's scales are fetched four
        // blocks ahead, the next tile's first ones during this tile's last blocks.
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t col0 = GLU ? 64 * half : 128 * half;
        float nx[4];
        auto source = [&](const Fp8Tile& t) -> const float* {
            if (row >= t.rows) return nullptr;
            const int r = c.rows ? __ldg(c.rows + t.row0 + row) : t.row0 + row;
            return r >= 0 && r < c.x_rows ? c.xs + r * c.xs_stride : nullptr;
        };
        auto fetch = [&](const float* p, int kb) {
            if (p && c.quads && kb + 4 <= KB) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(p + kb));
                nx[0] = v.x;
                nx[1] = v.y;
                nx[2] = v.z;
                nx[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) nx[i] = p && kb + i < KB ? __ldg(p + kb + i) : 0.f;
            }
        };
        // weight scales of the thread's columns
        auto wscale = [&](const Fp8Tile& t, int g) {
            const int nb = GLU ? t.col : min(2 * t.col + half, (c.N - 1) / kFp8Block);
            return c.ws[g] + t.e * c.ws_expert[g] + nb * c.ws_row[g];
        };
        int seq = 0;
        bool ok = true;
        int t = blockIdx.x;
        Fp8Tile tile = {0, 0, 0, 0};
        const float *sp = nullptr, *w0 = nullptr, *w1 = nullptr;
        float s0 = 0.f, s1 = 0.f;
        if (t < total) {
            tile = fp8_tile(c, groups, t, 0, kF8Tile, cols, false);
            sp = source(tile);
            fetch(sp, 0);
            w0 = wscale(tile, 0);
            s0 = __ldg(w0);
            if (GLU) {
                w1 = wscale(tile, 1);
                s1 = __ldg(w1);
            }
        }
        for (; t < total; t += gridDim.x) {
            Fp8Tile next = {0, 0, 0, 0};
            const float *sp_next = nullptr, *w0_next = nullptr, *w1_next = nullptr;
            if (t + (int)gridDim.x < total) {
                next = fp8_tile(c, groups, t + gridDim.x, tile.e, kF8Tile, cols, false);
                sp_next = source(next);
                w0_next = wscale(next, 0);
                if (GLU) w1_next = wscale(next, 1);
            }
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            float cur[4] = {0.f, 0.f, 0.f, 0.f};
            for (int kb = 0; kb < KB; ++kb, ++seq) {
                const int buf = seq & 1;
                if ((kb & 3) == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) cur[i] = nx[i];
                    if (kb + 4 < KB)
                        fetch(sp, kb + 4);
                    else
                        fetch(sp_next, 0);
                }
                const float f0 = cur[0] * s0, f1 = cur[0] * s1;
                cur[0] = cur[1];
                cur[1] = cur[2];
                cur[2] = cur[3];
                const bool last = kb + 1 == KB;
                if (!last || w0_next) s0 = __ldg(last ? w0_next : w0 + kb + 1);
                if (GLU && (!last || w1_next)) s1 = __ldg(last ? w1_next : w1 + kb + 1);
                const uint64_t g0 = f2_pack(__float_as_uint(f0), __float_as_uint(f0));
                const uint64_t g1 = GLU ? f2_pack(__float_as_uint(f1), __float_as_uint(f1)) : g0;
                ok = mbar_wait(tfull0 + 8 * buf, (seq >> 1) & 1, flags, err, wait_ns);
                tc_fence_after();
                const uint32_t base = lane_base + 256 * buf + col0;
                // 32 columns at a time (GLU: two of gate, two of up), the next ones on their way during the sums
                uint32_t v[2][32];
                f8_ld<32>(base, v[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f8_wait_ld<32>(v[i & 1]);
                    if (i < 3) {
                        f8_ld<32>(base + (GLU ? ((i + 1) >> 1) * 128 + ((i + 1) & 1) * 32 : (i + 1) * 32), v[(i + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        mbar_arrive_if(tempty0 + 8 * buf, lane == 0);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        f2_fma(acc[16 * i + j], f2_pack(v[i & 1][2 * j], v[i & 1][2 * j + 1]), GLU && i >= 2 ? g1 : g0);
                }
            }
            // the results: 128 columns, or 64 of silu(g) u
            constexpr int kMine = GLU ? 64 : 128;
            const int n0 = tile.col * Geo::kOut + half * kMine;
            const bool live = ok && row < tile.rows;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 p = f2_unpack(acc[i]), q = f2_unpack(acc[32 + i]);
                    acc[i] = f2_pack(__float_as_uint(silu_mul(p.x, q.x)), __float_as_uint(silu_mul(p.y, q.y)));
                }
            }
            const long long at = (long long)(tile.row0 + row) * c.y_stride + n0;
            if (GLU && c.dtype == NQ_E4M3) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    // (columns past N are sums over zeros)
                    const float2 p = f2_unpack(acc[i]);
                    if (n0 + 2 * i < c.N) m = bits_max(bits_max(m, p.x), p.y);
                }
                largest[half * 128 + row] = m;
                named_bar_sync(1 + quarter, 64);
                m = max(m, largest[(half ^ 1) * 128 + row]);
                named_bar_sync(1 + quarter, 64);
                const float s = fp8_scale(__uint_as_float(m));
                if (live) {
                    if (half == 0) c.ys[(tile.row0 + row) * c.ys_stride + tile.col] = s;
#pragma unroll
                    for (int i = 0; i < 64; i += 16) {
                        if (n0 + i >= c.N) break;
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 p = f2_unpack(acc[i / 2 + 2 * j]), q = f2_unpack(acc[i / 2 + 2 * j + 1]);
                            u[j] = fp8_codes(p.x / s, p.y / s, q.x / s, q.y / s);
                        }
                        *reinterpret_cast<uint4*>(c.y + at + i) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            } else if (c.wide) {
                uint16_t* const y = reinterpret_cast<uint16_t*>(c.y) + at;
                const bool bf16 = c.dtype == NQ_BF16;
#pragma unroll
                for (int i = 0; i < kMine; i += 16) {
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 p = f2_unpack(acc[i / 2 + j]);
                        u[j] = pack_16(p.x, p.y, bf16);
                    }
                    if (live && n0 + i + 16 <= c.N) {
                        store_32(y + i, u);
                    } else if (live) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (n0 + i + j < c.N) y[i + j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
                    }
                }
            } else {
                // rows at odd addresses: a warp's 32 x 32 results turned in shared memory, so that its lanes store
                // neighbouring columns (each its own row's: 32 memory sectors a store instead of two or three)
                uint16_t* const mine = turn + warp * 32 * 34;
                const bool bf16 = c.dtype == NQ_BF16;
                const int rows_here = ok ? min(32, tile.rows - 32 * quarter) : 0;
#pragma unroll
                for (int i = 0; i < kMine; i += 32) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 p = f2_unpack(acc[i / 2 + j]);
                        *reinterpret_cast<uint32_t*>(mine + lane * 34 + 2 * j) = pack_16(p.x, p.y, bf16);
                    }
                    __syncwarp();
                    if (n0 + i + lane < c.N)
                        for (int r = 0; r < rows_here; ++r)
                            reinterpret_cast<uint16_t*>(c.y)[(long long)(tile.row0 + 32 * quarter + r) * c.y_stride + n0 + i + lane] =
                                mine[r * 34 + lane];
                    __syncwarp();
                }
            }
            tile = next;
            sp = sp_next;
            w0 = w0_next;
            w1 = w1_next;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- few rows a group

template <int BN, bool GLU>
struct Fp8ColsGeo {
    static constexpr int kParts = GLU ? 2 : 1;
    static constexpr int kXBytes = BN * kF8Row;
    static constexpr int kStageBytes = kParts * kF8Tile * kF8Row + kXBytes;
    static constexpr int kBufs = 512 / (BN * kParts) < 4 ? 512 / (BN * kParts) : 4;
    static constexpr int kScaleBlocks = 4;       // blocks of K of a step of the scales' ring
    static constexpr int kScaleSteps = 3;
    static constexpr int kScaleBytes = kScaleSteps * kScaleBlocks * kParts * BN * 4;
    static constexpr int kCtrlBytes = 640 + 2048;   // barriers, flags; the warps' largest values [4][128]
    static constexpr int stages(int extra) {
        const int s = (kSmemLimit - 1024 - kScaleBytes - kCtrlBytes - f8_group_bytes(kMostExperts) - extra) / kStageBytes;
        return s < kF8MaxStages ? s : kF8MaxStages;
    }
    static constexpr int kStages = stages(0);
    static int smem(int E) { return 1024 + kStages * kStageBytes + kScaleBytes + kCtrlBytes + f8_group_bytes(E); }
};

template <int BN, bool GLU>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_cols_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8ColsGeo<BN, GLU>;
    constexpr int kStages = Geo::kStages, kParts = Geo::kParts, kBufs = Geo::kBufs, kBlocks = Geo::kScaleBlocks;
    constexpr int kSteps = Geo::kScaleSteps;
    const Fp8Call& c = a.c;
    extern __shared__ uint8_t f8_smem[];
    uint8_t* const ring = f8_smem + ((1024u - (smem_u32(f8_smem) & 1023u)) & 1023u);
    float* const scales = reinterpret_cast<float*>(ring + kStages * Geo::kStageBytes);   // [steps][blocks][parts][BN]
    uint8_t* const ctrl = reinterpret_cast<uint8_t*>(scales) + Geo::kScaleBytes;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
    // bars: full[16], empty[16], tfull[4], tempty[4], sfull[4], sempty[4], done
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kF8MaxStages, tfull0 = empty0 + 8 * kF8MaxStages;
    const uint32_t tempty0 = tfull0 + 32, sfull0 = tempty0 + 32, sempty0 = sfull0 + 32, done = sempty0 + 32;
    volatile int* const flags = reinterpret_cast<volatile int*>(ctrl + 448);     // [0] abort, [3] TMEM base
    int* const sums = reinterpret_cast<int*>(ctrl + 512);
    uint32_t* const largest = reinterpret_cast<uint32_t*>(ctrl + 640);           // [4 quarters][BN]
    Fp8Groups groups;
    groups.before = reinterpret_cast<int*>(ctrl + Geo::kCtrlBytes);
    groups.start = groups.before + c.E + 1;
    groups.end = groups.start + c.E;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t wait_ns = c.wait_ns;
    int* const err = c.err;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, kF8Epilogue);
        }
        for (int i = 0; i < kSteps; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, kF8Epilogue);
        }
        mbar_init(done, 1);
        flags[0] = 0;
        mbar_fence_init();
    }
    if (warp == 0) tmem_alloc(smem_u32(const_cast<int*>(flags) + 3), 512);
    grid_launch_dependents();
    grid_dependency_wait();
    const int cols = (c.N + kF8Tile - 1) / kF8Tile, KB = (c.K + kFp8Block - 1) / kFp8Block;
    const int total = fp8_groups(c, groups, BN, cols, sums);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];

    // (each branch begins with its own count: where the paths met again, everything would have to fit the smaller)
    if (warp >= kF8Epilogue) {
        regs_fewer<kF8OtherRegs>();
    if (warp == kF8Producer) {
        // ------------------------------------------------------------ copies
        int seq = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            int at[4];
            const int fours = f8_gather_rows(c, tile, at);
            for (int kb = 0; kb < KB && ok; ++kb, ++seq) {
                const int st = seq % kStages;
                if (seq >= kStages) ok = mbar_wait(empty0 + 8 * st, ((seq / kStages) - 1) & 1, flags, err, wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t wa = smem_u32(ring + st * Geo::kStageBytes), xa = wa + kParts * kF8Tile * kF8Row, bar = full0 + 8 * st;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)(kParts * kF8Tile * kF8Row + (c.rows ? fours * 4 : BN) * kF8Row));
#pragma unroll
                    for (int g = 0; g < kParts; ++g)
                        tma_load_3d(wa + g * kF8Tile * kF8Row, &a.wmap[g], kb * kFp8Block, tile.col * kF8Tile, tile.e, bar);
                    if (!c.rows) tma_load_2d(xa, &a.xmap, kb * kFp8Block, tile.row0, bar);
                }
                __syncwarp();
                if (lane < fours) tma_gather4(xa + 4 * lane * kF8Row, &a.xmap, kb * kFp8Block, at, bar);
            }
        }
        if (!ok)
            for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)
                mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
    } else if (warp == kF8Mma) {
        // ------------------------------------------------------------ MMA issuer
        const bool leader = elect_one();
        int seq = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            const uint32_t idesc = f8_idesc(kF8Tile, min(BN, max(16, (tile.rows + 15) / 16 * 16)));
            for (int kb = 0; kb < KB && ok; ++kb, ++seq) {
                const int st = seq % kStages, buf = seq % kBufs;
                ok = mbar_wait(full0 + 8 * st, (seq / kStages) & 1, flags, err, wait_ns);
                if (seq >= kBufs) ok = ok && mbar_wait(tempty0 + 8 * buf, ((seq / kBufs) - 1) & 1, flags, err, wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t wa = smem_u32(ring + st * Geo::kStageBytes), xa = wa + kParts * kF8Tile * kF8Row;
#pragma unroll
                for (int g = 0; g < kParts; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        f8_mma(tmem + (buf * kParts + g) * BN, smem_desc_sw128(wa + g * kF8Tile * kF8Row + 32 * j),
                               smem_desc_sw128(xa + 32 * j), idesc, j > 0 ? 1u : 0u, leader);
                tc_commit(empty0 + 8 * st, leader);
                tc_commit(tfull0 + 8 * buf, leader);
            }
        }
        tc_commit(done, leader);
        mbar_wait_drain(done, 0, kDrainNs);
    } else if (warp == kF8Scales) {
        // ------------------------------------------------------------ scales
        // The product of a row's and the weight block's scale, for four blocks of K a step.
        int step = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            constexpr int kPer = (BN + 31) / 32;
            const float* sp[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = 32 * i + lane;
                sp[i] = nullptr;
                if (r < tile.rows) {
                    const int s = c.rows ? __ldg(c.rows + tile.row0 + r) : tile.row0 + r;
                    if (s >= 0 && s < c.x_rows) sp[i] = c.xs + s * c.xs_stride;
                }
            }
            const float* w[kParts];
#pragma unroll
            for (int g = 0; g < kParts; ++g) w[g] = c.ws[g] + tile.e * c.ws_expert[g] + tile.col * c.ws_row[g];
            for (int kb = 0; kb < KB && ok; kb += kBlocks, ++step) {
                float sw[kParts][kBlocks], sx[kPer][kBlocks];
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int g = 0; g < kParts; ++g) sw[g][b] = kb + b < KB ? __ldg(w[g] + kb + b) : 0.f;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (sp[i] && c.quads && kb + 4 <= KB) {
                        const float4 v = __ldg(reinterpret_cast<const float4*>(sp[i] + kb));
                        sx[i][0] = v.x;
                        sx[i][1] = v.y;
                        sx[i][2] = v.z;
                        sx[i][3] = v.w;
                    } else {
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b) sx[i][b] = sp[i] && kb + b < KB ? __ldg(sp[i] + kb + b) : 0.f;
                    }
                }
                const int slot = step % kSteps;
                if (step >= kSteps) ok = mbar_wait(sempty0 + 8 * slot, ((step / kSteps) - 1) & 1, flags, err, wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                float* const to = scales + slot * kBlocks * kParts * BN;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int r = 32 * i + lane;
                    if (r < BN)
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                            for (int g = 0; g < kParts; ++g) to[(b * kParts + g) * BN + r] = sx[i][b] * sw[g][b];
                }
                __syncwarp();
                mbar_arrive_if(sfull0 + 8 * slot, lane == 0);
            }
        }
    }
    } else {
        // ------------------------------------------------------------ epilogue
        regs_more<kF8EpilogueRegs>();
        // Thread: a column of the result (a row of the weight) for half of the tile's rows.
        constexpr int kMine = BN / 2, kChunk = kMine < 32 ? kMine : 32;
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16) + half * kMine;
        int seq = 0, step = 0, e = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            uint64_t acc[kParts][kMine / 2];
#pragma unroll
            for (int g = 0; g < kParts; ++g)
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i) acc[g][i] = 0;
            const bool any = half * kMine < tile.rows;
            for (int kb = 0; kb < KB; ++kb, ++seq) {
                const int buf = seq % kBufs, slot = step % kSteps;
                if (kb % kBlocks == 0) ok = mbar_wait(sfull0 + 8 * slot, (step / kSteps) & 1, flags, err, wait_ns);
                ok = mbar_wait(tfull0 + 8 * buf, (seq / kBufs) & 1, flags, err, wait_ns);
                tc_fence_after();
                if (any) {
                    const float* const s = scales + (slot * kBlocks + kb % kBlocks) * kParts * BN + half * kMine;
#pragma unroll
                    for (int g = 0; g < kParts; ++g)
#pragma unroll
                        for (int i = 0; i < kMine; i += kChunk) {
                            uint32_t v[kChunk];
                            f8_ld<kChunk>(lane_base + (buf * kParts + g) * BN + i, v);
                            f8_wait_ld<kChunk>(v);
#pragma unroll
                            for (int j = 0; j < kChunk; j += 4) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + g * BN + i + j);
                                f2_fma(acc[g][(i + j) / 2], f2_pack(v[j], v[j + 1]), f.x);
                                f2_fma(acc[g][(i + j) / 2 + 1], f2_pack(v[j + 2], v[j + 3]), f.y);
                            }
                        }
                }
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(tempty0 + 8 * buf, lane == 0);
                if (kb % kBlocks == kBlocks - 1 || kb + 1 == KB) {
                    mbar_arrive_if(sempty0 + 8 * slot, lane == 0);
                    ++step;
                }
            }
            const int n = tile.col * kF8Tile + row;
            const int rows_here = ok ? min(kMine, tile.rows - half * kMine) : 0;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i) {
                    const float2 p = f2_unpack(acc[0][i]), q = f2_unpack(acc[1][i]);
                    acc[0][i] = f2_pack(__float_as_uint(silu_mul(p.x, q.x)), __float_as_uint(silu_mul(p.y, q.y)));
                }
            }
            const long long first = tile.row0 + half * kMine;
            if (GLU && c.dtype == NQ_E4M3) {
                // a row's largest over the tile's 128 columns: the warp's, then the four warps' of this half
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const float2 p = f2_unpack(acc[0][i / 2]);
                    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, n < c.N ? bits_max(0, i & 1 ? p.y : p.x) : 0u);
                    if (lane == 0) largest[quarter * BN + half * kMine + i] = m;
                }
                named_bar_sync(1 + half, 128);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    if (i < rows_here) {
                        uint32_t m = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) m = max(m, largest[q * BN + half * kMine + i]);
                        const float s = fp8_scale(__uint_as_float(m));
                        const float2 p = f2_unpack(acc[0][i / 2]);
                        if (row == 0) c.ys[(first + i) * c.ys_stride + tile.col] = s;
                        if (n < c.N) c.y[(first + i) * c.y_stride + n] = (uint8_t)fp8_codes((i & 1 ? p.y : p.x) / s, 0.f, 0.f, 0.f);
                    }
                }
                named_bar_sync(1 + half, 128);   // the next tile's largest use the same place
            } else if (n < c.N) {
                uint16_t* const y = reinterpret_cast<uint16_t*>(c.y) + first * c.y_stride + n;
                const bool bf16 = c.dtype == NQ_BF16;
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const float2 p = f2_unpack(acc[0][i / 2]);
                    if (i < rows_here) y[i * c.y_stride] = (uint16_t)pack_16(i & 1 ? p.y : p.x, 0.f, bf16);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace nq
