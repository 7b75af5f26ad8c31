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

constexpr int kF8Epilogue = 8;                   // epilogue warps of fp8_cols_kernel: 0..7, then
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
    int split;                                   // blocks that share a tile's K (fp8_cols_kernel)
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

// The products of one block of K (four MMAs of 32 codes) into a fresh accumulator, and an arrival when all before has
// been done: for one thread. Descriptors as smem_desc_sw128's: `a`, `b` are their low words. Over a pair of blocks
// (cta_group::2) the even block issues them for both, each holding its rows of A and D and half of B's, and the arrival is on
// the barrier at this address in both.
__device__ __forceinline__ uint32_t f8_desc(uint32_t addr) { return (addr & 0x3FFFF) >> 4; }
#define NQ_F8_MMA(group)                                                        \
    "{\n\t.reg .b64 x, y;\n\t.reg .pred p;\n\tsetp.ne.b32 p, 0, 0;\n\t"            \
    "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"                            \
    "tcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], x, y, %3, p;\n\t"        \
    "setp.eq.b32 p, 0, 0;\n\tadd.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"            \
    "tcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], x, y, %3, p;\n\t"        \
    "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"                                    \
    "tcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], x, y, %3, p;\n\t"        \
    "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"                                    \
    "tcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], x, y, %3, p;\n\t}"
template <bool PAIR = false>
__device__ __forceinline__ void f8_mma_block(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc) {
    constexpr uint32_t kHigh = (uint32_t)(((uint64_t)(1024 >> 4) << 32 | (1ull << 46) | (2ull << 61)) >> 32);
    if constexpr (PAIR)
        asm volatile(NQ_F8_MMA("2")::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(kHigh) : "memory");
    else
        asm volatile(NQ_F8_MMA("1")::"r"(d_tmem), "r"(a), "r"(b), "r"(idesc), "r"(kHigh) : "memory");
}
#undef NQ_F8_MMA
template <bool PAIR = false>
__device__ __forceinline__ void f8_commit(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void f8_alloc(uint32_t dst_smem) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dst_smem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst_smem, 512);
    }
}
template <bool PAIR>
__device__ __forceinline__ void f8_dealloc(uint32_t taddr) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
    else
        tmem_dealloc(taddr, 512);
}
// Arrival on a barrier of the pair's even block that publishes nothing outside TMEM.
__device__ __forceinline__ void f8_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A place in a ring of n, and the parity of the round.
template <int n>
struct F8Ring {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++at == n) {
            at = 0;
            parity ^= 1;
        }
    }
};

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
__device__ __forceinline__ int f8_gather_rows(const Fp8Call& c, const Fp8Tile& tile, int first, int most, int (&at)[4]) {
    if (!c.rows) return 0;
    const int lane = threadIdx.x & 31, rows = min(tile.rows - first, most);   // of the tile's rows from `first` on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = __ldg(c.rows + tile.row0 + min(first + 4 * lane + i, tile.rows - 1));
        at[i] = s >= 0 && s < c.x_rows ? s : c.x_past;
    }
    return rows > 0 ? (rows + 3) / 4 : 0;
}

// ---------------------------------------------------------------- many rows a group

// The scales' warp: for each row of a tile and each block of K the product of the row's scale and the weight block's, for
// PARTS weight blocks, four blocks of K a step, into a ring [step][block][part][ROWS]. KB blocks of K from k0 on; tiles
// t0, t0 + dt, ... of `high` rows, of which the block has ROWS from `first` on. wscale(tile, part): the weight's scales
// along K.
constexpr int kF8ScaleBlocks = 4, kF8ScaleSteps = 2;
constexpr int f8_scale_bytes(int rows, int parts) { return kF8ScaleSteps * kF8ScaleBlocks * parts * rows * 4; }
template <int ROWS, int PARTS, typename W>
__device__ __forceinline__ void f8_scales(const Fp8Call& c, const Fp8Groups& groups, int t0, int dt, int total, int high, int first,
                                          int cols, bool even, float* scales, uint32_t sfull0, uint32_t sempty0,
                                          volatile int* flags, int k0, int KB, W wscale) {
    constexpr int kPer = (ROWS + 31) / 32;
    const int lane = threadIdx.x & 31;
    int step = 0, e = 0;
    bool ok = true;
    for (int t = t0; t < total && ok; t += dt) {
        const Fp8Tile tile = fp8_tile(c, groups, t, e, high, cols, even);
        e = tile.e;
        const float* sp[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = first + 32 * i + lane;
            sp[i] = nullptr;
            if (r < tile.rows) {
                const int s = c.rows ? __ldg(c.rows + tile.row0 + r) : tile.row0 + r;
                if (s >= 0 && s < c.x_rows) sp[i] = c.xs + s * c.xs_stride + k0;
            }
        }
        const float* w[PARTS];
#pragma unroll
        for (int g = 0; g < PARTS; ++g) w[g] = wscale(tile, g) + k0;
        for (int kb = 0; kb < KB && ok; kb += kF8ScaleBlocks, ++step) {
            float sw[PARTS][kF8ScaleBlocks], sx[kPer][kF8ScaleBlocks];
#pragma unroll
            for (int b = 0; b < kF8ScaleBlocks; ++b)
#pragma unroll
                for (int g = 0; g < PARTS; ++g) sw[g][b] = kb + b < KB ? __ldg(w[g] + kb + b) : 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (sp[i] && c.quads && k0 % 4 == 0 && kb + 4 <= KB) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(sp[i] + kb));
                    sx[i][0] = v.x;
                    sx[i][1] = v.y;
                    sx[i][2] = v.z;
                    sx[i][3] = v.w;
                } else {
#pragma unroll
                    for (int b = 0; b < kF8ScaleBlocks; ++b) sx[i][b] = sp[i] && kb + b < KB ? __ldg(sp[i] + kb + b) : 0.f;
                }
            }
            const int slot = step % kF8ScaleSteps;
            if (step >= kF8ScaleSteps)
                ok = mbar_wait(sempty0 + 8 * slot, ((step / kF8ScaleSteps) - 1) & 1, flags, c.err, c.wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            float* const to = scales + slot * kF8ScaleBlocks * PARTS * ROWS;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = 32 * i + lane;
                if (r < ROWS)
#pragma unroll
                    for (int b = 0; b < kF8ScaleBlocks; ++b)
#pragma unroll
                        for (int g = 0; g < PARTS; ++g) to[(b * PARTS + g) * ROWS + r] = sx[i][b] * sw[g][b];
            }
            __syncwarp();
            mbar_arrive_if(sfull0 + 8 * slot, lane == 0);
        }
    }
}

template <bool GLU, bool PAIR>
struct Fp8RowsGeo {
    static constexpr int kOut = GLU ? 128 : 256; // columns of the result in a tile; D has 256: those, or gate and up
    static constexpr int kHigh = PAIR ? 256 : 128;               // rows of a tile
    static constexpr int kW = PAIR ? 128 : 256;  // the weights' rows that a block loads
    static constexpr int kStageBytes = (kF8Tile + kW) * kF8Row;
    static constexpr int kStages = PAIR ? 6 : 4;
    // A pair's products are issued in halves of 128 columns, each with its barriers and its warps, so that an accumulator
    // of the next block of K is free while the epilogue still adds the other half's. (Of a single block, whose
    // copies from L2 take longer than its products, the halves' second read of A from shared memory costs more.)
    static constexpr int kHalves = PAIR ? 2 : 1;
    static constexpr int kWarps = 16;            // of the epilogue
    static constexpr int kThreads = (kWarps + 4) * 32;
    static constexpr int kRegs = 104, kOtherRegs = 64;
    static_assert(kWarps * 32 * kRegs + 4 * 32 * kOtherRegs == kThreads * 96, "registers of a block");
    static constexpr int kScaleBytes = f8_scale_bytes(kF8Tile, 2);
    static constexpr int kTurnBytes = kWarps * 8 * 34 * 2;       // a warp's 8 x 32 results
    static constexpr int kLargestBytes = 4 * kF8Tile * 4;
    static constexpr int kCtrlBytes = 512 + kLargestBytes + kScaleBytes + kTurnBytes;
    static int smem(int E) { return 1024 + kStages * kStageBytes + kCtrlBytes + f8_group_bytes(E); }
};

template <bool GLU, bool PAIR>
__global__ void __launch_bounds__(Fp8RowsGeo<GLU, PAIR>::kThreads, 1) fp8_rows_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8RowsGeo<GLU, PAIR>;
    constexpr int kStages = Geo::kStages, kHalves = Geo::kHalves, kWarps = Geo::kWarps, kPair = PAIR ? 2 : 1;
    constexpr int kProducer = kWarps, kMma = kWarps + 1, kScales = kWarps + 2;
    const Fp8Call& c = a.c;
    extern __shared__ uint8_t f8_smem[];
    uint8_t* const ring = f8_smem + ((1024u - (smem_u32(f8_smem) & 1023u)) & 1023u);
    uint8_t* const ctrl = ring + kStages * Geo::kStageBytes;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
    // bars: full[8], empty[8], full_other[8] (the odd block's stages, passed on to the even one), tfull[2 halves][2],
    // tempty[2 halves][2], sfull[2], sempty[2], done
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 64, other0 = empty0 + 64, tfull0 = other0 + 64, tempty0 = tfull0 + 32;
    const uint32_t sfull0 = tempty0 + 32, sempty0 = sfull0 + 16, done = sempty0 + 16;
    volatile int* const flags = reinterpret_cast<volatile int*>(ctrl + 352);     // [0] abort, [3] TMEM base
    int* const sums = reinterpret_cast<int*>(ctrl + 384);
    uint32_t* const largest = reinterpret_cast<uint32_t*>(ctrl + 512);           // [4 column groups][128 rows]
    float* const scales = reinterpret_cast<float*>(ctrl + 512 + Geo::kLargestBytes);   // [steps][blocks][2][128 rows]
    uint16_t* const turn = reinterpret_cast<uint16_t*>(ctrl + 512 + Geo::kLargestBytes + Geo::kScaleBytes);
    Fp8Groups groups;
    groups.before = reinterpret_cast<int*>(ctrl + Geo::kCtrlBytes);
    groups.start = groups.before + c.E + 1;
    groups.end = groups.start + c.E;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0, first = rank * kF8Tile;     // this block's rows of a tile
    const int t0 = blockIdx.x / kPair, dt = gridDim.x / kPair;
    const uint64_t wait_ns = c.wait_ns;
    int* const err = c.err;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
            mbar_init(other0 + 8 * i, 1);
        }
        for (int i = 0; i < 2 * kHalves; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, kPair * kWarps / kHalves);
        }
        for (int i = 0; i < kF8ScaleSteps; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, kWarps);
        }
        mbar_init(done, 1);
        flags[0] = 0;
        mbar_fence_init();
    }
    if (warp == 0) f8_alloc<PAIR>(smem_u32(const_cast<int*>(flags) + 3));
    grid_launch_dependents();
    grid_dependency_wait();
    const int cols = (c.N + Geo::kOut - 1) / Geo::kOut, KB = (c.K + kFp8Block - 1) / kFp8Block;
    const int total = fp8_groups(c, groups, Geo::kHigh, cols, sums);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];
    if constexpr (PAIR) cluster_sync_all();      // both blocks' barriers are initialised

    // (each branch begins with its own count of registers: where the paths met again, everything would have to fit the smaller)
    if (warp >= kWarps) {
        regs_fewer<Geo::kOtherRegs>();
        if (warp == kProducer) {
            // -------------------------------------------------------- copies
            F8Ring<kStages> in;
            int seq = 0, e = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Fp8Tile tile = fp8_tile(c, groups, t, e, Geo::kHigh, cols, false);
                e = tile.e;
                int at[4];
                const int fours = f8_gather_rows(c, tile, first, kF8Tile, at);
                for (int kb = 0; kb < KB; ++kb, ++seq) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * in.at, in.parity ^ 1, flags, err, wait_ns));
                    if (!ok) break;
                    const uint32_t xa = smem_u32(ring) + in.at * Geo::kStageBytes, wa = xa + kF8Tile * kF8Row, bar = full0 + 8 * in.at;
                    in.next();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, (uint32_t)(Geo::kW * kF8Row + (c.rows ? fours * 4 : kF8Tile) * kF8Row));
                        const int k = kb * kFp8Block;
                        if (GLU && PAIR) {       // a block each of gate and up
                            tma_load_3d(wa, &a.wmap[rank], k, tile.col * 128, tile.e, bar);
                        } else if (GLU) {
                            tma_load_3d(wa, &a.wmap[0], k, tile.col * 128, tile.e, bar);
                            tma_load_3d(wa + 128 * kF8Row, &a.wmap[1], k, tile.col * 128, tile.e, bar);
                        } else {
                            tma_load_3d(wa, &a.wmap[0], k, tile.col * 256 + rank * 128, tile.e, bar);
                        }
                        if (!c.rows) tma_load_2d(xa, &a.xmap, k, tile.row0 + first, bar);
                    }
                    __syncwarp();
                    if (lane < fours) tma_gather4(xa + 4 * lane * kF8Row, &a.xmap, kb * kFp8Block, at, bar);
                }
            }
            if (!ok)
                for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)
                    mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
        } else if (PAIR && warp == kMma && rank == 1) {
            // -------------------------------------------------------- the odd block's stages, passed on
            F8Ring<kStages> in;
            bool ok = true;
            const uint32_t to = cluster_map(other0, 0);
            for (int t = t0; t < total && ok; t += dt)
                for (int kb = 0; kb < KB && ok; ++kb) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(full0 + 8 * in.at, in.parity, flags, err, wait_ns));
                    if (ok && lane == 0) f8_arrive_remote(to + 8 * in.at);
                    in.next();
                }
        } else if (warp == kMma) {
            // -------------------------------------------------------- MMA issuer
            if (elect_one()) {
                F8Ring<kStages> in;
                F8Ring<2> out;
                int e = 0;
                bool ok = true;
                const uint32_t x0 = f8_desc(smem_u32(ring));
                auto wait_free = [&](uint32_t bar) {
                    if constexpr (PAIR)
                        return mbar_wait_cluster(bar, out.parity ^ 1, flags, err, wait_ns);
                    else
                        return mbar_wait(bar, out.parity ^ 1, flags, err, wait_ns);
                };
                for (int t = t0; t < total && ok; t += dt) {
                    const Fp8Tile tile = fp8_tile(c, groups, t, e, Geo::kHigh, cols, false);
                    e = tile.e;
                    const int n = PAIR ? 256 / kHalves : (GLU ? 256 : min(256, (c.N - tile.col * Geo::kOut + 15) / 16 * 16));
                    const uint32_t idesc = f8_idesc(kPair * kF8Tile, n);
                    for (int kb = 0; kb < KB && ok; ++kb) {
                        const uint32_t x = x0 + in.at * (Geo::kStageBytes / 16);
                        ok = mbar_wait(full0 + 8 * in.at, in.parity, flags, err, wait_ns);
                        if (PAIR) ok = ok && mbar_wait_cluster(other0 + 8 * in.at, in.parity, flags, err, wait_ns);
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) {
                            ok = ok && wait_free(tempty0 + 8 * (2 * h + out.at));
                            if (!ok) break;
                            tc_fence_after();
                            f8_mma_block<PAIR>(tmem + 256 * out.at + 128 * h, x, x + (kF8Tile + 64 * h) * kF8Row / 16, idesc);
                            f8_commit<PAIR>(tfull0 + 8 * (2 * h + out.at));
                        }
                        if (!ok) break;
                        f8_commit<PAIR>(empty0 + 8 * in.at);
                        in.next();
                        out.next();
                    }
                }
                f8_commit<PAIR>(done);           // every MMA has completed before TMEM can be freed
                mbar_wait_drain(done, 0, kDrainNs);
            }
            __syncwarp();
        } else if (warp == kScales) {
            // of the two blocks of columns, or of gate and up
            f8_scales<kF8Tile, 2>(c, groups, t0, dt, total, Geo::kHigh, first, cols, false, scales, sfull0, sempty0, flags, 0, KB,
                                  [&](const Fp8Tile& tile, int g) {
                                      const int nb = GLU ? tile.col : min(2 * tile.col + g, (c.N - 1) / kFp8Block);
                                      return c.ws[GLU ? g : 0] + tile.e * c.ws_expert[GLU ? g : 0] + nb * c.ws_row[GLU ? g : 0];
                                  });
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread: a row and 64 columns of D, two runs of 32 that begin at d0 and d1: neighbours, or gate and up of the same
        // 32 columns of the result, which begin at n0 of the tile's. A pair's D has in each half of 128 columns 64 from either
        // block's weights.
        regs_more<Geo::kRegs>();
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
        const int half = PAIR ? group >> 1 : 0, sub = group & 1;
        constexpr int kMine = GLU ? 32 : 64;
        int d0, d1, n0, part;                    // part: whose scales
        if (GLU) {
            d0 = PAIR ? 128 * half + 32 * sub : 32 * group;
            d1 = d0 + (PAIR ? 64 : 128);
            n0 = 32 * group;
            part = 0;
        } else {
            d0 = 64 * group;
            d1 = d0 + 32;
            n0 = PAIR ? 128 * sub + 64 * half : 64 * group;
            part = n0 >> 7;
        }
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t tfull = tfull0 + 16 * half;
        // where this warp frees an accumulator: the issuing block's barrier
        const uint32_t tempty = (PAIR && rank == 1 ? cluster_map(tempty0, 0) : tempty0) + 16 * half;
        F8Ring<2> in;
        F8Ring<kF8ScaleSteps> sc;
        int e = 0;
        bool ok = true;
        for (int t = t0; t < total; t += dt) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, Geo::kHigh, cols, false);
            e = tile.e;
            uint64_t acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0;
            for (int kb = 0; kb < KB; ++kb) {
                const int block = kb % kF8ScaleBlocks;
                if (block == 0) mbar_wait(sfull0 + 8 * sc.at, sc.parity, flags, err, wait_ns);
                const float* const s = scales + (sc.at * kF8ScaleBlocks + block) * 2 * kF8Tile + row;
                const uint32_t f0 = __float_as_uint(s[part * kF8Tile]), f1 = GLU ? __float_as_uint(s[kF8Tile]) : f0;
                ok = mbar_wait(tfull + 8 * in.at, in.parity, flags, err, wait_ns);
                tc_fence_after();
                const uint32_t base = lane_base + 256 * in.at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[16];
                    f8_ld<16>(base + (i < 2 ? d0 + 16 * i : d1 + 16 * (i - 2)), v);
                    f8_wait_ld<16>(v);
                    if (i == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (PAIR && rank == 1) {
                            if (lane == 0) f8_arrive_remote(tempty + 8 * in.at);
                        } else {
                            mbar_arrive_if(tempty + 8 * in.at, lane == 0);
                        }
                    }
                    const uint64_t f = f2_pack(i < 2 ? f0 : f1, i < 2 ? f0 : f1);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f2_fma(acc[8 * i + j], f2_pack(v[2 * j], v[2 * j + 1]), f);
                }
                in.next();
                if (block == kF8ScaleBlocks - 1 || kb + 1 == KB) {
                    __syncwarp();
                    mbar_arrive_if(sempty0 + 8 * sc.at, lane == 0);
                    sc.next();
                }
            }
            // the results: 64 columns, or 32 of silu(g) u
            const int n = tile.col * Geo::kOut + n0, my_row = tile.row0 + first + row;
            const bool live = ok && first + row < tile.rows;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 p = f2_unpack(acc[i]), q = f2_unpack(acc[16 + i]);
                    acc[i] = f2_pack(__float_as_uint(silu_mul(p.x, q.x)), __float_as_uint(silu_mul(p.y, q.y)));
                }
            }
            const long long at = (long long)my_row * c.y_stride + n;
            if (GLU && c.dtype == NQ_E4M3) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 p = f2_unpack(acc[i]);
                    if (n + 2 * i < c.N) m = bits_max(bits_max(m, p.x), p.y);
                }
                largest[group * kF8Tile + row] = m;
                named_bar_sync(1 + quarter, 128);        // the row's four warps
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max(m, largest[i * kF8Tile + row]);
                named_bar_sync(1 + quarter, 128);        // the next tile's use the same place
                const float s = fp8_scale(__uint_as_float(m));
                if (live) {
                    if (group == 0) c.ys[my_row * c.ys_stride + tile.col] = s;
#pragma unroll
                    for (int i = 0; i < kMine; i += 16) {
                        if (n + i >= c.N) break;
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 p = f2_unpack(acc[(i / 2 + 2 * j) & 31]), q = f2_unpack(acc[(i / 2 + 2 * j + 1) & 31]);
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
                    if (live && n + i + 16 <= c.N) {
                        store_32(y + i, u);
                    } else if (live) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (n + i + j < c.N) y[i + j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
                    }
                }
            } else {
                // rows at odd addresses: a warp's results turned in shared memory, 8 x 32 at a time, so that its lanes store
                // neighbouring columns (each its own row's: 32 memory sectors a store instead of two or three)
                uint16_t* const mine = turn + warp * 8 * 34;
                const bool bf16 = c.dtype == NQ_BF16;
                const int row0 = tile.row0 + first + 32 * quarter, rows_here = ok ? min(32, tile.rows - first - 32 * quarter) : 0;
#pragma unroll
                for (int i = 0; i < kMine; i += 32)
                    for (int r0 = 0; r0 < 32; r0 += 8) {
                        if ((lane & 24) == r0)
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float2 p = f2_unpack(acc[i / 2 + j]);
                                *reinterpret_cast<uint32_t*>(mine + (lane & 7) * 34 + 2 * j) = pack_16(p.x, p.y, bf16);
                            }
                        __syncwarp();
                        if (n + i + lane < c.N)
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                if (r < rows_here - r0)
                                    reinterpret_cast<uint16_t*>(c.y)[(long long)(row0 + r0 + r) * c.y_stride + n + i + lane] = mine[r * 34 + lane];
                        __syncwarp();
                    }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();      // nothing arrives on, or multiplies in, a block that has left
    if (warp == 0) {
        tc_fence_after();
        f8_dealloc<PAIR>(tmem);
    }
}

// ---------------------------------------------------------------- few rows a group

template <int BN, bool GLU>
struct Fp8ColsGeo {
    static constexpr int kParts = GLU ? 2 : 1;
    static constexpr int kStageBytes = kParts * kF8Tile * kF8Row + BN * kF8Row;
    // Blocks of K of a hand-over from the tensor cores to the epilogue, which costs it about 400 cycles whatever it is of;
    // at most half of TMEM, so that the next is computed meanwhile.
    static constexpr int kStep = 256 / (BN * kParts) < 4 ? 256 / (BN * kParts) : 4;
    static constexpr int kBufCols = kStep * kParts * BN;
    static constexpr int kBufs = 512 / kBufCols < 4 ? 512 / kBufCols : 4;
    static constexpr int kScaleBytes = f8_scale_bytes(BN, kParts);
    static constexpr int kCtrlBytes = 640 + 2048;   // barriers, flags; the warps' largest values [4][128]
    static constexpr int kRoom = (kSmemLimit - 1024 - kScaleBytes - kCtrlBytes - f8_group_bytes(kMostExperts)) / kStageBytes;
    static constexpr int kStages = kRoom < kF8MaxStages ? kRoom : kF8MaxStages;
    static_assert(kParts * BN * kF8Tile * 4 <= kStages * kStageBytes, "room for a tile's partial sums in the ring");
    static int smem(int E) { return 1024 + kStages * kStageBytes + kScaleBytes + kCtrlBytes + f8_group_bytes(E); }
};

// split > 1: a cluster of so many blocks takes a tile, each a part of K; their sums are added on chip, in the blocks' order.
// Such a launch has a cluster for every tile.
template <int BN, bool GLU>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_cols_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8ColsGeo<BN, GLU>;
    constexpr int kStages = Geo::kStages, kParts = Geo::kParts, kBufs = Geo::kBufs, kStep = Geo::kStep;
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
    const int split = c.split, rank = split > 1 ? (int)cluster_rank() : 0;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(tfull0 + 8 * i, 1);
            mbar_init(tempty0 + 8 * i, kF8Epilogue);
        }
        for (int i = 0; i < kF8ScaleSteps; ++i) {
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
    const int cols = (c.N + kF8Tile - 1) / kF8Tile, blocks = (c.K + kFp8Block - 1) / kFp8Block;
    // this block's part of K
    const int k0 = split > 1 ? (int)((long long)blocks * rank / split) : 0;
    const int KB = (split > 1 ? (int)((long long)blocks * (rank + 1) / split) : blocks) - k0;
    const int total = fp8_groups(c, groups, BN, cols, sums);
    const int t0 = split > 1 ? blockIdx.x / split : blockIdx.x, dt = split > 1 ? gridDim.x / split : gridDim.x;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];

    // (each branch begins with its own count of registers: where the paths met again, everything would have to fit the smaller)
    if (warp >= kF8Epilogue) {
        regs_fewer<kF8OtherRegs>();
        if (warp == kF8Producer) {
            // -------------------------------------------------------- copies
            F8Ring<kStages> in;
            int seq = 0, e = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += dt) {
                const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
                e = tile.e;
                int at[4];
                const int fours = f8_gather_rows(c, tile, 0, BN, at);
                for (int kb = 0; kb < KB; ++kb, ++seq) {
                    const int k = (k0 + kb) * kFp8Block;
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * in.at, in.parity ^ 1, flags, err, wait_ns));
                    if (!ok) break;
                    const uint32_t wa = smem_u32(ring) + in.at * Geo::kStageBytes, xa = wa + kParts * kF8Tile * kF8Row, bar = full0 + 8 * in.at;
                    in.next();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, (uint32_t)(kParts * kF8Tile * kF8Row + (c.rows ? fours * 4 : BN) * kF8Row));
#pragma unroll
                        for (int g = 0; g < kParts; ++g)
                            tma_load_3d(wa + g * kF8Tile * kF8Row, &a.wmap[g], k, tile.col * kF8Tile, tile.e, bar);
                        if (!c.rows) tma_load_2d(xa, &a.xmap, k, tile.row0, bar);
                    }
                    __syncwarp();
                    if (lane < fours) tma_gather4(xa + 4 * lane * kF8Row, &a.xmap, k, at, bar);
                }
            }
            if (!ok)
                for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)
                    mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
        } else if (warp == kF8Mma) {
            // -------------------------------------------------------- MMA issuer (one thread: see fp8_rows_kernel)
            if (elect_one()) {
                F8Ring<kStages> in;
                F8Ring<kBufs> out;
                int e = 0;
                bool ok = true;
                const uint32_t w0 = f8_desc(smem_u32(ring));
                for (int t = t0; t < total && ok; t += dt) {
                    const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
                    e = tile.e;
                    const uint32_t idesc = f8_idesc(kF8Tile, (tile.rows + 15) / 16 * 16);
                    for (int kb = 0; kb < KB && ok;) {
                        ok = mbar_wait(tempty0 + 8 * out.at, out.parity ^ 1, flags, err, wait_ns);
                        for (int i = 0; i < kStep && kb < KB && ok; ++i, ++kb) {
                            ok = mbar_wait(full0 + 8 * in.at, in.parity, flags, err, wait_ns);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t w = w0 + in.at * (Geo::kStageBytes / 16), x = w + kParts * kF8Tile * kF8Row / 16;
                            const uint32_t d = tmem + out.at * Geo::kBufCols + i * kParts * BN;
#pragma unroll
                            for (int g = 0; g < kParts; ++g) f8_mma_block(d + g * BN, w + g * kF8Tile * kF8Row / 16, x, idesc);
                            f8_commit(empty0 + 8 * in.at);
                            in.next();
                        }
                        if (ok) f8_commit(tfull0 + 8 * out.at);
                        out.next();
                    }
                }
                f8_commit(done);
                mbar_wait_drain(done, 0, kDrainNs);
            }
            __syncwarp();
        } else if (warp == kF8Scales) {
            f8_scales<BN, kParts>(c, groups, t0, dt, total, BN, 0, cols, true, scales, sfull0, sempty0, flags, k0, KB,
                                  [&](const Fp8Tile& tile, int g) { return c.ws[g] + tile.e * c.ws_expert[g] + tile.col * c.ws_row[g]; });
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread: a column of the result (a row of the weight) for half of the tile's rows.
        regs_more<kF8EpilogueRegs>();
        constexpr int kMine = BN / 2, kChunk = kMine < 32 ? kMine : 32;
        constexpr int kAtOnce = 64 / kChunk < kStep ? 64 / kChunk : kStep;   // blocks of K whose chunk is loaded before one wait
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16) + half * kMine;
        int step = 0, sstep = 0, e = 0;
        bool ok = true;
        for (int t = t0; t < total; t += dt) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            uint64_t acc[kParts][kMine / 2];
#pragma unroll
            for (int g = 0; g < kParts; ++g)
#pragma unroll
                for (int i = 0; i < kMine / 2; ++i) acc[g][i] = 0;
            const bool any = half * kMine < tile.rows;
            for (int kb = 0; kb < KB; kb += kStep, ++step) {
                const int buf = step % kBufs, slot = sstep % kF8ScaleSteps, block = kb % kF8ScaleBlocks;
                if (block == 0) ok = mbar_wait(sfull0 + 8 * slot, (sstep / kF8ScaleSteps) & 1, flags, err, wait_ns);
                ok = mbar_wait(tfull0 + 8 * buf, (step / kBufs) & 1, flags, err, wait_ns);
                tc_fence_after();
                if (any) {
                    // (of blocks past the last, sums and scales of an earlier step: not added)
                    const int here = min(kStep, KB - kb);
                    const float* const s = scales + (slot * kF8ScaleBlocks + block) * kParts * BN + half * kMine;
#pragma unroll
                    for (int i0 = 0; i0 < kStep; i0 += kAtOnce)
#pragma unroll
                        for (int g = 0; g < kParts; ++g)
#pragma unroll
                            for (int i = 0; i < kMine; i += kChunk) {
                                uint32_t v[kAtOnce][kChunk];
#pragma unroll
                                for (int q = 0; q < kAtOnce; ++q)
                                    f8_ld<kChunk>(lane_base + buf * Geo::kBufCols + ((i0 + q) * kParts + g) * BN + i, v[q]);
#pragma unroll
                                for (int q = 0; q < kAtOnce; ++q) f8_wait_ld<kChunk>(v[q]);
#pragma unroll
                                for (int q = 0; q < kAtOnce; ++q)
                                    if (i0 + q < here)
#pragma unroll
                                        for (int j = 0; j < kChunk; j += 4) {
                                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(s + ((i0 + q) * kParts + g) * BN + i + j);
                                            f2_fma(acc[g][(i + j) / 2], f2_pack(v[q][j], v[q][j + 1]), f.x);
                                            f2_fma(acc[g][(i + j) / 2 + 1], f2_pack(v[q][j + 2], v[q][j + 3]), f.y);
                                        }
                            }
                }
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(tempty0 + 8 * buf, lane == 0);
                if (block + kStep == kF8ScaleBlocks || kb + kStep >= KB) {
                    mbar_arrive_if(sempty0 + 8 * slot, lane == 0);
                    ++sstep;
                }
            }
            if (split > 1) {
                // partial sums [part][row of x][column] into the ring: its last copies have been used
                float* const ex = reinterpret_cast<float*>(ring) + half * kMine * kF8Tile + row;
#pragma unroll
                for (int g = 0; g < kParts; ++g)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        const float2 p = f2_unpack(acc[g][i / 2]);
                        ex[(g * BN + i) * kF8Tile] = i & 1 ? p.y : p.x;
                    }
                break;
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
    if (split > 1) {
        // a warp a row: the blocks' sums of its 128 columns, four a lane
        cluster_sync_all();
        if (t0 < total && !flags[0]) {
            const Fp8Tile tile = fp8_tile(c, groups, t0, 0, BN, cols, true);
            const int n = tile.col * kF8Tile + 4 * lane;
            for (int i = rank * (kF8Threads / 32) + warp; i < tile.rows; i += split * (kF8Threads / 32)) {
                float v[kParts][4] = {};
                for (int q = 0; q < split; ++q)
#pragma unroll
                    for (int g = 0; g < kParts; ++g) {
                        float4 p;
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                                     : "r"(cluster_map(smem_u32(ring) + ((g * BN + i) * kF8Tile + 4 * lane) * 4, q))
                                     : "memory");
                        v[g][0] += p.x;
                        v[g][1] += p.y;
                        v[g][2] += p.z;
                        v[g][3] += p.w;
                    }
                if constexpr (GLU)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[0][j] = silu_mul(v[0][j], v[kParts - 1][j]);
                const long long at = (tile.row0 + i) * c.y_stride + n;
                if (GLU && c.dtype == NQ_E4M3) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = n < c.N ? bits_max(m, v[0][j]) : m;
                    const float s = fp8_scale(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m)));
                    if (lane == 0) c.ys[(tile.row0 + i) * c.ys_stride + tile.col] = s;
                    if (n < c.N)         // (N a multiple of 16)
                        *reinterpret_cast<uint32_t*>(c.y + at) = fp8_codes(v[0][0] / s, v[0][1] / s, v[0][2] / s, v[0][3] / s);
                } else {
                    uint16_t* const y = reinterpret_cast<uint16_t*>(c.y) + at;
                    const bool bf16 = c.dtype == NQ_BF16;
                    const uint32_t lo = pack_16(v[0][0], v[0][1], bf16), hi = pack_16(v[0][2], v[0][3], bf16);
                    if (c.wide && n + 4 <= c.N) {
                        *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
                    } else {
                        if (n < c.N) y[0] = (uint16_t)lo;
                        if (n + 1 < c.N) y[1] = (uint16_t)(lo >> 16);
                        if (n + 2 < c.N) y[2] = (uint16_t)hi;
                        if (n + 3 < c.N) y[3] = (uint16_t)(hi >> 16);
                    }
                }
            }
        }
        cluster_sync_all();                      // no block leaves while another reads its sums
    }
}

}  // namespace nq
