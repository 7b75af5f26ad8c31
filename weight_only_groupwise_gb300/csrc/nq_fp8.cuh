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

constexpr int kF8MaxStages = 16;
constexpr int kF8MostSplit = 8;                  // blocks that share a tile's K: a portable cluster
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
    bool wide;                                   // results' rows aligned to 16 bytes
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
// been done: for one thread. Descriptors as smem_desc_sw128's: `a`, `b` are their low words.
__device__ __forceinline__ uint32_t f8_desc(uint32_t addr) { return (addr & 0x3FFFF) >> 4; }
__device__ __forceinline__ void f8_mma_block(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc) {
    constexpr uint32_t kHigh = (uint32_t)(((uint64_t)(1024 >> 4) << 32 | (1ull << 46) | (2ull << 61)) >> 32);
    asm volatile(
        "{\n\t.reg .b64 x, y;\n\t.reg .pred p;\n\tsetp.ne.b32 p, 0, 0;\n\t"
        "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\tadd.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t"
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t"
        "add.s64 x, x, 2;\n\tadd.s64 y, y, 2;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a), "r"(b), "r"(idesc), "r"(kHigh)
        : "memory");
}
__device__ __forceinline__ void f8_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
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

__device__ __forceinline__ void f8_copy_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Four rows of a 2-D map (box one row high) by their numbers; one outside the tensor reads as zeros.
__device__ __forceinline__ void f8_gather4(uint32_t dst, const CUtensorMap* map, int c0, const int (&r)[4], uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void f8_prefetch(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
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

__device__ __forceinline__ uint32_t pack_16(float lo, float hi, bool bf16) {
    if (bf16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// silu(g) u = g e^g u / (1 + e^g) below zero and g u / (1 + e^-g) above, with the exponential and the quotient of the special
// function unit: a tile's 16384 of them were a sixth of its time (32 blocks of K) with expf and a division. The divisor stays
// between 1 and 2: that quotient is 0 for divisors above 2^126, which 1 + e^-g is for gates below -87.3. The
// exponential's argument is rounded: an error of |g| 2^-23 at most, with two places each of the two functions and a half
// of the sum and of each product. (2048 x 5120 x 17408: 324.8 us, 323.0 with g u / (1 + e^-g) for all; 324.2 with that
// where a thread has no gate below -87.)
__device__ __forceinline__ float f8_silu_mul(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.f + e) * u;
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

// All threads of a block: `sums` has room for a number of each warp. Returns the call's tiles. By expert, waits for the
// preceding kernel, whose offsets they may be; a dense call's threads wait where they first read or write what it may have.
__device__ __forceinline__ int fp8_groups(const Fp8Call& c, const Fp8Groups& g, int high, int cols, int* sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    int total = 0;
    if (!c.offsets) {                            // one group
        total = (c.M + high - 1) / high * cols;
        if (tid == 0) {
            g.before[0] = g.start[0] = 0;
            g.before[1] = total;
            g.end[0] = c.M;
        }
        return total;
    }
    grid_dependency_wait();
    for (int e0 = 0; e0 < c.E; e0 += threads) {
        const int e = e0 + tid;
        int r0 = 0, r1 = 0;
        if (e < c.E) {
            r0 = min(max(__ldg(c.offsets + e), 0), c.M);
            r1 = max(min(__ldg(c.offsets + e + 1), c.M), r0);
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
    int lo = from, hi = g.before[from + 1] > t ? from : c.E - 1;     // the last group with before <= t and tiles
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
    uint32_t i = t - g.before[lo], in_band = n, band = 0;
    if (n > kF8Band) {
        band = i / (uint32_t)(kF8Band * cols);
        in_band = min(kF8Band, n - (int)band * kF8Band);
        i -= band * kF8Band * cols;
    }
    o.col = (int)(in_band == 1 ? i : i / in_band);
    const int r = (int)(band * kF8Band + i - o.col * in_band);
    const int each = even && n > 1 ? ((r1 - r0 + n - 1) / n + 15) / 16 * 16 : high;
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

// The scales' warp: for each row of a tile and each block of K the product of the row's scale and the weight block's, for
// PARTS weight blocks, four blocks of K a step, into a ring [step][block][part][ROWS]. KB blocks of K from k0 on; tiles
// t0, t0 + dt, ... wscale(tile, part): the weight's scales along K.
constexpr int kF8ScaleBlocks = 4, kF8ScaleSteps = 2;
constexpr int f8_scale_bytes(int rows, int parts) { return kF8ScaleSteps * kF8ScaleBlocks * parts * rows * 4; }
template <int ROWS, int PARTS, typename W>
__device__ __forceinline__ void f8_scales(const Fp8Call& c, const Fp8Groups& groups, int t0, int dt, int total, int cols, bool even,
                                          float* scales, uint32_t sfull0, uint32_t sempty0,
                                          volatile int* flags, int k0, int KB, W wscale) {
    constexpr int kPer = (ROWS + 31) / 32;
    const int lane = threadIdx.x & 31;
    int step = 0, e = 0;
    bool ok = true;
    grid_dependency_wait();
    for (int t = t0; t < total && ok; t += dt) {
        const Fp8Tile tile = fp8_tile(c, groups, t, e, ROWS, cols, even);
        e = tile.e;
        const float* sp[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = 32 * i + lane;
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

// Roles: 16 epilogue warps, a producer, an MMA issuer, a warp for the scales. A tile is 128 rows by 256 columns of D.
// Bound by the power limit: 4096 x 5120 x 17408 takes 308 us at first and 334 in a loop of seconds (2.19 PFLOP/s,
// 1890 MHz of 2070, 1360 W), where the copies and products alone, with almost no epilogue, take 249 and 282. What was
// tried: 8 epilogue warps of 128 sums a thread 320 us, without registers handed to them 751 (spills); sums two at a time
// (fma.rn.f32x2) 307, its operands' pairing costs the moves that it saves; loads from TMEM issued during the sums 311; pairs
// of blocks sharing a tile of 256 rows (cta_group::2) 334 to 359, with half of the copies.
//
// BULK, for short sums (K), of which a tile's 64 KB of results are a large part: results go to shared memory and from
// there by bulk copies, a row each, while the next tile's sums are added. That takes the room of a stage.
template <bool GLU, bool BULK>
struct Fp8RowsGeo {
    static_assert(!(GLU && BULK), "of SwiGLU results there is half as much");
    static constexpr int kOut = GLU ? 128 : 256; // columns of the result in a tile; D has 256: those, or gate and up
    static constexpr int kStageBytes = (kF8Tile + 256) * kF8Row;
    static constexpr int kStages = BULK ? 3 : 4;
    static constexpr int kWarps = 16;            // of the epilogue
    static constexpr int kThreads = (kWarps + 4) * 32;
    static constexpr int kRegs = 104, kOtherRegs = 64;           // a block begins with 96 a thread
    static_assert(kWarps * 32 * kRegs + 4 * 32 * kOtherRegs == kThreads * 96, "registers of a block");
    static constexpr int kScaleBytes = f8_scale_bytes(kF8Tile, 2);
    // bytes of a row of results in shared memory, 16 x odd, so that lanes meet no bank twice: a tile's 256 columns, or the 64
    // (GLU: 32) of a warp, 8 rows at a time
    static constexpr int kPitch = BULK ? 528 : 144;
    static constexpr int kTurnBytes = BULK ? kF8Tile * kPitch : kWarps * 8 * kPitch;
    static constexpr int kCtrlBytes = 512 + kScaleBytes + kTurnBytes;
    static_assert(kTurnBytes >= 4 * kF8Tile * 4, "room for the rows' largest values");
    static int smem(int E) { return 1024 + kStages * kStageBytes + kCtrlBytes + f8_group_bytes(E); }
};

template <bool GLU, bool BULK>
__global__ void __launch_bounds__(Fp8RowsGeo<GLU, BULK>::kThreads, 1) fp8_rows_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8RowsGeo<GLU, BULK>;
    constexpr int kStages = Geo::kStages, kWarps = Geo::kWarps;
    constexpr int kProducer = kWarps, kMma = kWarps + 1, kScales = kWarps + 2;
    const Fp8Call& c = a.c;
    extern __shared__ uint8_t f8_smem[];
    uint8_t* const ring = f8_smem + ((1024u - (smem_u32(f8_smem) & 1023u)) & 1023u);
    uint8_t* const ctrl = ring + kStages * Geo::kStageBytes;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl);
    // bars: full[8], empty[8], tfull[2], tempty[2], sfull[2], sempty[2], done
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 64, tfull0 = empty0 + 64, tempty0 = tfull0 + 16;
    const uint32_t sfull0 = tempty0 + 16, sempty0 = sfull0 + 16, done = sempty0 + 16;
    volatile int* const flags = reinterpret_cast<volatile int*>(ctrl + 352);     // [0] abort, [3] TMEM base
    int* const sums = reinterpret_cast<int*>(ctrl + 384);
    float* const scales = reinterpret_cast<float*>(ctrl + 512);                  // [steps][blocks][2][128 rows]
    uint8_t* const turn = ctrl + 512 + Geo::kScaleBytes;
    uint32_t* const largest = reinterpret_cast<uint32_t*>(turn);                 // [4 column groups][128 rows]
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
            mbar_init(tempty0 + 8 * i, kWarps);
        }
        for (int i = 0; i < kF8ScaleSteps; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, kWarps);
        }
        mbar_init(done, 1);
        flags[0] = 0;
        mbar_fence_init();
        f8_prefetch(&a.wmap[0]);
        if (GLU) f8_prefetch(&a.wmap[1]);
        f8_prefetch(&a.xmap);
    }
    if (warp == 0) tmem_alloc(smem_u32(const_cast<int*>(flags) + 3), 512);
    // Codes can be the weight of the next call, which reads it ahead of this kernel's end, so that it is not let start early.
    // (It costs 2 us: SwiGLU calls of 16 x 4096 x 4096 behind each other 12.7 us, 10.5 where they start early.)
    if (c.dtype != NQ_E4M3) grid_launch_dependents();
    const int cols = (c.N + Geo::kOut - 1) / Geo::kOut, KB = (c.K + kFp8Block - 1) / kFp8Block;
    const int total = fp8_groups(c, groups, kF8Tile, cols, sums);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];

    // (each branch begins with its own count of registers: where the paths met again, everything would have to fit the smaller)
    if (warp >= kWarps) {
        regs_fewer<Geo::kOtherRegs>();
        if (warp == kProducer) {
            // -------------------------------------------------------- copies
            F8Ring<kStages> in;
            int seq = 0, e = 0;
            bool ok = true;
            const int late = c.offsets ? 0 : min(kStages, KB);
            auto x_late = [&](int n) {           // rows of x of the first n stages, of a dense call's first tile
                const Fp8Tile tile = fp8_tile(c, groups, blockIdx.x, 0, kF8Tile, cols, false);
                grid_dependency_wait();
                for (int j = 0; j < n; ++j)
                    f8_copy_2d(smem_u32(ring) + j * Geo::kStageBytes, &a.xmap, j * kFp8Block, tile.row0, full0 + 8 * j);
            };
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Fp8Tile tile = fp8_tile(c, groups, t, e, kF8Tile, cols, false);
                e = tile.e;
                int at[4];
                const int fours = f8_gather_rows(c, tile, at);
                for (int kb = 0; kb < KB; ++kb, ++seq) {
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(empty0 + 8 * in.at, in.parity ^ 1, flags, err, wait_ns));
                    if (!ok) break;
                    const uint32_t xa = smem_u32(ring) + in.at * Geo::kStageBytes, wa = xa + kF8Tile * kF8Row, bar = full0 + 8 * in.at;
                    const int k = kb * kFp8Block;
                    in.next();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(bar, (uint32_t)((256 + (c.rows ? fours * 4 : kF8Tile)) * kF8Row));
                        tma_load_3d(wa, &a.wmap[0], k, tile.col * Geo::kOut, tile.e, bar);
                        if (GLU) tma_load_3d(wa + 128 * kF8Row, &a.wmap[1], k, tile.col * 128, tile.e, bar);
                        // (the first stages' weights are on their way before the preceding kernel has ended: late)
                        if (seq >= late && !c.rows) f8_copy_2d(xa, &a.xmap, k, tile.row0, bar);
                        if (seq + 1 == late) x_late(late);
                    }
                    __syncwarp();
                    if (lane < fours) f8_gather4(xa + 4 * lane * kF8Row, &a.xmap, k, at, bar);
                }
            }
            if (!ok && lane == 0 && seq < late) x_late(seq);
            __syncwarp();
            // The last copies into each stage: the block must not leave while they are on their way, and any warp may give up
            // waiting for them after this one has asked for them all. (Otherwise they have long been waited for.)
            for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)
                mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
        } else if (warp == kMma) {
            // -------------------------------------------------------- MMA issuer: one thread
            if (elect_one()) {
                F8Ring<kStages> in;
                F8Ring<2> out;
                int e = 0;
                bool ok = true;
                const uint32_t x0 = f8_desc(smem_u32(ring));
                grid_dependency_wait();          // (a wait's time is its own: x's rows are asked for from then on)
                for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                    const Fp8Tile tile = fp8_tile(c, groups, t, e, kF8Tile, cols, false);
                    e = tile.e;
                    const uint32_t idesc = f8_idesc(kF8Tile, GLU ? 256 : min(256, (c.N - tile.col * Geo::kOut + 15) / 16 * 16));
                    for (int kb = 0; kb < KB; ++kb) {
                        ok = mbar_wait(full0 + 8 * in.at, in.parity, flags, err, wait_ns) &&
                             mbar_wait(tempty0 + 8 * out.at, out.parity ^ 1, flags, err, wait_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t x = x0 + in.at * (Geo::kStageBytes / 16);
                        f8_mma_block(tmem + 256 * out.at, x, x + kF8Tile * kF8Row / 16, idesc);
                        f8_commit(tfull0 + 8 * out.at);
                        f8_commit(empty0 + 8 * in.at);
                        in.next();
                        out.next();
                    }
                }
                f8_commit(done);                 // every MMA has completed before TMEM can be freed
                mbar_wait_drain(done, 0, kDrainNs);
            }
            __syncwarp();
        } else if (warp == kScales) {
            // of the two blocks of columns, or of gate and up
            f8_scales<kF8Tile, 2>(c, groups, blockIdx.x, gridDim.x, total, cols, false, scales, sfull0, sempty0, flags, 0, KB,
                                  [&](const Fp8Tile& tile, int g) {
                                      const int nb = GLU ? tile.col : min(2 * tile.col + g, (c.N - 1) / kFp8Block);
                                      return c.ws[GLU ? g : 0] + tile.e * c.ws_expert[GLU ? g : 0] + nb * c.ws_row[GLU ? g : 0];
                                  });
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread: a row and 64 columns of D, two runs of 32 that begin at d0 and d1: neighbours, or gate and up of the same
        // 32 columns of the result.
        regs_more<Geo::kRegs>();
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
        constexpr int kMine = GLU ? 32 : 64;
        const int d0 = kMine * group, d1 = GLU ? 128 + d0 : 32 + d0, part = GLU ? 0 : group >> 1;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        F8Ring<2> in;
        F8Ring<kF8ScaleSteps> sc;
        int e = 0;
        bool ok = true;
        grid_dependency_wait();                  // the results may be in use
        // BULK: eight lanes of a warp have a row each of the finished tile to send. Results leave an SM at some 32 bytes a cycle
        // and hold up the copies' requests behind them, so that they go one by one during the first half of the next tile's
        // blocks of K (24570 rows of 128 experts x 2048, us, at once and so: K = 256 44.2, 45.3; 384 59.9, 51.7; 512 66.1,
        // 59.3; 768 80.2, 74.3; 1536 125.8, 118.4).
        const int my_row = 32 * quarter + 8 * group + lane, due_at = lane * KB / 16;
        uint16_t* due = nullptr;
        int due_bytes = 0;
        auto send = [&] {
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(due), "r"(smem_u32(turn + my_row * Geo::kPitch)),
                         "r"(due_bytes)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            due = nullptr;
        };
        for (int t = blockIdx.x; t < total; t += gridDim.x) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, kF8Tile, cols, false);
            e = tile.e;
            float acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0.f;
            for (int kb = 0; kb < KB; ++kb) {
                const int block = kb % kF8ScaleBlocks;
                if (block == 0) mbar_wait(sfull0 + 8 * sc.at, sc.parity, flags, err, wait_ns);
                const float* const s = scales + (sc.at * kF8ScaleBlocks + block) * 2 * kF8Tile + row;
                const float f0 = s[part * kF8Tile], f1 = GLU ? s[kF8Tile] : f0;
                ok = mbar_wait(tfull0 + 8 * in.at, in.parity, flags, err, wait_ns);
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
                        mbar_arrive_if(tempty0 + 8 * in.at, lane == 0);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[16 * i + j] = fmaf(__uint_as_float(v[j]), i < 2 ? f0 : f1, acc[16 * i + j]);
                }
                if (BULK && due && kb == due_at) send();
                in.next();
                if (block == kF8ScaleBlocks - 1 || kb + 1 == KB) {
                    __syncwarp();
                    mbar_arrive_if(sempty0 + 8 * sc.at, lane == 0);
                    sc.next();
                }
            }
            // the results: 64 columns, or 32 of silu(g) u
            const int n = tile.col * Geo::kOut + d0;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = f8_silu_mul(acc[i], acc[32 + i]);
            }
            if (GLU && c.dtype == NQ_E4M3) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (n + i < c.N) m = bits_max(m, acc[i]);
                largest[group * kF8Tile + row] = m;
                named_bar_sync(1 + quarter, 128);        // the row's four warps
#pragma unroll
                for (int i = 0; i < 4; ++i) m = max(m, largest[i * kF8Tile + row]);
                named_bar_sync(1 + quarter, 128);        // the next tile's use the same place
                const float s = fp8_scale(__uint_as_float(m)), r = 1.f / s;
                if (ok && row < tile.rows) {
                    const long long at = tile.row0 + row;
                    if (group == 0) c.ys[at * c.ys_stride + tile.col] = s;
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        if (n + i >= c.N) break;
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float* const p = acc + i + 4 * j;
                            u[j] = fp8_codes(p[0] * r, p[1] * r, p[2] * r, p[3] * r);
                        }
                        *reinterpret_cast<uint4*>(c.y + at * c.y_stride + n + i) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            } else if (BULK) {
                // (results aligned to 16 bytes, N a multiple of 8)
                const bool bf16 = c.dtype == NQ_BF16;
                uint8_t* const mine = turn + row * Geo::kPitch + 2 * d0;
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                named_bar_sync(1 + quarter, 128);        // the tile before has been read
#pragma unroll
                for (int j = 0; j < kMine; j += 8)
                    *reinterpret_cast<uint4*>(mine + 2 * j) =
                        make_uint4(pack_16(acc[j], acc[j + 1], bf16), pack_16(acc[j + 2], acc[j + 3], bf16),
                                   pack_16(acc[j + 4], acc[j + 5], bf16), pack_16(acc[j + 6], acc[j + 7], bf16));
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                named_bar_sync(1 + quarter, 128);
                const int n1 = tile.col * Geo::kOut;
                if (lane < 8 && ok && my_row < tile.rows)
                    due = reinterpret_cast<uint16_t*>(c.y) + (long long)(tile.row0 + my_row) * c.y_stride + n1;
                due_bytes = 2 * min(Geo::kOut, c.N - n1);
            } else {
                // Turned in shared memory, 8 rows at a time, so that a store writes whole lines (of 4 or 8 rows, or, where rows
                // are not aligned, 64 bytes of one) instead of a sector of each of 32.
                uint8_t* const mine = turn + warp * 8 * Geo::kPitch;
                const bool bf16 = c.dtype == NQ_BF16;
                const int row0 = tile.row0 + 32 * quarter, rows_here = ok ? min(32, tile.rows - 32 * quarter) : 0;
                uint16_t* const y = reinterpret_cast<uint16_t*>(c.y) + n;
                uint32_t u[kMine / 2];
#pragma unroll
                for (int j = 0; j < kMine / 2; ++j) u[j] = pack_16(acc[2 * j], acc[2 * j + 1], bf16);
                constexpr int kLanes = kMine / 8, kRows = 32 / kLanes;   // lanes of a row's 16-byte pieces, rows of a store
                const int piece = lane % kLanes, sub = lane / kLanes;
                const bool whole = c.wide && n + 8 * piece + 8 <= c.N;
                for (int r0 = 0; r0 < rows_here; r0 += 8) {
                    if ((lane & 24) == r0)
#pragma unroll
                        for (int j = 0; j < kLanes; ++j)
                            *reinterpret_cast<uint4*>(mine + (lane & 7) * Geo::kPitch + 16 * j) =
                                make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
                    __syncwarp();
                    if (c.wide) {
#pragma unroll
                        for (int r = 0; r < 8; r += kRows) {
                            const uint4 q = *reinterpret_cast<const uint4*>(mine + (r + sub) * Geo::kPitch + 16 * piece);
                            uint16_t* const to = y + (long long)(row0 + r0 + r + sub) * c.y_stride + 8 * piece;
                            if (r0 + r + sub >= rows_here) continue;
                            if (whole) {
                                *reinterpret_cast<uint4*>(to) = q;
                            } else {
                                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (n + 8 * piece + j < c.N) to[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
                            }
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < 8; ++r)
#pragma unroll
                            for (int i = 0; i < kMine; i += 32)
                                if (r0 + r < rows_here && n + i + lane < c.N)
                                    y[(long long)(row0 + r0 + r) * c.y_stride + i + lane] =
                                        *reinterpret_cast<const uint16_t*>(mine + r * Geo::kPitch + 2 * (i + lane));
                    }
                    __syncwarp();
                }
            }
        }
        if (BULK && due) send();
        if (BULK) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
    // Warps of the epilogue: 16 where a tile has 64 rows or more (256 x 4096 x 5120: 18.8 us with 8, 16.5 so), else 8, which
    // have registers for the loads of more blocks of K at a time.
    static constexpr int kWarps = BN >= 64 ? 16 : 8;
    static constexpr int kThreads = (kWarps + 4) * 32;
    static constexpr int kRegs = kWarps == 16 ? 104 : 216, kOtherRegs = kWarps == 16 ? 64 : 72;
    static_assert(kWarps * 32 * kRegs + 4 * 32 * kOtherRegs == kThreads * (kWarps == 16 ? 96 : 168), "registers of a block");
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
__global__ void __launch_bounds__(Fp8ColsGeo<BN, GLU>::kThreads, 1) fp8_cols_kernel(const __grid_constant__ Fp8Args a) {
    using Geo = Fp8ColsGeo<BN, GLU>;
    constexpr int kStages = Geo::kStages, kParts = Geo::kParts, kBufs = Geo::kBufs, kStep = Geo::kStep, kWarps = Geo::kWarps;
    constexpr int kProducer = kWarps, kMma = kWarps + 1, kScales = kWarps + 2;
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
            mbar_init(tempty0 + 8 * i, kWarps);
        }
        for (int i = 0; i < kF8ScaleSteps; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(sempty0 + 8 * i, kWarps);
        }
        mbar_init(done, 1);
        flags[0] = 0;
        mbar_fence_init();
        f8_prefetch(&a.wmap[0]);
        if (GLU) f8_prefetch(&a.wmap[1]);
        f8_prefetch(&a.xmap);
    }
    if (warp == 0) tmem_alloc(smem_u32(const_cast<int*>(flags) + 3), 512);
    if (c.dtype != NQ_E4M3) grid_launch_dependents();   // (as in fp8_rows_kernel)
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
    if (warp >= kWarps) {
        regs_fewer<Geo::kOtherRegs>();
        if (warp == kProducer) {
            // -------------------------------------------------------- copies
            F8Ring<kStages> in;
            int seq = 0, e = 0;
            bool ok = true;
            const int late = c.offsets ? 0 : min(kStages, KB);   // (as in fp8_rows_kernel)
            auto x_late = [&](int n) {
                const Fp8Tile tile = fp8_tile(c, groups, t0, 0, BN, cols, true);
                grid_dependency_wait();
                for (int j = 0; j < n; ++j)
                    f8_copy_2d(smem_u32(ring) + j * Geo::kStageBytes + kParts * kF8Tile * kF8Row, &a.xmap, (k0 + j) * kFp8Block,
                               tile.row0, full0 + 8 * j);
            };
            for (int t = t0; t < total && ok; t += dt) {
                const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
                e = tile.e;
                int at[4];
                const int fours = f8_gather_rows(c, tile, at);
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
                        if (seq >= late && !c.rows) f8_copy_2d(xa, &a.xmap, k, tile.row0, bar);
                        if (seq + 1 == late) x_late(late);
                    }
                    __syncwarp();
                    if (lane < fours) f8_gather4(xa + 4 * lane * kF8Row, &a.xmap, k, at, bar);
                }
            }
            if (!ok && lane == 0 && seq < late) x_late(seq);
            __syncwarp();
            for (int j = seq > kStages ? seq - kStages : 0; j < seq; ++j)   // (as in fp8_rows_kernel)
                mbar_wait_drain(full0 + 8 * (j % kStages), (j / kStages) & 1, kDrainNs);
        } else if (warp == kMma) {
            // -------------------------------------------------------- MMA issuer (one thread: see fp8_rows_kernel)
            if (elect_one()) {
                F8Ring<kStages> in;
                F8Ring<kBufs> out;
                int e = 0;
                bool ok = true;
                const uint32_t w0 = f8_desc(smem_u32(ring));
                grid_dependency_wait();          // (as in fp8_rows_kernel)
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
        } else if (warp == kScales) {
            f8_scales<BN, kParts>(c, groups, t0, dt, total, cols, true, scales, sfull0, sempty0, flags, k0, KB,
                                  [&](const Fp8Tile& tile, int g) { return c.ws[g] + tile.e * c.ws_expert[g] + tile.col * c.ws_row[g]; });
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Thread: a column of the result (a row of the weight) for a part of the tile's rows.
        regs_more<Geo::kRegs>();
        constexpr int kMine = BN / (kWarps / 4), kChunk = kMine < 32 ? kMine : 32;
        // blocks of K whose chunk is loaded before one wait, as far as registers go
        constexpr int kRoom = (kWarps == 16 ? 32 : 64) / kChunk, kAtOnce = kRoom < kStep ? kRoom : kStep;
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16) + group * kMine;
        int step = 0, sstep = 0, e = 0;
        bool ok = true;
        grid_dependency_wait();                  // the results may be in use
        for (int t = t0; t < total; t += dt) {
            const Fp8Tile tile = fp8_tile(c, groups, t, e, BN, cols, true);
            e = tile.e;
            float acc[kParts][kMine];
#pragma unroll
            for (int g = 0; g < kParts; ++g)
#pragma unroll
                for (int i = 0; i < kMine; ++i) acc[g][i] = 0.f;
            const bool any = group * kMine < tile.rows;
            for (int kb = 0; kb < KB; kb += kStep, ++step) {
                const int buf = step % kBufs, slot = sstep % kF8ScaleSteps, block = kb % kF8ScaleBlocks;
                if (block == 0) ok = mbar_wait(sfull0 + 8 * slot, (sstep / kF8ScaleSteps) & 1, flags, err, wait_ns);
                ok = mbar_wait(tfull0 + 8 * buf, (step / kBufs) & 1, flags, err, wait_ns);
                tc_fence_after();
                if (any) {
                    // (of blocks past the last, sums and scales of an earlier step: not added)
                    const int here = min(kStep, KB - kb);
                    const float* const s = scales + (slot * kF8ScaleBlocks + block) * kParts * BN + group * kMine;
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
                                            const float4 f = *reinterpret_cast<const float4*>(s + ((i0 + q) * kParts + g) * BN + i + j);
                                            float* const to = acc[g] + i + j;
                                            to[0] = fmaf(__uint_as_float(v[q][j]), f.x, to[0]);
                                            to[1] = fmaf(__uint_as_float(v[q][j + 1]), f.y, to[1]);
                                            to[2] = fmaf(__uint_as_float(v[q][j + 2]), f.z, to[2]);
                                            to[3] = fmaf(__uint_as_float(v[q][j + 3]), f.w, to[3]);
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
                float* const ex = reinterpret_cast<float*>(ring) + group * kMine * kF8Tile + row;
#pragma unroll
                for (int g = 0; g < kParts; ++g)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) ex[(g * BN + i) * kF8Tile] = acc[g][i];
                break;
            }
            const int n = tile.col * kF8Tile + row;
            const int rows_here = ok ? min(kMine, tile.rows - group * kMine) : 0;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < kMine; ++i) acc[0][i] = f8_silu_mul(acc[0][i], acc[1][i]);
            }
            const long long first = tile.row0 + group * kMine;
            if (GLU && c.dtype == NQ_E4M3) {
                // a row's largest over the tile's 128 columns: the warp's, then the four warps' with these rows
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, n < c.N ? bits_max(0, acc[0][i]) : 0u);
                    if (lane == 0) largest[quarter * BN + group * kMine + i] = m;
                }
                named_bar_sync(1 + group, 128);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    if (i < rows_here) {
                        uint32_t m = 0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) m = max(m, largest[q * BN + group * kMine + i]);
                        const float s = fp8_scale(__uint_as_float(m)), r = 1.f / s;
                        if (row == 0) c.ys[(first + i) * c.ys_stride + tile.col] = s;
                        if (n < c.N) c.y[(first + i) * c.y_stride + n] = (uint8_t)fp8_codes(acc[0][i] * r, 0.f, 0.f, 0.f);
                    }
                }
                named_bar_sync(1 + group, 128);  // the next tile's largest use the same place
            } else if (n < c.N) {
                uint16_t* const y = reinterpret_cast<uint16_t*>(c.y) + first * c.y_stride + n;
                const bool bf16 = c.dtype == NQ_BF16;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i < rows_here) y[i * c.y_stride] = (uint16_t)pack_16(acc[0][i], 0.f, bf16);
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
        grid_dependency_wait();
        cluster_sync_all();
        if (t0 < total && !flags[0]) {
            const Fp8Tile tile = fp8_tile(c, groups, t0, 0, BN, cols, true);
            const int n = tile.col * kF8Tile + 4 * lane;
            for (int i = rank * (Geo::kThreads / 32) + warp; i < tile.rows; i += split * (Geo::kThreads / 32)) {
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
                    for (int j = 0; j < 4; ++j) v[0][j] = f8_silu_mul(v[0][j], v[kParts - 1][j]);
                const long long at = (tile.row0 + i) * c.y_stride + n;
                if (GLU && c.dtype == NQ_E4M3) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) m = n < c.N ? bits_max(m, v[0][j]) : m;
                    const float s = fp8_scale(__uint_as_float(__reduce_max_sync(0xFFFFFFFFu, m))), r = 1.f / s;
                    if (lane == 0) c.ys[(tile.row0 + i) * c.ys_stride + tile.col] = s;
                    if (n < c.N)         // (N a multiple of 16)
                        *reinterpret_cast<uint32_t*>(c.y + at) = fp8_codes(v[0][0] * r, v[0][1] * r, v[0][2] * r, v[0][3] * r);
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
