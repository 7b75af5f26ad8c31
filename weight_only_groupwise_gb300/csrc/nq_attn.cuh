// nq_attn.cuh -- attention of a chunk of new tokens over a paged KV cache (nq_attn_paged):
//
//   O[t, h] = sum_j softmax_j(scale q[t, h] . K[j, h / G]) V[j, h / G]
//
// over the keys j that token t sees: with p its position, 0 <= j <= p and, with a window W,
// j > p - W or j < sinks. One pass over the keys with the running maximum and sum of the
// softmax, on the fifth-generation tensor cores.
//
// Tiles. A query tile is the G query heads of floor(128 / G) tokens of one (request, KV head), up
// to 128 rows: row i is token i / G, head i % G, so the heads share every key that is loaded,
// whatever the number of new tokens (one, a verify round's 8, a prompt chunk's thousands), and
// a tile is one box of q as [token][head][dim]. A key tile is 128 keys, cut at
// multiples of 128, so a page (16..256 keys) never straddles two tiles unless it holds both.
// Keys that no row of the query tile sees are not loaded, tile by tile.
//
// Work split. KV heads are handled in gangs of blocks, a head a block (the largest divisor of the
// heads that leaves at most 1/16 of the SMs without work), so that the rows of a page, which hold
// all heads, are read from memory at about the same time. The (query tile, key tile) pairs of the
// whole call, in the order request, gang of heads, query tile, key tile, are cut into one equal
// range per gang (stream-K): ragged lengths and few rows need no other rule. A boundary within
// kAttnSnap units of a query tile's begin or end moves there, where a range is long enough to
// take it, and one inside a tile of up to kAttnWhole units always: a split costs about as much as so
// many units (partials written, joined). Where no tile can be longer the join is not launched. A
// query tile whose keys are spread over several blocks is written as fp32 partials with their
// maxima and sums; attn_join_kernel adds them in block order, so the result does not depend on
// timing. Every block finds its range by itself from the lengths on the device: no host copy of the
// lengths, no plan to keep, no waits between blocks.
//
// Pairs. For prompts of 256 columns (attn_uses_pairs) two blocks of a cluster take a query tile of 256
// rows: each its 128 rows of Q, S, P and O, half of the keys of a K tile, half of the columns of a
// V tile, and the even block issues the products for both (cta_group::2). That halves the copies
// and the reads of K and V from shared memory, which alone take a block longer than its products
// (320 KB a key tile at 128 bytes a cycle: 2560 cycles, against 2048).
//
// Roles of a block's 12 warps (one block per SM):
//   * warps 0..7 -- softmax: thread = row (TMEM lane) and half of the tile's 128 columns. The two
//     halves of a row exchange maxima through shared memory. The accumulator is rescaled only
//     when a row's maximum grows by more than 2^8 in the exponential's argument (p <= 256 stays
//     exact enough in 16 bits, the sum is fp32); p is rounded to the 16-bit type of the cache
//     for the second product, which takes 16-bit operands: against 64 bits O is off by 0.0021 (bf16, relative) where
//     probabilities of 32 bits and the output's rounding alone leave 0.0017, 0.00027 and 0.00021 in fp16. (Alternate
//     tiles for the two groups of four warps, each with an accumulator of its own, were slower: 267
//     us against 253 for 64 one-token requests of 128 columns.)
//   * warps 8 and 11 -- producers of K and of V: TMA copies of pages (a 4-D map of the cache: dim,
//     row, head, block) into a ring of shared-memory slots, 128-byte swizzled, in the order the MMA
//     warp consumes them: K 0, K 1, V 0, K 2, V 1, ... The page ids are the map's last coordinate:
//     an id outside the cache reads as zeros instead of faulting, and no offset is formed in 32 bits.
//     Two warps, because a page of 16 keys makes copies of 2 KB, whose issue was the limit.
//   * warp 9 -- MMA issuer: S = Q K^T (both from shared memory), O += P V (P from TMEM, V from
//     shared memory as the N-major operand). S is double buffered: the product of tile j + 1 is
//     issued before that of P of tile j, so that the tensor cores work during the softmax.
//   * warp 10 -- the query tile into shared memory, one TMA box a 64-column panel (small boxes where
//     they are enough: a box of 128 rows costs a one-token call 1.5 us). Rows past the tile's own
//     (other requests' tokens, zeros, leftovers) are computed and dropped.
// TMEM: O in columns 0..dim-1, the S buffers (P over them) in columns 256.. and 384...
//
// Rows of V that no row of the tile sees (past the last key, before a window) may hold anything,
// NaN included, and 0 x NaN would reach the sum. Whole pages of them are never read: their id becomes
// -1, which loads as zeros. The others' rows the softmax warps zero in shared memory (all of them
// zeroed there: 46.5 -> 48.4 us for 3 windowed requests, 219 -> 234 for 4096 tokens from scratch).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "nq_common.cuh"
#include "nq_step.h"
#include "nq_tc.cuh"

namespace nq {

constexpr int kAttnKeys = 128;                    // keys of a tile
constexpr int kAttnThreads = 12 * 32;
constexpr int kAttnSoftmaxWarps = 8;
constexpr int kAttnProducerK = 8, kAttnMma = 9, kAttnLoader = 10, kAttnProducerV = 11;
constexpr int kAttnMaxRequests = 8192;            // the scan's 8 bytes a request fit the tile buffers
constexpr int kAttnSCol = 256;                    // TMEM column of the first S buffer
constexpr int kAttnMaxSlots = 8;
constexpr int kAttnCtrlBytes = 3072;
constexpr int kAttnSnap = 6;                      // units by which a range may grow or shrink to avoid a split
constexpr int kAttnWhole = 4;                     // a query tile of up to so many units is never split
constexpr float kAttnLazy = 8.f;                  // log2 of the growth that forces a rescale
// fp16 probabilities are stored times 2^7 (sums too, so that it cancels): at most 2^15, and keys count down to 2^-32
// of the largest instead of 2^-25, of which 2^18 keys have 0.8 % of the sum.
constexpr float kAttnLift = 7.f;

// Shared-memory geometry for a head dimension: the K slot holds 128 keys x min(D, 128) columns,
// the V slot as many bytes: 128 keys x D, or 64 keys x 256. (Slots of 16 KB, twice as many barrier
// steps a tile, were slower: 635 us against 600 for a 2048-token chunk of 256 columns.)
template <int D, bool PAIR = false>
struct AttnGeo {
    static constexpr int kDK = PAIR || D < 128 ? D : 128;    // columns of a K slot
    static constexpr int kKKeys = PAIR ? 64 : 128;           // keys of a K slot
    static constexpr int kKSlots = D / kDK;                  // K slots of a key tile
    static constexpr int kDV = PAIR ? D / 2 : D;             // columns of a V slot
    static constexpr int kVKeys = D == 256 && !PAIR ? 64 : 128;  // keys of a V slot
    static constexpr int kVSlots = kAttnKeys / kVKeys;
    static constexpr int kSlotBytes = kKKeys * kDK * 2;
    static constexpr int kQBytes = kAttnRows * D * 2;
    static constexpr int kSlots = D == 256 ? 5 : (D == 128 ? 6 : 8);
    static constexpr int kSmem = kQBytes + kSlots * kSlotBytes + kAttnCtrlBytes;
    static_assert(kSmem <= kSmemLimit && kSlots <= kAttnMaxSlots, "shared memory");
    static_assert(kVKeys * kDV * 2 == kSlotBytes, "one slot size");
    static_assert(kQBytes + kSlots * kSlotBytes >= kAttnMaxRequests * 8, "room for the scan");
};

struct AttnArgs {
    CUtensorMap qmap, kmap, vmap;      // qmap: {dim, query heads, tokens}, boxes of 64 x group x tile_tokens
    CUtensorMap qfew;                  // the same with boxes of few_tokens
    uint16_t* out;
    long long out_stride;              // between tokens, elements
    bool wide;                         // whether out's rows are aligned to 32 bytes
    const int* table;
    long long table_stride;
    const int* q_start;
    const int* kv_lens;
    int R, tokens, heads, group;       // heads: KV heads; group: query heads per KV head
    int gang;                          // blocks (pairs) that take the heads of a range together
    int gangs, turns;                  // gangs of the launch; times that a gang goes through the heads
    int tile_tokens;                   // tokens of a query tile: a block's, or two blocks' of a pair
    int block_tokens;                  // tokens of a block: 128 / group
    int stride;                        // blocks from a split's part to the next: gang, times two for pairs
    int few_tokens;                    // tokens of a small box: the fewest whose rows are a multiple of 8
    int page_shift, max_keys;
    int window, sinks;                 // window 0: none, and then no sinks
    float scale_log2;                  // scale x log2(e)
    float* part;                       // [2 blocks][D][128 rows] partial accumulators
    float2* ml;                        // [2 blocks][128] (maximum, sum)
    int4* splits;                      // [blocks][2]: request, head, first token, rows; parts
    int* dev_err;
    unsigned long long wait_ns;
};

// ---------------------------------------------------------------- the work

struct AttnReq {
    int q0, n, kv;                     // first token, new tokens, keys
};

__device__ __forceinline__ AttnReq attn_req(const AttnArgs& a, int b, int e, int kv) {
    AttnReq q;
    q.q0 = min(max(b, 0), a.tokens);
    q.n = min(max(e, q.q0), a.tokens) - q.q0;
    q.kv = min(max(kv, 0), a.max_keys);
    return q;
}
__device__ __forceinline__ AttnReq attn_req(const AttnArgs& a, int r) {
    return attn_req(a, a.q_start[r], a.q_start[r + 1], a.kv_lens[r]);
}

// x / y for non-negative x and positive y, in 32 bits where they fit.
__device__ __forceinline__ long long attn_div(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// A query tile: its tokens, and the key tiles it reads, kt(i) = i < first ? i : i + skip.
struct AttnTile {
    int token0, rows;                  // first token in the request, rows (tokens x group)
    int pf, pl;                        // positions of the first and the last token
    int hi, lo;                        // keys seen by some row: [lo, hi) and the sinks
    int n, first, skip;
};

__device__ __forceinline__ int attn_tiles(const AttnArgs& a, const AttnReq& q) {
    return q.n <= a.tile_tokens ? min(q.n, 1) : (q.n + a.tile_tokens - 1) / a.tile_tokens;
}

__device__ __forceinline__ AttnTile attn_tile(const AttnArgs& a, const AttnReq& q, int qt) {
    AttnTile t;
    t.token0 = qt * a.tile_tokens;
    const int tokens = min(a.tile_tokens, q.n - t.token0);
    t.rows = tokens * a.group;
    t.pf = q.kv - q.n + t.token0;
    t.pl = t.pf + tokens - 1;
    t.hi = max(0, t.pl + 1);
    t.lo = a.window > 0 ? min(max(0, t.pf - a.window + 1), t.hi) : 0;
    const int se = min(a.sinks, t.hi);
    const int ns = (se + kAttnKeys - 1) / kAttnKeys, lt = t.lo / kAttnKeys, ht = (t.hi + kAttnKeys - 1) / kAttnKeys;
    // the sinks' tiles and the window's, one range if they meet
    t.first = se > 0 && ns < lt ? ns : 0;
    t.skip = se == 0 || ns < lt ? lt - t.first : 0;
    t.n = ht - t.skip;
    return t;
}

// Units of a query tile (0 past the last).
__device__ __forceinline__ int attn_tile_units(const AttnArgs& a, const AttnReq& q, int qt, int nqt) {
    return qt < nqt ? max(1, attn_tile(a, q, qt).n) : 0;
}

// A block's walk over its range of units: segments of query tiles. A tile that sees no key
// counts one unit (its rows are zeros).
struct AttnWalk {
    long long left, at;                // units left, global index of the next one
    AttnReq rq;
    AttnTile t;
    int me;                            // the block, or the pair of blocks
    int r, h, qt, nqt;
    int k0, k1, units;                 // the segment: units k0..k1 of the tile's `units`
    int next_b, next_e, next_kv;       // request r + 1 as it lies in memory, fetched ahead
    __device__ __forceinline__ void fetch(const AttnArgs& a) {
        if (r + 1 < a.R) {
            next_b = __ldg(a.q_start + r + 1);
            next_e = __ldg(a.q_start + r + 2);
            next_kv = __ldg(a.kv_lens + r + 1);
        }
    }
    // The next request.
    __device__ __forceinline__ void enter(const AttnArgs& a) {
        ++r;
        rq = attn_req(a, next_b, next_e, next_kv);
        nqt = attn_tiles(a, rq);
        fetch(a);
    }
    __device__ __forceinline__ void cut(int from) {
        units = max(1, t.n);
        k0 = from;
        k1 = (int)min((long long)units, from + left);
    }
    // Finds unit u: of request r_, whose units are base..base + all - 1. Whole warps call this: the
    // lanes look for the query tile together. Returns the unit's place in its tile.
    __device__ __forceinline__ int find(const AttnArgs& a, int r_, const AttnReq& rq_, long long base, long long all,
                                        long long u) {
        r = r_;
        rq = rq_;
        nqt = attn_tiles(a, rq);
        const long long per = a.turns == 1 ? all : attn_div(all, a.turns);
        const int turn = a.turns == 1 ? 0 : (int)attn_div(u - base, per);
        h = turn * a.gang + me % a.gang;
        long long rem = (u - base) - turn * per;
        const int lane = threadIdx.x & 31;
        for (qt = 0; nqt > 1; qt += 32) {
            const int n_ = attn_tile_units(a, rq, qt + lane, nqt);
            long long x = n_;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d) x += y;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, x > rem);
            if (past || qt + 32 >= nqt) {
                const int src = past ? __ffs(past) - 1 : 0;
                rem -= __shfl_sync(0xFFFFFFFFu, x - n_, src);
                qt += src;
                break;
            }
            rem -= __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        t = attn_tile(a, rq, qt);
        units = max(1, t.n);
        return (int)rem;
    }
    // Where a boundary `from` units into this tile is: moved to the tile's begin or end if that is near.
    __device__ __forceinline__ int snapped(int from, int snap) const {
        if (units <= kAttnWhole) return 2 * from < units ? 0 : units;
        return from <= snap ? 0 : (units - from <= snap ? units : from);
    }
    // Begins a range of n units at unit u, `from` units into the tile found.
    __device__ __forceinline__ void begin(const AttnArgs& a, long long u, int from, long long n) {
        at = u;
        left = n;
        k0 = k1 = units;
        if (left <= 0) return;
        fetch(a);
        if (from == units)
            next(a);                   // the next tile's begin
        else
            cut(from);
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ void next(const AttnArgs& a) {
        left -= k1 - k0;
        at += k1 - k0;
        if (left <= 0) return;
        if (++qt == nqt) {
            qt = 0;
            h += a.gang;
            if (h >= a.heads) {
                h = me % a.gang;
                do {
                    enter(a);
                } while (nqt == 0 && r < a.R - 1);
            }
        }
        t = attn_tile(a, rq, qt);
        cut(0);
    }
    __device__ __forceinline__ int tiles() const { return t.n == 0 ? 0 : k1 - k0; }
    __device__ __forceinline__ int key_tile(int j) const {
        const int i = k0 + j;
        return i < t.first ? i : i + t.skip;
    }
};

// Units of a request per KV head: all query tiles' key tiles. Of long requests (the bits of `big`) the
// warp's lanes share the tiles, and the warps of a block take every `warps`-th, into `sums`.
__device__ __forceinline__ long long attn_units(const AttnArgs& a, const AttnReq& q, bool live, unsigned& big) {
    const int nqt = live ? attn_tiles(a, q) : 0;
    long long w = 0;
    if (nqt <= 2)
        for (int i = 0; i < nqt; ++i) w += max(1, attn_tile(a, q, i).n);
    big = __ballot_sync(0xFFFFFFFFu, nqt > 2);
    return w;
}
__device__ __forceinline__ void attn_units_long(const AttnArgs& a, const AttnReq& q, unsigned big, int warp, int warps,
                                                long long* sums) {
    for (int i = 0; big; ++i, big &= big - 1) {
        if (i % warps != warp) continue;
        const int src = __ffs(big) - 1;
        AttnReq s;
        s.q0 = 0;
        s.n = __shfl_sync(0xFFFFFFFFu, q.n, src);
        s.kv = __shfl_sync(0xFFFFFFFFu, q.kv, src);
        const int m = attn_tiles(a, s);
        long long v = 0;
        for (int k = threadIdx.x & 31; k < m; k += 32) v += max(1, attn_tile(a, s, k).n);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        if ((threadIdx.x & 31) == 0) sums[src] = v;
    }
}

// ---------------------------------------------------------------- instructions

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// D (+)= A * B with both operands in shared memory; predicated like tc_mma.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate, bool issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"((uint32_t)issue)
        : "memory");
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzled layout: rows of 128
// bytes hold 64 consecutive N of one K; 8 K make a 1024-byte atom (stride between groups of 8 K),
// `panel` bytes lead to the next 64 N.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t addr, uint32_t panel) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// The same over a pair of blocks (cta_group::2): issued by the even block of the cluster for both,
// each holding its rows of A and D and half of B's N. A commit arrives on the barrier at this
// address in both blocks.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, bool issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"((uint32_t)issue)
        : "memory");
}
__device__ __forceinline__ void tc_mma_pair_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate, bool issue) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"((uint32_t)issue)
        : "memory");
}
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, bool issue) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(
            bar),
        "r"((uint32_t)issue), "h"((uint16_t)3)
        : "memory");
}

// Arrival on a barrier of another block of the cluster that publishes nothing outside TMEM.
__device__ __forceinline__ void mbar_arrive_remote_cta(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

#define NQ_R4(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3])
#define NQ_O4(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3])

// 32 consecutive columns of the thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : NQ_O4(v, 0), NQ_O4(v, 4), NQ_O4(v, 8), NQ_O4(v, 12), NQ_O4(v, 16), NQ_O4(v, 20), NQ_O4(v, 24), NQ_O4(v, 28)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        NQ_R4(v, 0), NQ_R4(v, 4), NQ_R4(v, 8), NQ_R4(v, 12), NQ_R4(v, 16), NQ_R4(v, 20), NQ_R4(v, 24), NQ_R4(v, 28)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        NQ_R4(v, 0), NQ_R4(v, 4), NQ_R4(v, 8), NQ_R4(v, 12)
        : "memory");
}
#undef NQ_R4
#undef NQ_O4

// The device's base-2 exponential instruction (2 ulp): the softmax's p is rounded to 16 bits.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 32 bytes to global memory: one store where they are aligned (a row of the output is a lane's, so every
// 16-byte store of a warp touches 32 lines), else two.
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8], bool aligned) {
    if (aligned)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                     "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                     : "memory");
    else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// Bits 0..n-1 of 64, for any n.
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}

__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

// Instruction descriptor: D fp32, A and B of one 16-bit type, A K-major, B K-major or (b_mn)
// N-major, M = m, N = n.
constexpr uint32_t attn_idesc(bool bf16, int m, int n, bool b_mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// ---------------------------------------------------------------- the kernel

template <int D, bool BF16, bool PAIR>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    using Geo = AttnGeo<D, PAIR>;
    constexpr int kBlocks = PAIR ? 2 : 1;      // blocks of a query tile
    constexpr int kSlots = Geo::kSlots, kKS = Geo::kKSlots, kVS = Geo::kVSlots, kDK = Geo::kDK, kVK = Geo::kVKeys;
    constexpr int kKK = Geo::kKKeys, kDV = Geo::kDV;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    extern __shared__ __align__(1024) uint8_t attn_smem[];
    uint8_t* const qmem = attn_smem;
    uint8_t* const ring = attn_smem + Geo::kQBytes;
    uint8_t* const ctrl = ring + kSlots * Geo::kSlotBytes;
    float* const red = reinterpret_cast<float*>(ctrl);                      // [2][2 groups][128]
    uint64_t* const bars = reinterpret_cast<uint64_t*>(ctrl + 2048);
    // bars: full[8], empty[8], s_full[2], p_ready[2], pv_done[2], o_free, q_full, q_free, done, and of the
    // leading block of a pair: the other's q_full and full[8], passed on
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kAttnMaxSlots, sfull0 = empty0 + 8 * kAttnMaxSlots;
    const uint32_t pready0 = sfull0 + 16, pvdone0 = pready0 + 16, ofree = pvdone0 + 16, qfull = ofree + 8, qfree = qfull + 8;
    const uint32_t done = qfree + 8, qfull_other = done + 8, full_other0 = qfull_other + 8;
    volatile int* const flags = reinterpret_cast<volatile int*>(ctrl + 2048 + 320);
    // flags: [0] abort, [3] TMEM base
    long long* const warp_sums = reinterpret_cast<long long*>(ctrl + 2048 + 384);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint64_t wait_ns = a.wait_ns;
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, 1);
            mbar_init(full_other0 + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull0 + 8 * i, 1);
            mbar_init(pready0 + 8 * i, kBlocks * kAttnSoftmaxWarps);
            mbar_init(pvdone0 + 8 * i, 1);
        }
        mbar_init(ofree, kBlocks * kAttnSoftmaxWarps);
        mbar_init(qfull, 1);
        mbar_init(qfull_other, 1);
        mbar_init(qfree, 1);
        mbar_init(done, 1);
        // the swizzled tiles need a 1024-byte base
        flags[0] = (smem_u32(attn_smem) & 1023u) != 0;
        if (flags[0]) atomicOr(a.dev_err, kDevErrTimeout);
        mbar_fence_init();
    }
    if (warp == 0) {
        if constexpr (PAIR)
            tmem_alloc_pair(smem_u32(const_cast<int*>(flags) + 3), 512);
        else
            tmem_alloc(smem_u32(const_cast<int*>(flags) + 3), 512);
    }
    grid_dependency_wait();

    // The block's range of units. Up to 32 requests every warp scans by itself, one a lane; more are
    // scanned by the block into the ring buffers (free until the first copies).
    AttnWalk w;
    w.me = blockIdx.x / kBlocks;
    w.left = 0;
    long long total = 0, blocks = 1;   // blocks: ranges with work
    int snap = 0;
    // locate(u): finds unit u in w, and returns its place in its tile
    struct Plan {
        AttnWalk walk;
        int from[2], to[2];
    };
    Plan* const plan = reinterpret_cast<Plan*>(ctrl + 2048 + 640);
    static_assert(2048 + 640 + sizeof(Plan) <= kAttnCtrlBytes, "room for the plan");
    auto range = [&](auto locate) {
        const long long me = w.me / a.gang;
        // no range is empty but between whole tiles: the join takes every block from a tile's first to
        // its last as a part
        blocks = max(1ll, min((long long)a.gangs, total));
        snap = total > 2 * kAttnSnap * blocks ? kAttnSnap : 0;
        const long long e0 = total * me, e1 = e0 + total;
        long long u0, u1;
        if (e1 >> 32 == 0) {           // both quotients at once
            u0 = (uint32_t)e0 / (uint32_t)blocks;
            u1 = (uint32_t)e1 / (uint32_t)blocks;
        } else {
            u0 = e0 / blocks;
            u1 = e1 / blocks;
        }
        u0 = min(u0, total);
        u1 = min(u1, total);
        if (u0 >= u1) return;
        // half of the warps look for the begin, half for the end (each search is a chain of some 0.9 us)
        const bool last = warp >= kAttnThreads / 64;
        int from = 0, to = 0;
        if (!last || u1 < total) {
            from = locate(last ? u1 : u0);
            to = w.snapped(from, snap);
        }
        if (lane == 0 && (warp == 0 || warp == kAttnThreads / 64)) {
            if (!last) plan->walk = w;
            plan->from[last] = from;
            plan->to[last] = to;
        }
        __syncthreads();
        w = plan->walk;
        u0 += plan->to[0] - plan->from[0];
        u1 += plan->to[1] - plan->from[1];
        w.begin(a, u0, plan->to[0], u1 - u0);
    };
    if (a.R <= 32) {
        AttnReq rq = {0, 0, 0};
        if (lane < a.R) rq = attn_req(a, lane);
        unsigned big;                  // the same in every warp
        long long mine = attn_units(a, rq, lane < a.R, big);
        if (big) {
            attn_units_long(a, rq, big, warp, kAttnThreads / 32, warp_sums);
            __syncthreads();
            if ((big >> lane) & 1) mine = warp_sums[lane];
        }
        mine *= a.turns;
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long u = __shfl_up_sync(0xFFFFFFFFu, upto, d);
            if (lane >= d) upto += u;
        }
        total = __shfl_sync(0xFFFFFFFFu, upto, 31);
        range([&](long long u) {
            const int r = min(__popc(__ballot_sync(0xFFFFFFFFu, upto <= u)), a.R - 1);
            AttnReq q;
            q.q0 = __shfl_sync(0xFFFFFFFFu, rq.q0, r);
            q.n = __shfl_sync(0xFFFFFFFFu, rq.n, r);
            q.kv = __shfl_sync(0xFFFFFFFFu, rq.kv, r);
            return w.find(a, r, q, __shfl_sync(0xFFFFFFFFu, upto - mine, r), __shfl_sync(0xFFFFFFFFu, mine, r), u);
        });
    } else {
        long long* const upto = reinterpret_cast<long long*>(attn_smem);
        for (int r0 = 0; r0 < a.R; r0 += kAttnThreads) {
            const int r = r0 + tid;
            AttnReq rq = {0, 0, 0};
            if (r < a.R) rq = attn_req(a, r);
            unsigned big;
            long long x = attn_units(a, rq, r < a.R, big);
            if (big) {
                attn_units_long(a, rq, big, 0, 1, upto + r0 + 32 * warp);
                __syncwarp();
                if ((big >> lane) & 1) x = upto[r];
            }
            x *= a.turns;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d) x += u;
            }
            __syncthreads();           // the sums of the round before have been read
            if (lane == 31) warp_sums[warp] = x;
            __syncthreads();
            long long before = total;
#pragma unroll
            for (int i = 0; i < kAttnThreads / 32; ++i) {
                const long long s = warp_sums[i];
                if (i < warp) before += s;
                total += s;
            }
            if (r < a.R) upto[r] = before + x;
        }
        __syncthreads();
        range([&](long long u) {
            int lo = 0, hi = a.R - 1;  // the first request whose units pass u
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (upto[mid] > u)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const long long base = lo > 0 ? upto[lo - 1] : 0;
            return w.find(a, lo, attn_req(a, lo), base, upto[lo] - base, u);
        });
        fence_proxy_async_smem();      // the scan's buffers go to the copy engine
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)flags[3];
    // One arrival of the warp on a barrier of the leading block. The second block's releases at cluster scope
    // where the warp's lanes have written shared memory that the leader's products read (`published`: the rows of
    // V that they zeroed before their last __syncwarp). Else block scope will do, and is much cheaper: what is in TMEM
    // is ordered by tcgen05's own fences, and a copy's writes are released by the copy itself, at cluster scope, on the
    // barrier that the arrival passes on. (At cluster scope every softmax arrival cost a tile 1100 cycles; those
    // of the copies alone took 2048 tokens over 16384 from 590 us to 650.)
    const uint32_t to_leader = PAIR ? cluster_map(full0, 0) - full0 : 0;
    auto arrive_leader = [&](uint32_t bar, bool published) {
        if (PAIR && rank == 1) {
            if (lane == 0 && published) mbar_arrive_remote(bar + to_leader);
            if (lane == 0 && !published) mbar_arrive_remote_cta(bar + to_leader);
        } else {
            mbar_arrive_if(bar, lane == 0);
        }
    };
    if constexpr (PAIR) cluster_sync_all();    // both blocks' barriers are initialised

    if (warp == kAttnProducerK || warp == kAttnProducerV) {
        // ------------------------------------------------------------ producers
        const bool is_v = warp == kAttnProducerV;
        // a box is `rows` keys of a page; a slot holds slot_keys keys x slot_cols columns
        const int slot_keys = is_v ? kVK : kKK, slot_cols = is_v ? kDV : kDK, slots = is_v ? kVS : kKS;
        const int rows = min(1 << a.page_shift, slot_keys), row_bits = __ffs(rows) - 1;
        const int page_rows = min(1 << a.page_shift, kAttnKeys), page_bits = __ffs(page_rows) - 1;
        const int ids_of = kAttnKeys >> page_bits, page_mask = (1 << a.page_shift) - 1, panels = slot_cols / 64;
        const CUtensorMap* const map = is_v ? &a.vmap : &a.kmap;
        int base = 0;                      // slots filled by the segments before, by both producers
        uint32_t filled = 0, parity = 0;   // per slot: whether this warp filled it, and the phase
        bool ok = flags[0] == 0;
        // block ids of key tile kt, one a lane: -1, which reads as zeros, where no row sees any of the keys
        auto ids = [&](const AttnWalk& k, int kt) {
            const int key = kt * kAttnKeys + lane * page_rows;
            const bool seen = key < k.t.hi && (key < a.sinks || key + page_rows > k.t.lo);
            return lane < ids_of && seen ? __ldg(a.table + k.r * a.table_stride + (key >> a.page_shift)) : -1;
        };
        for (; w.more() && ok; w.next(a)) {
            const int n = w.tiles();
            if (n == 0) continue;
            int id = ids(w, w.key_tile(0)), id_next = n > 1 ? ids(w, w.key_tile(1)) : -1;
            for (int j = 0; j < n && ok; ++j) {
                const int id_after = j + 2 < n ? ids(w, w.key_tile(j + 2)) : -1;
                int seq = base + (is_v ? kKS + j * (kKS + kVS) + (j + 1 < n ? kKS : 0)
                                       : (j == 0 ? 0 : kKS + (j - 1) * (kKS + kVS)));
                for (int s = 0; s < slots; ++s, ++seq) {
                    const int slot = seq % kSlots;
                    // (a barrier is at most one phase behind: what the fill before this one had to wait
                    // for comes after the use of this slot two rounds ago)
                    if (seq >= kSlots) ok = mbar_wait(empty0 + 8 * slot, ((seq / kSlots) - 1) & 1, flags, a.dev_err, wait_ns);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    // a pair's blocks load half of the keys of K, half of the columns of V
                    const int off = is_v ? s * kVK : rank * kKK, key0 = w.key_tile(j) * kAttnKeys + off;
                    // V is filled whole, with zeros past the keys: 0 x what a slot held before may be NaN
                    int boxes = slot_keys >> row_bits;
                    if (!is_v) boxes = max(0, min(boxes, (w.t.hi - key0 + rows - 1) >> row_bits));
                    const uint32_t bar = full0 + 8 * slot, dst = smem_u32(ring + slot * Geo::kSlotBytes);
                    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * rows * slot_cols * 2));
                    __syncwarp();
                    const int copies = boxes * panels, col0 = is_v ? rank * kDV : s * kDK;
                    for (int o0 = 0; o0 < copies; o0 += 32) {
                        const int o = o0 + lane, box = o / panels, panel = o % panels;
                        const int at = off + box * rows;
                        const int block = __shfl_sync(0xFFFFFFFFu, id, (at >> page_bits) & 31);
                        if (o < copies)
                            tma_load_4d(dst + panel * (slot_keys * 128) + box * rows * 128, map, col0 + panel * 64,
                                        (key0 + box * rows) & page_mask, w.h, block, bar);
                    }
                    filled |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | ((uint32_t)((seq / kSlots) & 1) << slot);
                }
                id = id_next;
                id_next = id_after;
            }
            base += n * (kKS + kVS);
        }
        if (!ok)                           // aborted: this warp's last copy into each slot
            for (int i = 0; i < kSlots; ++i)
                if ((filled >> i) & 1) mbar_wait_drain(full0 + 8 * i, (parity >> i) & 1, kDrainNs);
    } else if (PAIR && rank == 1 && warp == kAttnMma) {
        // ------------------------------------------------------------ the second block's copies, passed on
        int seq = 0, seg = 0;
        bool ok = flags[0] == 0;
        for (; w.more() && ok; w.next(a)) {
            const int n = w.tiles();
            if (n == 0) continue;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(qfull, seg & 1, flags, a.dev_err, wait_ns));
            if (ok) arrive_leader(qfull_other, false);
            for (int i = 0; i < n * (kKS + kVS) && ok; ++i, ++seq) {
                const int slot = seq % kSlots;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(full0 + 8 * slot, (seq / kSlots) & 1, flags, a.dev_err, wait_ns));
                if (ok) arrive_leader(full_other0 + 8 * slot, false);
            }
            ++seg;
        }
    } else if (warp == kAttnMma) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdescS = attn_idesc(BF16, kBlocks * kAttnRows, kAttnKeys, false);
        constexpr uint32_t kIdescO = attn_idesc(BF16, kBlocks * kAttnRows, D, true);
        auto commit = [&](uint32_t bar, bool issue) {
            if constexpr (PAIR)
                tc_commit_pair(bar, issue);
            else
                tc_commit(bar, issue);
        };
        // a slot is full, in both blocks of a pair
        auto wait_full = [&](int slot, uint32_t parity) {
            bool there = mbar_wait(full0 + 8 * slot, parity, flags, a.dev_err, wait_ns);
            if (PAIR) there = there && mbar_wait_cluster(full_other0 + 8 * slot, parity, flags, a.dev_err, wait_ns);
            return there;
        };
        // a barrier on which the softmax warps (of both blocks) arrive
        auto wait_warps = [&](uint32_t bar, uint32_t parity) {
            if constexpr (PAIR)
                return mbar_wait_cluster(bar, parity, flags, a.dev_err, wait_ns);
            else
                return mbar_wait(bar, parity, flags, a.dev_err, wait_ns);
        };
        const bool leader = elect_one();
        const uint32_t qbase = smem_u32(qmem), ring0 = smem_u32(ring);
        int seq = 0, g = 0, seg = 0;
        bool ok = flags[0] == 0;
        auto score = [&](int gt) {         // S of the tile with global count gt
            const uint32_t s_col = tmem + kAttnSCol + kAttnKeys * (gt & 1);
            for (int s = 0; s < kKS; ++s) {
                const int slot = seq % kSlots;
                ok = __all_sync(0xFFFFFFFFu, ok && wait_full(slot, (seq / kSlots) & 1));
                if (!ok) return;
                tc_fence_after();
                const uint32_t kbase = ring0 + slot * Geo::kSlotBytes;
#pragma unroll
                for (int i = 0; i < kDK / 16; ++i) {
                    const uint64_t ad = smem_desc_sw128(qbase + (s * (kDK / 64) + i / 4) * (kAttnRows * 128) + 32 * (i % 4));
                    const uint64_t bd = smem_desc_sw128(kbase + (i / 4) * (kKK * 128) + 32 * (i % 4));
                    if constexpr (PAIR)
                        tc_mma_pair_ss(s_col, ad, bd, kIdescS, i > 0 ? 1u : 0u, leader);
                    else
                        tc_mma_ss(s_col, ad, bd, kIdescS, (s > 0 || i > 0) ? 1u : 0u, leader);
                }
                commit(empty0 + 8 * slot, leader);
                ++seq;
            }
            commit(sfull0 + 8 * (gt & 1), leader);
        };
        for (; w.more() && ok; w.next(a)) {
            const int n = w.tiles();
            if (n == 0) continue;
            ok = mbar_wait(qfull, seg & 1, flags, a.dev_err, wait_ns);
            if (PAIR) ok = ok && mbar_wait_cluster(qfull_other, seg & 1, flags, a.dev_err, wait_ns);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            score(g);
            for (int j = 0; j < n && ok; ++j, ++g) {
                if (j + 1 < n) score(g + 1);
                if (!ok) break;
                if (j == n - 1) commit(qfree, leader);
                const int buf = g & 1;
                ok = wait_warps(pready0 + 8 * buf, (g >> 1) & 1);
                if (ok && j == 0 && seg > 0) ok = wait_warps(ofree, (seg - 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t p_col = tmem + kAttnSCol + kAttnKeys * buf;
                for (int s = 0; s < kVS; ++s) {
                    const int slot = seq % kSlots;
                    ok = __all_sync(0xFFFFFFFFu, ok && wait_full(slot, (seq / kSlots) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t vbase = ring0 + slot * Geo::kSlotBytes;
#pragma unroll
                    for (int i = 0; i < kVK / 16; ++i) {
                        const int key = s * kVK + 16 * i;    // its half of P starts at column 64 * (key / 64)
                        const uint32_t ac = p_col + 64 * (key / 64) + (key % 64) / 2;
                        const uint64_t bd = smem_desc_mn128(vbase + i * 2048, kVK * 128);
                        const uint32_t add = (j > 0 || s > 0 || i > 0) ? 1u : 0u;
                        if constexpr (PAIR)
                            tc_mma_pair(tmem, ac, bd, kIdescO, add, leader);
                        else
                            tc_mma(tmem, ac, bd, kIdescO, add, leader);
                    }
                    commit(empty0 + 8 * slot, leader);
                    ++seq;
                }
                if (ok) commit(pvdone0 + 8 * buf, leader);
            }
            ++seg;
        }
        // every MMA has completed before TMEM can be freed
        commit(done, leader);
        mbar_wait_drain(done, 0, kDrainNs);
    } else if (warp == kAttnLoader) {
        // ------------------------------------------------------------ query tiles
        int seg = 0;
        bool ok = flags[0] == 0;
        for (; w.more() && ok; w.next(a)) {
            if (w.tiles() == 0) continue;
            if (seg > 0) ok = mbar_wait(qfree, (seg - 1) & 1, flags, a.dev_err, wait_ns);
            if (!ok) break;
            // few tokens: as many small boxes as they fill
            const int rows_here = min(max(w.t.rows - rank * a.block_tokens * a.group, 1), a.block_tokens * a.group);
            const int box = a.few_tokens * a.group, n = (rows_here + box - 1) / box;
            const bool few = n * box <= kAttnRows && n <= 4;
            const int rows = few ? n * box : a.block_tokens * a.group, copies = (few ? n : 1) * (D / 64);
            if (lane == 0) mbar_arrive_expect_tx(qfull, (uint32_t)(rows * D * 2));
            __syncwarp();
            if (lane < copies) {
                const int panel = lane % (D / 64), i = lane / (D / 64);
                tma_load_3d(smem_u32(qmem) + panel * (kAttnRows * 128) + i * box * 128, few ? &a.qfew : &a.qmap, 64 * panel,
                            w.h * a.group, w.rq.q0 + w.t.token0 + rank * a.block_tokens + i * a.few_tokens, qfull);
            }
            __syncwarp();
            ++seg;
        }
        if (!ok && seg > 0) mbar_wait_drain(qfull, (seg - 1) & 1, kDrainNs);
    } else {
        // ------------------------------------------------------------ softmax
        // pv_done of a buffer may be waited for in any of its phases or in none: S of tile g is full
        // only after the products of tile g - 2 and all before it (one thread commits both).
        // These warps never leave their loops early: after an abort the waits return at once, and
        // the pairs' barriers stay matched.
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
        const float c = a.scale_log2;
        const int row_token = row / a.group, row_head = row - row_token * a.group;
        int g = 0, seq = 0;
        int4 split0 = make_int4(-1, 0, 0, 0);
        int split_count = 0;
        for (; w.more(); w.next(a)) {
            const AttnTile& t = w.t;
            const int n = w.tiles();
            const bool whole = w.k0 == 0 && w.k1 == w.units;
            // this block's part of the tile
            const int token0 = t.token0 + rank * a.block_tokens;
            const int rows = min(max(t.rows - rank * a.block_tokens * a.group, 0), a.block_tokens * a.group);
            const int pf = t.pf + rank * a.block_tokens, pl = min(pf + a.block_tokens - 1, t.pl);
            const bool valid = row < rows;
            if (w.k0 == 0 && !whole) {
                // the last unit's owner: ranges begin at floor(total c / blocks), and one that begins near
                // the tile's end at that; it is the same block of its gang
                const long long stop = w.at + w.units;
                long long c = (stop * blocks - 1) / total;
                const int from = (int)max(0ll, attn_div(total * c, blocks) - w.at);
                if (w.snapped(from, snap) == w.units) --c;
                split0 = make_int4(w.r, w.h, token0, rows);
                split_count = (int)c - w.me / a.gang + 1;
            }
            uint16_t* const orow = a.out + (w.rq.q0 + token0 + row_token) * a.out_stride +
                                   (long long)(w.h * a.group + row_head) * D + half * (D / 2);
            if (n == 0) {                  // no key is seen
                if (valid)
#pragma unroll
                    for (int i = 0; i < D / 2; i += 8) *reinterpret_cast<uint4*>(orow + i) = make_uint4(0, 0, 0, 0);
                continue;
            }
            const bool active = 32 * quarter < rows;
            const int p = pf + row_token;
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int j = 0; j < n; ++j, ++g) {
                const int buf = g & 1, key0 = w.key_tile(j) * kAttnKeys;
                bool published = false;        // whether rows of V have been zeroed
                ok = mbar_wait(sfull0 + 8 * buf, (g >> 1) & 1, flags, a.dev_err, wait_ns);
                tc_fence_after();
                if (active) {
                    const uint32_t s_col = lane_base + kAttnSCol + kAttnKeys * buf + 64 * half;
                    const bool masked = key0 + kAttnKeys - 1 > pf || (a.window > 0 && key0 < pl - a.window + 1);
                    // the thread's 64 columns of S, which are the keys from kk on; keys that the row does not
                    // see as -inf
                    uint32_t v[64];
                    const int kk = key0 + 64 * half;
                    tmem_ld32(s_col, v);
                    tmem_ld32(s_col + 32, v + 32);
                    tmem_wait_ld();
                    if (masked) {
                        uint64_t see = low_bits(p - kk + 1);
                        if (a.window > 0) see &= ~low_bits(p - a.window + 1 - kk) | low_bits(a.sinks - kk);
                        const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            v[i] = (see0 & (1u << i)) ? v[i] : 0xFF800000u;
                            v[32 + i] = (see1 & (1u << i)) ? v[32 + i] : 0xFF800000u;
                        }
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            m4[e] = fmaxf(m4[e], fmaxf(__uint_as_float(v[i + e]), __uint_as_float(v[i + 4 + e])));
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    float* const x = red + (g & 1) * 256;
                    x[half * 128 + row] = mx;
                    named_bar_sync(1 + quarter, 64);
                    mx = fmaxf(fmaxf(mx, x[(half ^ 1) * 128 + row]), m);
                    // keep the old maximum while the new one is within 2^kAttnLazy of it
                    const bool grow = valid && mx > m && !((mx - m) * c <= kAttnLazy);
                    if (j > 0 && __any_sync(0xFFFFFFFFu, grow)) {
                        const float f = grow ? exp2_fast((m - mx) * c) : 1.f;
                        mbar_wait(pvdone0 + 8 * (buf ^ 1), ((g - 1) >> 1) & 1, flags, a.dev_err, wait_ns);
                        tc_fence_after();
                        const uint32_t o_col = lane_base + half * (D / 2);
#pragma unroll
                        for (int i = 0; i < D / 2; i += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_col + i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_col + i, o);
                        }
                        l *= f;
                    }
                    if (grow) m = mx;
                    const float off = m == -INFINITY ? 0.f : fmaf(-m, c, BF16 ? 0.f : kAttnLift);
                    // p = 2^(c s + off), rounded, over S; their sum joins l. In two parts, so that the first is
                    // stored while the second is computed.
                    const uint64_t cc = pack2(__float_as_uint(c), __float_as_uint(c));
                    const uint64_t oo = pack2(__float_as_uint(off), __float_as_uint(off));
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 x2 = unpack2(fma2(pack2(v[32 * q + i], v[32 * q + i + 1]), cc, oo));
                            const float e0 = exp2_fast(x2.x), e1 = exp2_fast(x2.y);
                            sum[(i / 2) & 3] = add2(sum[(i / 2) & 3], pack2(__float_as_uint(e0), __float_as_uint(e1)));
                            pk[i / 2] = pack16<BF16>(e0, e1);
                        }
                        tmem_st16(s_col + 16 * q, pk);
                    }
                    const float2 s2 = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                    l += s2.x + s2.y;
                    tmem_wait_st();
                }
                if (key0 + kAttnKeys > t.hi || min(t.lo, key0 + kAttnKeys) > max(key0, a.sinks)) {
                    // the V slots of tile j: after K of the first tile, each tile's V follows the next tile's K
                    // (S of the tile is there, so the slots up to its K have been filled; where a slot's fill before
                    // this one comes later, the tile before is waited for, or the barrier may be one fill behind)
                    if (kKS + 2 * kVS > kSlots && j > 0)
                        ok = mbar_wait(pvdone0 + 8 * (buf ^ 1), ((g - 1) >> 1) & 1, flags, a.dev_err, wait_ns) && ok;
                    const int v0 = seq + kKS + j * (kKS + kVS) + (j + 1 < n ? kKS : 0);
                    for (int s = 0; s < kVS; ++s)
                        ok = mbar_wait(full0 + 8 * ((v0 + s) % kSlots), ((v0 + s) / kSlots) & 1, flags, a.dev_err, wait_ns) && ok;
                    if (ok) {
                        // a thread's 16-byte chunk of the rows, every kStep-th row
                        constexpr int kChunks = kDV / 8, kStep = kAttnSoftmaxWarps * 32 / kChunks;
                        const int ch = tid % kChunks;
                        auto zero = [&](int from, int to) {
                            from -= key0;
                            to = min(to - key0, kAttnKeys);
                            for (int key = from + tid / kChunks; key < to; key += kStep) {
                                uint8_t* const slot = ring + ((v0 + key / kVK) % kSlots) * Geo::kSlotBytes;
                                *reinterpret_cast<uint4*>(slot + (ch / 8) * (kVK * 128) + (key % kVK) * 128 + (ch % 8) * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                        };
                        // Keys that no row sees in pages with others that some row does (V's producer leaves out
                        // whole pages): from the last key on, up to the window, from the sinks on
                        const int page = min(1 << a.page_shift, kAttnKeys);
                        const int tail = t.hi & (page - 1) ? t.hi & -kAttnKeys : -1;
                        const int head = (t.lo & (page - 1)) && t.lo > a.sinks ? t.lo & -kAttnKeys : -1;
                        const int first = (a.sinks & (page - 1)) && a.sinks < t.lo ? a.sinks & -kAttnKeys : -1;
                        if (key0 == tail) zero(t.hi, (t.hi + page - 1) & -page);
                        if (key0 == head) zero(max(t.lo & -page, a.sinks), t.lo);
                        if (key0 == first) zero(a.sinks, min((a.sinks + page - 1) & -page, t.lo));
                        fence_proxy_async_smem();
                        published = true;
                    }
                }
                tc_fence_before();
                __syncwarp();
                arrive_leader(pready0 + 8 * buf, published);
            }
            seq += n * (kKS + kVS);
            // the tile's rows: finished, or a partial with its maximum and sum
            ok = mbar_wait(pvdone0 + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, flags, a.dev_err, wait_ns);
            tc_fence_after();
            if (active) {
                float* const x = red + (g & 1) * 256;
                x[half * 128 + row] = l;
                named_bar_sync(1 + quarter, 64);
                l += x[(half ^ 1) * 128 + row];
                named_bar_sync(1 + quarter, 64);       // the next tile's maxima use the same buffer
                const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
                float* const pcol = a.part + ((size_t)slot * D + half * (D / 2)) * kAttnRows + row;
                const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                for (int i = 0; i < D / 2; i += 32) {
                    uint32_t o[32];
                    tmem_ld32(lane_base + half * (D / 2) + i, o);
                    tmem_wait_ld();
                    if (valid && ok) {
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                uint32_t u[8];
#pragma unroll
                                for (int q = 0; q < 8; ++q)
                                    u[q] = pack16<BF16>(__uint_as_float(o[e + 2 * q]) * inv, __uint_as_float(o[e + 2 * q + 1]) * inv);
                                store32(orow + i + e, u, a.wide);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) pcol[(i + e) * kAttnRows] = __uint_as_float(o[e]);
                        }
                    }
                }
                if (!whole && valid && half == 0) a.ml[slot * kAttnRows + row] = make_float2(m, l);
            }
            tc_fence_before();
            __syncwarp();
            arrive_leader(ofree, false);
        }
        // output rows past the requests' are zeros
        const int last_start = __ldg(a.q_start + a.R);
        for (int i = min(max(last_start, 0), a.tokens) + blockIdx.x; i < a.tokens; i += gridDim.x)
            for (int e = tid; e < a.heads * a.group * (D / 8); e += kAttnSoftmaxWarps * 32)
                reinterpret_cast<uint4*>(a.out + i * a.out_stride)[e] = make_uint4(0, 0, 0, 0);
        if (tid == 0) {
            a.splits[2 * blockIdx.x] = split0;
            a.splits[2 * blockIdx.x + 1] = make_int4(split_count, 0, 0, 0);
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();    // nothing arrives on, or multiplies in, a block that has left
    if (warp == 0) {
        tc_fence_after();
        if constexpr (PAIR)
            tmem_dealloc_pair(tmem, 512);
        else
            tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- the join

constexpr int kJoinThreads = 256;
constexpr int kJoinBlocksY = 16;   // most blocks of a split's items
constexpr int kJoinParts = 8;      // most threads that share an item's partials

// Adds the partials of the query tiles that were split over several blocks, in block order:
// O = sum_i 2^(c (m_i - M)) O_i / sum_i 2^(c (m_i - M)) l_i. An item is 8 columns of a row; blocks
// (x, *) share the items of the tile that block x of the attention kernel opened, neighbouring lanes
// taking neighbouring rows (partials are stored column by column). Up to 8 threads share an
// item's partials, each with a running maximum, so that few rows with many partials are read in
// parallel. Bound by latency: two or three rounds of loads.
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, 3) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    __shared__ float acc[kJoinThreads][11];    // 8 columns, maximum, sum (odd stride: no bank conflicts)
    grid_launch_dependents();
    grid_dependency_wait();
    const int tid = threadIdx.x;
    const int4 s = a.splits[2 * blockIdx.x];
    if (s.x >= 0) {
        const int count = a.splits[2 * blockIdx.x + 1].x, rows = s.w;
        const AttnReq rq = attn_req(a, s.x);
        const float c = a.scale_log2;
        const int parts = count >= 8 ? 8 : (count >= 4 ? 4 : 1), per = kJoinThreads / parts;
        const int part = tid / per, items = rows * (D / 8);
        for (int i0 = blockIdx.y * per; i0 < items; i0 += gridDim.y * per) {
            const int item = i0 + tid % per, group = item / rows, row = item - group * rows;
            float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.f;
            if (item < items) {
#pragma unroll 3
                for (int i = part; i < count; i += parts) {
                    const int slot = 2 * ((int)blockIdx.x + i * a.stride) + (i == 0 ? 1 : 0);
                    const float2 ml = a.ml[slot * kAttnRows + row];
                    const float* src = a.part + ((size_t)slot * D + group * 8) * kAttnRows + row;
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = src[e * kAttnRows];
                    const float mx = fmaxf(m, ml.x), ref = mx == -INFINITY ? 0.f : mx;
                    const float f = exp2_fast((m - ref) * c), fi = exp2_fast((ml.x - ref) * c);
                    l = l * f + ml.y * fi;
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + v[e] * fi;
                    m = mx;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[tid][e] = o[e];
            acc[tid][8] = m;
            acc[tid][9] = l;
            __syncthreads();
            if (tid < per && item < items) {
                float mx = -INFINITY;
                for (int i = 0; i < parts; ++i) mx = fmaxf(mx, acc[i * per + tid][8]);
                if (mx == -INFINITY) mx = 0.f;
                float total = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = 0.f;
                for (int i = 0; i < parts; ++i) {
                    const float* x = acc[i * per + tid];
                    const float f = exp2_fast((x[8] - mx) * c);
                    total += f * x[9];
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] += f * x[e];
                }
                const float inv = total == 0.f ? 0.f : 1.f / total;
                const int token = row / a.group, head = s.y * a.group + row - token * a.group;
                uint4 u;
                u.x = pack16<BF16>(o[0] * inv, o[1] * inv);
                u.y = pack16<BF16>(o[2] * inv, o[3] * inv);
                u.z = pack16<BF16>(o[4] * inv, o[5] * inv);
                u.w = pack16<BF16>(o[6] * inv, o[7] * inv);
                *reinterpret_cast<uint4*>(a.out + (rq.q0 + s.z + token) * a.out_stride +
                                          (long long)head * D + group * 8) = u;
            }
            __syncthreads();
        }
    }
}

}  // namespace nq
