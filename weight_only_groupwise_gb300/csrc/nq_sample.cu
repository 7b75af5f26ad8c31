// nq_sample.cu -- the choice of the next token (nq_sample): temperature, top-k, top-p and min-p,
// with the random numbers given as one Exp(1) variate per token. Among the kept tokens, the
// argmax of d_i - log(noise_i), d_i = (l_i - max) / T, is token i with probability proportional
// to exp(d_i) (the first of independent exponential clocks of rates exp(d_i) to ring): no
// cumulative sum decides the token, so rounding moves the choice only where two scores are
// within an ulp of each other.
//
// A row is a thread-block cluster, a slice of the row a block, kept in shared memory when it fits
// (one read of the logits from memory). Three ways through a row:
//   * no top-k and no top-p: the cluster's maximum, then one pass that takes the argmax (the race).
//     The score is first estimated with the fast logarithm; only tokens that could beat the
//     thread's best are scored exactly.
//   * a cut that few tokens pass (the common case): kept tokens are a prefix of the row's order
//     (logit descending, index ascending). Every block sorts its threads' maxima; the k-th of
//     them bounds the block's k-th token from below, so the tokens from there up, little more than k,
//     hold its first k. They are handed to one block, which sorts them and settles the row: one
//     barrier of the cluster. top-p alone tries the same with the first 48 of each block, if
//     those can hold the share (one row of 152064 then takes 13 us, 23 where they cannot; with 96 tokens 19 and
//     24, with 24 tokens 13 and 27, and fewer rows are settled).
//   * a cut among many tokens: the race over all tokens, then one pass that sums what lies before
//     its winner. If that is less than k tokens, or than the share p, the winner is kept, and so
//     is the winner of the kept ones. Else all kept tokens lie before it, and the race is run
//     again among those. A winner lies at a random place of the mass, so it is kept with the
//     probability of the kept mass, 1 + ln(1 / kept mass) races on average; the same pass halves the
//     interval that holds the cut, so that 65 races are the most whatever the noise.
//   * both such a top-k and a top-p: the share is one of top-k's mass. A histogram of the cluster's
//     tokens by the distance to the maximum finds the bin of top-k's cut, which bounds that mass
//     to a few tokens' weights: enough to judge nearly every winner. Else the bin's tokens are sorted by
//     one block; a bin of more tokens than that block can sort (far tails, many equal logits) is
//     cut again by the bits of the logits' ordered integers, at most three times.
// The race lists the tokens that may be kept in shared memory, so that all threads share them
// (64 rows with min-p 31 -> 20 us); a race over all tokens needs no list.
// A token's weight is one whole number of 2^-44 of the maximum's, whichever way its row takes, and sums of
// weights are integers: a cut depends neither on an order of summation nor on the blocks of a row. (V 2^-45 of the
// mass, 1.6e-8 at the largest vocabulary, is the most that the rounding moves. With 2^-30 a tail of half a million tokens
// could be 2e-4 off.) The mass of a row whose top-p is tried with few tokens is first known as a float sum; a winner
// that lies within that sum's error of the cut is left to the trials.
//
// Bound by the latency of these few steps for few rows, by instructions per token and barriers
// for many (the logits' bytes alone would take a fraction of it). Measured, replayed in a graph: one row of 152064
// bf16, top-k 50 and top-p 0.9, 10.3 us; 64 of them 17; 64 with mixed settings 47 to 67, 256 of 128257 fp32 121 to 152
// (by the random numbers). With histograms of the mass in place of the trials the mixed ones took 79 and 157.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_launch.h"
#include "nq_step.h"

namespace cg = cooperative_groups;

namespace nq {

namespace {

typedef unsigned long long u64;

constexpr int kSaThreads = 512;
constexpr int kSaWarps = kSaThreads / 32;
constexpr int kSaBins = 2048;
constexpr int kSaPer = kSaBins / kSaThreads;   // bins of a thread
constexpr int kSaList = 4 * kSaThreads;        // tokens the settling block can sort
constexpr int kSaTokens = kSaBins + 2 * kSaList;   // kept tokens a block lists before it scores them
constexpr int kSaTryP = 48;                    // tokens a block hands over for top-p alone
constexpr int kSaMaxCluster = 8;
constexpr int kSaMaxSlice = 65535;
constexpr int kSaMaxVocab = kSaMaxSlice / 16 * 16 * kSaMaxCluster;
constexpr int kSaSliceBytes = 160 * 1024;      // most shared memory for a slice
constexpr int kSaTwoBytes = 86 * 1024;          // up to here two blocks fit an SM
constexpr float kSaRange = 32.f;               // distance to the maximum covered by the bins
constexpr float kSaLeastT = 0.75f;             // in units of max(T, this)
constexpr float kSaOne = 1073741824.f;         // 2^30: the unit of the try's float sums
constexpr int kSaHigh = 23;                    // a weight is a sum of two parts, of 2^-21 and of 2^-(21 + this)
constexpr u64 kSaWhole = 1ull << (21 + kSaHigh);   // the weight of the maximum
// Error of the try's mass, relative: 136 fp32 sums a thread (8.1e-6), exponents up to 31 rounded three times (3.9e-6), 512
// truncations a block (4.8e-7), and the weights' own rounding: below 1.3e-5.
constexpr float kSaMassError = 3.0517578e-5f;
constexpr uint32_t kSaNone = 0x007FFFFFu;      // ordered integer of -inf

struct SampleArgs {
    const void* logits;
    long long stride;
    const float* noise;
    long long noise_stride;
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    int* tokens;
    int V, slice, resident;                    // tokens of a slice; whether slices stay in shared memory
};

// Order-preserving integer of a float; NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// (value, lowest index) as one ordered integer.
__device__ __forceinline__ u64 ranked(uint32_t key, int i) { return ((u64)key << 32) | (0xFFFFFFFFu - (uint32_t)i); }
__device__ __forceinline__ int index_of(u64 v) { return (int)(0xFFFFFFFFu - (uint32_t)v); }

// The least integer that is not below p * w (0 < p < 1; at least 1: the first token is always
// kept), by integers: fp64 runs at a small fraction of the integer rate.
__device__ __forceinline__ u64 share_of(float p, u64 w) {
    if (!(p > 0.f)) return 1;
    const uint32_t u = __float_as_uint(p), ex = u >> 23;
    const u64 mant = ex ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;
    const int shift = 150 - (int)(ex ? ex : 1);      // p = mant * 2^-shift, shift >= 24
    if (shift > 100) return 1;
    const unsigned __int128 v = (unsigned __int128)mant * w, one = (unsigned __int128)1 << shift;
    const u64 t = (u64)((v + one - 1) >> shift);
    return t > 0 ? t : 1;
}

struct Found {             // the bin of a cut by count: the tokens before it and in it
    int bin, before, count;
    int none;              // fewer tokens than that
};

// Tokens of a higher rank than (at, index): from `next` up, or `at` itself below the index.
struct Above {
    float at, next;
    int index;
    __device__ __forceinline__ explicit Above(u64 rank)
        : at(key_value((uint32_t)(rank >> 32))), next(key_value((uint32_t)(rank >> 32) + 1)),
          index((int)min(0xFFFFFFFFu - (uint32_t)rank, 0x7FFFFFFFu)) {}
    // for a chunk of n tokens from i0: values from here up, and whether the index falls inside
    __device__ __forceinline__ float least(int i0, int n) const { return i0 + n <= index ? at : next; }
    // (no token is below index 0, which a chunk may begin before)
    __device__ __forceinline__ bool inside(int i0, int n) const { return index > 0 && i0 < index && i0 + n > index; }
};

struct Share {             // what a block hands to the settling one besides its first tokens
    float weight, listed_weight;   // sums of its tokens' weights and of the handed ones, for its own maximum
    float top;             // its maximum
    int count;             // tokens handed over
    uint32_t low;          // its other tokens lie below this key (0: there are none)
    int fail;              // its first tokens do not fit
};

struct SaShared {
    union {
        struct {
            unsigned hist[kSaBins];
            u64 list[kSaList];
        };
        int kept_tokens[kSaTokens];
    };
    u64 part[2][kSaMaxCluster];                // cluster exchange, alternating
    u64 part_w[2][kSaMaxCluster];
    u64 warp[kSaWarps];
    u64 warp_w[kSaWarps];
    Share share[kSaMaxCluster];
    Found found;
    u64 cut;
    u64 kept, target, target_hi;               // of the trials: the least rank known to be kept; bounds of the share
    uint32_t bound;
    int listed, verdict;
};

__device__ __forceinline__ void unpack_chunk(const uint4& u, float (&x)[4], float) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack_chunk(const uint4& u, float (&x)[8], __nv_bfloat16) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack_chunk(const uint4& u, float (&x)[8], __half) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void load4(const uint8_t* p, float (&x)[4], float) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x;
    x[1] = u.y;
    x[2] = u.z;
    x[3] = u.w;
}
template <typename T>
__device__ __forceinline__ void load4(const uint8_t* p, float (&x)[4], T) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    float v[8];
    unpack_chunk(make_uint4(u.x, u.y, 0, 0), v, T());
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = v[e];
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
struct Row {
    static constexpr int E = 16 / (int)sizeof(T);      // elements of a 16-byte chunk
    const T* base;                             // the row
    const uint8_t* smem;                       // the slice's chunks, or null
    int begin, end;                            // the slice
    int lead;                                  // elements before `begin` in the first chunk
    int chunks;
    // Chunk c: E consecutive tokens from first(c), those outside the slice as -inf.
    __device__ __forceinline__ int first(int c) const { return begin - lead + c * E; }
    __device__ __forceinline__ uint4 from_global(int c) const {
        const int i0 = first(c);
        if (i0 >= begin && i0 + E <= end) return __ldg(reinterpret_cast<const uint4*>(base + i0));
        alignas(16) T x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = i0 + e >= begin && i0 + e < end ? base[i0 + e] : T(-INFINITY);
        return *reinterpret_cast<const uint4*>(x);
    }
    __device__ __forceinline__ float value(int i) const {
        return as_float(smem ? reinterpret_cast<const T*>(smem)[i - first(0)] : base[i]);
    }
    __device__ __forceinline__ void load(int c, float (&x)[E]) const {
        unpack_chunk(smem ? reinterpret_cast<const uint4*>(smem)[c] : from_global(c), x, T());
    }
};

// The cluster's first barrier, in two halves: a block may address another's shared memory only once that
// one has begun to run, which being placed together does not make sure.
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_begun() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Block-wide maximum of v, in every thread.
__device__ __forceinline__ u64 block_max(u64 v, SaShared& s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const u64 o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = o > v ? o : v;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s.warp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s.warp[threadIdx.x & (kSaWarps - 1)];
#pragma unroll
    for (int d = kSaWarps / 2; d > 0; d >>= 1) {
        const u64 o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = o > v ? o : v;
    }
    return v;
}

// Inclusive scans of (x, y) over the block; the totals in tx, ty.
__device__ __forceinline__ void block_scan(u64& x, u64& y, u64& tx, u64& ty, SaShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const u64 ux = __shfl_up_sync(0xFFFFFFFFu, x, d), uy = __shfl_up_sync(0xFFFFFFFFu, y, d);
        if (lane >= d) {
            x += ux;
            y += uy;
        }
    }
    __syncthreads();
    if (lane == 31) {
        s.warp[warp] = x;
        s.warp_w[warp] = y;
    }
    __syncthreads();
    tx = ty = 0;
    u64 bx = 0, by = 0;
#pragma unroll
    for (int i = 0; i < kSaWarps; ++i) {
        if (i == warp) {
            bx = tx;
            by = ty;
        }
        tx += s.warp[i];
        ty += s.warp_w[i];
    }
    x += bx;
    y += by;
}

// Bitonic sort, descending, of N consecutive values a thread: partners in the thread, in the warp
// (shuffles), and only then through shared memory (`buf`, N values a thread).
template <int N, typename U>
__device__ __forceinline__ void block_sort(U (&v)[N], U* buf) {
    const int tid = threadIdx.x;
    auto pick = [](U a, U b, bool larger) { return (a > b) == larger ? a : b; };
    for (int len = 2; len <= kSaThreads * N; len *= 2)
        for (int d = len / 2; d > 0; d /= 2) {
            if (d >= 32 * N) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < N; ++j) buf[tid * N + j] = v[j];
                __syncthreads();
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int i = tid * N + j;
                    v[j] = pick(v[j], buf[i ^ d], ((i & d) == 0) == ((i & len) == 0));
                }
            } else if (d >= N) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int i = tid * N + j;
                    v[j] = pick(v[j], __shfl_xor_sync(0xFFFFFFFFu, v[j], d / N), ((i & d) == 0) == ((i & len) == 0));
                }
            } else {
#pragma unroll
                for (int dd = 1; dd < N; dd *= 2)
                    if (d == dd) {
#pragma unroll
                        for (int j = 0; j < N; ++j)
                            if ((j & dd) == 0) {
                                const U a = v[j], b = v[j | dd];
                                const bool desc = ((tid * N + j) & len) == 0;
                                v[j] = pick(a, b, desc);
                                v[j | dd] = pick(a, b, !desc);
                            }
                    }
            }
        }
    __syncthreads();
}

// (l - top) / T from e = top - l: a quotient by the reciprocal with one correction is the rounded
// one away from the ends of the range of T, where the division itself is used.
struct Scaler {
    float temp, inv;
    bool usual;
    __device__ __forceinline__ explicit Scaler(float t) : temp(t), inv(1.f / t), usual(t >= 1e-6f && t <= 1e6f) {}
    __device__ __forceinline__ float operator()(float e) const {
        if (!usual || !(e < 1e30f)) return -e / temp;
        const float q = e * inv;
        return -fmaf(fmaf(-q, temp, e), inv, q);
    }
};

// A token's weight relative to the maximum's, from e = top - l.
struct WeightParts {
    unsigned high;         // of 2^-21, and of 2^-44: up to 2^21, and 2^22 either way
    int low;
};
struct Weigher {
    float c;
    // (never 0, so that an infinite distance weighs nothing at an infinite temperature)
    __device__ __forceinline__ explicit Weigher(float temp)
        : c(-fmaxf(1.4426950408889634f * fminf(1.f / temp, 1e30f), 1e-45f)) {}
    __device__ __forceinline__ float exp(float e) const {
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(e * c));
        return y;
    }
    // Rounded to 2^-44, without conversions: a sum with 1.5 x 2^n has its value in its low bits. Threads add the
    // parts in 32 bits (136 tokens at most).
    __device__ __forceinline__ WeightParts parts(float e) const {
        const float w = exp(e), a = w + 6.f, b = (w - (a - 6.f)) + 0x1.8p-21f;
        return {__float_as_uint(a) - __float_as_uint(6.f), (int)(__float_as_uint(b) - __float_as_uint(0x1.8p-21f))};
    }
    static __device__ __forceinline__ u64 sum(unsigned high, int low) { return ((u64)high << kSaHigh) + (u64)(long long)low; }
    __device__ __forceinline__ u64 operator()(float e) const {
        const WeightParts w = parts(e);
        return sum(w.high, w.low);
    }
};

struct Settings {
    float p, floor_d;
    int k;
    bool by_k, by_p;
};

// The settling block: the row's token from the cluster's first tokens (n of them, gathered in
// s.list), N a thread. Returns the token, or -1 if top-p alone cannot be settled among them: because they
// may not hold the share, or because the winner is kept by one bound of the share (least, most) and not by the other.
template <int N>
__device__ __forceinline__ int settle(SaShared& s, int n, float m, uint32_t bound, u64 least, u64 most, const Settings& o,
                                      const Scaler& scaled, const Weigher& weight, const float* noise) {
    const int tid = threadIdx.x;
    u64 v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = tid * N + j < n ? s.list[tid * N + j] : 0;
    block_sort<N>(v, s.list);
    const uint32_t top = order_key(m);
    const int last = o.by_k ? min(n, o.k) : n;             // tokens that may be kept
    float d[N], z[N];
    u64 wt[N], x = 0, y = 0, unused, sum;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        z[j] = 1.f;
        d[j] = 0.f;
        wt[j] = 0;
        if (tid * N + j < last) {
            const uint32_t key = (uint32_t)(v[j] >> 32);
            z[j] = __ldg(noise + index_of(v[j]));
            if (key != top) d[j] = scaled(m - key_value(key));
            wt[j] = weight(key != top ? m - key_value(key) : 0.f);
        }
        y += wt[j];
    }
    const u64 own = y;
    block_scan(x, y, unused, sum, s);
    y -= own;
    const u64 target = !o.by_p ? ~0ull : (o.by_k ? share_of(o.p, sum) : most);
    u64 best = 0, best_unsure = 0;             // the best of all that may be kept, of those that `least` does not keep
    bool reached = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int at = tid * N + j;
        if (at < last) {
            if (at == 0 || (y < target && d[j] >= o.floor_d)) {
                const u64 c = ranked(order_key(d[j] - logf(z[j])), index_of(v[j]));
                best = c > best ? c : best;
                if (!o.by_k && at > 0 && y >= least) best_unsure = c;
            }
            y += wt[j];
            // the cut has to lie among tokens that no block has kept back
            reached |= (uint32_t)(v[j] >> 32) >= bound && y >= target;
        }
    }
    best = block_max(best, s);
    if (o.by_k) return index_of(best);
    const bool unsure = __syncthreads_or(best_unsure == best);
    const bool settled = bound == 0 || __syncthreads_or(reached);
    return settled && !unsure ? index_of(best) : -1;
}

// The at-th (from 0) of the n tokens in s.list, in the row's order.
template <int N>
__device__ __forceinline__ u64 nth(SaShared& s, int n, int at) {
    const int tid = threadIdx.x;
    u64 v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = tid * N + j < n ? s.list[tid * N + j] : 0;
    block_sort<N>(v, s.list);
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (tid * N + j == at) s.cut = v[j];
    __syncthreads();
    return s.cut;
}

template <typename T, int PerSm>
__global__ void __launch_bounds__(kSaThreads, PerSm) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t sa_slice[];
    __shared__ SaShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x;
    const int r = blockIdx.x / C;
    constexpr int E = Row<T>::E;

    if (C > 1) cluster_begun();            // waited for below, where the slice has been loaded
    grid_launch_dependents();
    grid_dependency_wait();

    Row<T> row;
    row.base = static_cast<const T*>(a.logits) + (long long)r * a.stride;
    row.begin = min(rank * a.slice, a.V);
    row.end = min(row.begin + a.slice, a.V);
    row.lead = (int)((reinterpret_cast<uintptr_t>(row.base + row.begin) & 15u) / sizeof(T));
    row.chunks = row.end > row.begin ? (row.lead + row.end - row.begin + E - 1) / E : 0;
    row.smem = nullptr;
    const float* const noise = a.noise + (long long)r * a.noise_stride;
    const float temp = a.temperature ? a.temperature[r] : 1.f;
    const float p = a.top_p ? a.top_p[r] : 1.f, least = a.min_p ? a.min_p[r] : 0.f;
    const int k = a.top_k ? a.top_k[r] : 0;
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f, greedy = !(temp > 0.f);
    const float floor_d = least > 0.f ? logf(fminf(least, 1.f)) : -INFINITY;

    // exchange: every block's values to every block of the cluster
    int turn = 0;
    auto exchange = [&](u64 v, u64 w) {
        turn ^= 1;
        __syncthreads();
        if (tid < C) {
            *cl.map_shared_rank(&s.part[turn][rank], tid) = v;
            *cl.map_shared_rank(&s.part_w[turn][rank], tid) = w;
        }
        cl.sync();
    };
    auto cluster_max = [&](u64 v) {
        v = block_max(v, s);
        if (C == 1) return v;
        exchange(v, 0);
        v = s.part[turn][0];
        for (int i = 1; i < C; ++i) v = s.part[turn][i] > v ? s.part[turn][i] : v;
        return v;
    };
    const Scaler scaled(temp);
    const Weigher weight(temp);
    const Settings set = {p, floor_d, k, by_k, by_p};

    // The noise of the slice on its way to L2, for rows that need all of it.
    auto prefetch = [&]() {
        const uintptr_t a0 = (reinterpret_cast<uintptr_t>(noise + row.begin) + 15) & ~(uintptr_t)15;
        const uintptr_t a1 = reinterpret_cast<uintptr_t>(noise + row.end) & ~(uintptr_t)15;
        if (tid == 0 && a1 > a0)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a0), "r"((uint32_t)(a1 - a0)) : "memory");
    };
    const int cap = kSaList / C;
    const bool try_few = !greedy && (by_k ? k <= cap : by_p);
    if (!greedy && !try_few && !(least > 0.f)) prefetch();

    // The slice goes to shared memory (all copies in flight at once); every thread's maximum.
    if (a.resident) {
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            const int i0 = row.first(c);
            if (i0 >= row.begin && i0 + E <= row.end)
                cp_async16(smem_u32(sa_slice) + c * 16, row.base + i0);
            else
                reinterpret_cast<uint4*>(sa_slice)[c] = row.from_global(c);
        }
        cp_async_wait_all();
        row.smem = sa_slice;               // threads read back what they copied themselves
    }
    float high = -INFINITY;
    for (int c = tid; c < row.chunks; c += kSaThreads) {
        float x[E];
        row.load(c, x);
#pragma unroll
        for (int e = 0; e < E; ++e) high = fmaxf(high, x[e]);   // ignores NaN
    }
    if (C > 1) cluster_wait_begun();       // from here on blocks store into one another's shared memory

    // ---------------------------------------------------------------- a cut that few tokens pass
    u64 row_top = 0;
    if (try_few) {
        // at least `want` of the block's tokens are not below the want-th of its threads' maxima
        const int want = by_k ? k : kSaTryP;
        uint32_t key[1] = {order_key(high)};
        block_sort<1>(key, reinterpret_cast<uint32_t*>(&s.hist[0]));
        if (tid == 0) {
            s.warp[0] = key[0];
            s.listed = 0;
        }
        if (tid == want - 1) s.bound = key[0];
        __syncthreads();
        const float top_here = key_value((uint32_t)s.warp[0]);
        const bool all = want > kSaThreads || s.bound <= kSaNone;
        const uint32_t low = all ? kSaNone + 1 : s.bound;
        const float low_value = key_value(low);
        const bool inf_here = top_here == INFINITY;
        u64* const mine = cl.map_shared_rank(&s.list[0], 0) + rank * cap;
        float w = 0.f, lw = 0.f;
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float v[E], we[E];
            row.load(c, v);
            unsigned hit = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) hit |= v[e] >= low_value ? 1u << e : 0u;
            if (!by_k) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    we[e] = inf_here ? (v[e] == INFINITY ? 1.f : 0.f) : weight.exp(top_here - v[e]);
                    w += we[e] > 0.f ? we[e] : 0.f;        // not NaN
                }
            }
            if (hit) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((hit >> e) & 1) {
                        const int at = atomicAdd(&s.listed, 1);
                        if (at < cap) mine[at] = ranked(order_key(v[e]), row.first(c) + e);
                        if (!by_k) lw += we[e];
                    }
            }
        }
        // the threads' sums in a fixed order: as integers
        u64 x = (u64)(w * kSaOne), y = (u64)(lw * kSaOne), all_w = 0, all_lw = 0;
        if (by_k)
            __syncthreads();
        else
            block_scan(x, y, all_w, all_lw, s);
        if (!by_k && (float)all_lw < p * (float)all_w && !(least > 0.f)) prefetch();      // not likely to do
        if (tid < C) {
            Share h;
            h.weight = (float)all_w;
            h.listed_weight = (float)all_lw;
            h.top = top_here;
            h.count = min(s.listed, cap);
            h.low = all ? 0u : low;
            h.fail = s.listed > cap;
            *cl.map_shared_rank(&s.share[rank], tid) = h;
        }
        cl.sync();
        float m = -INFINITY, mass = 0.f, listed = 0.f;
        uint32_t bound = 0;
        bool fail = false;
        for (int i = 0; i < C; ++i) m = fmaxf(m, s.share[i].top);
        for (int i = 0; i < C; ++i) {
            const Share& h = s.share[i];
            fail |= h.fail != 0;
            bound = max(bound, h.low);
            if (!by_k && h.weight > 0.f) {
                const float f = h.top == m ? 1.f : expf(scaled(m - h.top));
                mass += h.weight * f;
                listed += h.listed_weight * f;
            }
        }
        // top-p alone: the listed tokens must be able to hold the share
        if (!by_k) fail |= !(listed >= p * mass * 0.9999f);
        if (!fail) {
            if (rank == 0) {
                // the blocks' parts, brought together (each is read before it is written over)
                int n = 0, from = 0;
                u64 part[kSaList / kSaThreads];
                for (int i = 0; i < C; ++i) n += s.share[i].count;
#pragma unroll
                for (int j = 0; j < kSaList / kSaThreads; ++j) {
                    int at = j * kSaThreads + tid;
                    part[j] = 0;
                    if (at < n) {
                        for (from = 0; at >= s.share[from].count; ++from) at -= s.share[from].count;
                        part[j] = s.list[from * cap + at];
                    }
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kSaList / kSaThreads; ++j) s.list[j * kSaThreads + tid] = part[j];
                __syncthreads();
                int token = -1;
                bool settled = n == 0;
                if (n > 0) {
                    const float unit = (float)kSaWhole / kSaOne;
                    u64 lo = 0, hi = 0;
                    if (!by_k) {
                        lo = share_of(p, (u64)(mass * unit * (1.f - kSaMassError)));
                        hi = share_of(p, (u64)(mass * unit * (1.f + kSaMassError)));
                    }
                    token = n <= kSaThreads       ? settle<1>(s, n, m, bound, lo, hi, set, scaled, weight, noise)
                            : n <= 2 * kSaThreads ? settle<2>(s, n, m, bound, lo, hi, set, scaled, weight, noise)
                                                  : settle<4>(s, n, m, bound, lo, hi, set, scaled, weight, noise);
                    settled = token >= 0;
                }
                if (settled && tid == 0) a.tokens[r] = token;
                if (!by_k && tid < C) *cl.map_shared_rank(&s.verdict, tid) = settled ? 1 : 0;
            }
            if (by_k) return;
            cl.sync();
            if (s.verdict) return;
        }
        row_top = order_key(m);
    } else {
        row_top = cluster_max(order_key(high));
    }
    const uint32_t top = (uint32_t)row_top;
    if (top <= kSaNone) {                          // nothing to choose from
        if (rank == 0 && tid == 0) a.tokens[r] = -1;
        return;
    }
    const float m = key_value(top);
    if (greedy) {
        u64 best = 0;
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float x[E];
            row.load(c, x);
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                if (x[e] == m) best = max(best, ranked(top, row.first(c) + e));
        }
        best = cluster_max(best);
        if (rank == 0 && tid == 0) a.tokens[r] = index_of(best);
        return;
    }
    // An infinite maximum has all the mass: distances 0 and infinity.
    const bool inf_row = m == INFINITY;
    auto below = [&](float x) { return inf_row ? (x == INFINITY ? 0.f : INFINITY) : m - x; };

    // ---------------------------------------------------------------- top-k's cut among many tokens
    auto clear = [&]() {
        __syncthreads();
        for (int i = tid; i < kSaBins; i += kSaThreads) s.hist[i] = 0;
        __syncthreads();
    };
    // The bin of the k-th token, `base` tokens lying before the bins.
    auto find = [&](int base) {
        if (tid == 0) s.found.none = 1;
        cl.sync();
        const int sec = kSaBins / C, per = sec > kSaThreads ? sec / kSaThreads : 1;
        const int b0 = rank * sec + tid * per;
        const bool mine = tid * per < sec;
        unsigned cnt[kSaPer];
        u64 x = 0, unused = 0, tx, ty;
#pragma unroll
        for (int i = 0; i < kSaPer; ++i) {
            cnt[i] = 0;
            if (mine && i < per) {
#pragma unroll
                for (int c = 0; c < kSaMaxCluster; ++c)
                    if (c < C) cnt[i] += cl.map_shared_rank(&s.hist[0], c)[b0 + i];
                x += cnt[i];
            }
        }
        const u64 own = x;
        block_scan(x, unused, tx, ty, s);
        x -= own;
        if (C > 1) {
            exchange(tx, 0);
            for (int i = 0; i < rank; ++i) x += s.part[turn][i];
        }
        x += base;
#pragma unroll
        for (int i = 0; i < kSaPer; ++i) {
            if (mine && i < per && x < (u64)k && x + cnt[i] >= (u64)k) {
                const Found f = {b0 + i, (int)x, (int)cnt[i], 0};
                for (int c = 0; c < C; ++c) *cl.map_shared_rank(&s.found, c) = f;
            }
            x += cnt[i];
        }
        cl.sync();
        return s.found;
    };
    const float scale = (kSaBins / kSaRange) / fmaxf(temp, kSaLeastT);
    // the last bin takes everything past the range
    auto place = [&](float d) { return fminf(d * scale, (float)(kSaBins - 1)); };
    auto bin_of = [&](float d) { return (int)place(d); };
    // The cut in the bin f, if its tokens can be sorted: all blocks hand them to the first.
    auto sort_bin = [&](const Found& f) {
        u64* const list = cl.map_shared_rank(&s.list[0], 0);
        int* const listed = cl.map_shared_rank(&s.listed, 0);
        if (tid == 0) s.listed = 0;
        cl.sync();
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float x[E];
            row.load(c, x);
            unsigned hit = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) hit |= x[e] > -INFINITY && bin_of(below(x[e])) == f.bin ? 1u << e : 0u;
            if (hit) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((hit >> e) & 1) list[atomicAdd(listed, 1)] = ranked(order_key(x[e]), row.first(c) + e);
            }
        }
        cl.sync();
        if (rank == 0) {
            const int at = k - 1 - f.before;
            const u64 found = f.count <= kSaThreads ? nth<1>(s, f.count, at) : nth<4>(s, f.count, at);
            if (tid > 0 && tid < C) *cl.map_shared_rank(&s.cut, tid) = found;
        }
        cl.sync();
        return s.cut;
    };
    // The same by the bits of the bin's keys: down to one key, and the first tokens at it.
    auto refine_bin = [&](const Found& f) {
        u64 most = 0, fewest = 0;
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float x[E];
            row.load(c, x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] > -INFINITY && bin_of(below(x[e])) == f.bin) {
                    const uint32_t key = order_key(x[e]);
                    most = max(most, (u64)key);
                    fewest = max(fewest, (u64)(0xFFFFFFFFu - key));
                }
        }
        uint32_t hi = (uint32_t)cluster_max(most), lo = 0xFFFFFFFFu - (uint32_t)cluster_max(fewest);
        int before = f.before;
        while (lo < hi) {
            const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
            clear();
            for (int c = tid; c < row.chunks; c += kSaThreads) {
                float x[E];
                row.load(c, x);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t key = order_key(x[e]);
                    if (key >= lo && key <= hi) atomicAdd(&s.hist[(hi - key) >> shift], 1u);
                }
            }
            const Found g = find(before);
            if (g.none) break;             // cannot be: the interval holds the cut
            before = g.before;
            hi -= (uint32_t)g.bin << shift;
            const uint32_t least_key = hi - ((1u << shift) - 1);
            lo = least_key > lo && least_key <= hi ? least_key : lo;
        }
        // the index of the last of the tokens at the key that are kept
        const u64 ties = (u64)(k - before);
        const float at = key_value(hi);
        u64 x = 0, y = 0, tx, ty, seen = 0, last = 0;
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float v[E];
            row.load(c, v);
#pragma unroll
            for (int e = 0; e < E; ++e) x += v[e] == at ? 1 : 0;
        }
        block_scan(x, y, tx, ty, s);
        if (C > 1) {
            exchange(tx, 0);
            for (int i = 0; i < rank; ++i) seen += s.part[turn][i];
        }
        for (int c0 = 0; c0 < row.chunks; c0 += kSaThreads) {
            const int c = c0 + tid;
            float v[E];
            u64 own = 0;
            if (c < row.chunks) {
                row.load(c, v);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) own += v[e] == at ? 1 : 0;
            x = own;
            y = 0;
            block_scan(x, y, tx, ty, s);
            x += seen - own;                   // tokens at the cut before this chunk
            seen += tx;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (v[e] == at && x++ < ties) last = (u64)(row.first(c) + e) + 1;
        }
        last = cluster_max(last);
        return ranked(hi, (int)last - 1);
    };
    Found f = {0, 0, 0, 1};
    if (by_k && by_p) {
        clear();
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float x[E];
            row.load(c, x);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (x[e] > -INFINITY) atomicAdd(&s.hist[bin_of(below(x[e]))], 1u);
        }
        f = find(0);
    }

    // ---------------------------------------------------------------- the race over the row
    // First by an estimate of the score (fast logarithm, product with 1 / T), each thread its best
    // two; then exactly, where a thread's best is within the estimate's error of the block's.
    u64 from = ((u64)kSaNone << 32) | 0xFFFFFFFFu;     // only tokens of higher ranks may be kept
    const float floor_e = -floor_d * temp;
    const float floor_lo = least > 0.f ? floor_e * 0.99999f : INFINITY, floor_hi = least > 0.f ? floor_e * 1.00001f : INFINITY;
    const float step = fminf(scaled.inv, 1e30f);
    auto estimate = [&](float v, float z) {
        const float sc = fmaf(-0.6931472f, __log2f(z), -below(v) * step);
        return sc == sc ? sc : -INFINITY;
    };
    // the tokens of a chunk that may be kept, as bits; false for NaN and -inf
    auto kept_of = [&](int c, const Above& set, float (&v)[E]) {
        row.load(c, v);
        const int i0 = row.first(c);
        const float low = set.least(i0, E);
        unsigned kept = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) kept |= v[e] >= low ? 1u << e : 0u;
        if (set.inside(i0, E)) {
#pragma unroll
            for (int e = 0; e < E; ++e) kept |= v[e] == set.at && i0 + e < set.index ? 1u << e : 0u;
        }
        if (kept && least > 0.f) {
            unsigned edge = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float d = below(v[e]);
                kept &= d > floor_hi ? ~(1u << e) : ~0u;
                edge |= d > floor_lo ? 1u << e : 0u;
            }
            if (kept & edge) {                         // as near to min-p's distance as rounding reaches
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((edge >> e) & 1 && !(scaled(below(v[e])) >= floor_d)) kept &= ~(1u << e);
            }
        }
        return kept;
    };
    auto race = [&]() {
        const Above set(from);
        float first = -INFINITY, second = -INFINITY;
        int first_i = -1;
        const bool all = set.at == -INFINITY && !(least > 0.f) && row.smem && !inf_row &&
                         (reinterpret_cast<uintptr_t>(noise + row.first(0)) & 15u) == 0;
        if (all) {
            // every token: four loads of noise in flight, nothing to choose
            const int groups = row.chunks > 0 ? (row.lead + row.end - row.begin + 3) / 4 : 0;
            for (int g = tid; g < groups; g += 4 * kSaThreads) {
                float4 u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i0 = row.first(0) + 4 * (g + j * kSaThreads);
                    if (i0 >= row.begin && i0 + 4 <= row.end) {
                        u[j] = __ldg(reinterpret_cast<const float4*>(noise + i0));
                    } else {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = i0 + e >= row.begin && i0 + e < row.end ? __ldg(noise + i0 + e) : 1.f;
                        u[j] = make_float4(w[0], w[1], w[2], w[3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = 4 * (g + j * kSaThreads);
                    if (at >= 4 * groups) break;
                    float x[4];
                    load4(row.smem + at * sizeof(T), x, T());
                    const float w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {          // NaN is never over
                        const float sc = fmaf(-0.6931472f, __log2f(w[e]), (x[e] - m) * step);
                        const bool over = sc > first;
                        second = over ? first : fmaxf(second, sc);
                        first = over ? sc : first;
                        first_i = over ? row.first(0) + at + e : first_i;
                    }
                }
            }
        } else {
            // the kept tokens are listed, so that all threads share them, and scored when the list is full
            __syncthreads();
            if (tid == 0) s.listed = 0;
            __syncthreads();
            const int lane = tid & 31;
            for (int c0 = 0; c0 < row.chunks; c0 += kSaThreads) {
                float v[E];
                const unsigned kept = c0 + tid < row.chunks ? kept_of(c0 + tid, set, v) : 0u;
                int at = 0;
                if (__any_sync(0xFFFFFFFFu, kept)) {
                    int upto = __popc(kept);
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        const int o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                        if (lane >= d) upto += o;
                    }
                    if (lane == 31) at = atomicAdd(&s.listed, upto);
                    at = __shfl_sync(0xFFFFFFFFu, at, 31) + upto - __popc(kept);
                    for (unsigned k2 = kept; k2; k2 &= k2 - 1) s.kept_tokens[at++] = row.first(c0 + tid) + __ffs(k2) - 1;
                }
                // the last of the warp's places is its last lane's
                const bool last = c0 + kSaThreads >= row.chunks;
                if (!__syncthreads_or(at > kSaTokens - kSaThreads * E) && !last) continue;
                const int n = s.listed;
                for (int i = tid; i < n; i += 4 * kSaThreads) {
                    int t[4];
                    float z[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i + j * kSaThreads < n) {
                            t[j] = s.kept_tokens[i + j * kSaThreads];
                            z[j] = __ldg(noise + t[j]);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i + j * kSaThreads < n) {
                            const float sc = estimate(row.value(t[j]), z[j]);
                            const bool over = sc > first || first_i < 0;
                            second = over ? first : fmaxf(second, sc);
                            first = over ? sc : first;
                            first_i = over ? t[j] : first_i;
                        }
                }
                if (last) break;
                __syncthreads();
                if (tid == 0) s.listed = 0;
                __syncthreads();
            }
        }
        // the estimate is off by less than this (unusual temperatures: not relied on)
        const float lead = key_value((uint32_t)block_max(first_i < 0 && !all ? 0 : order_key(first), s));
        auto may_win = [&](float sc) {
            if (!scaled.usual || lead == -INFINITY) return true;
            return sc > -INFINITY && !(sc + (2e-3f + 4e-6f * fabsf(sc)) < lead);
        };
        u64 best = 0;
        auto exact = [&](float l, float noise_i, int i) {
            float sc = scaled(below(l)) - logf(noise_i);
            if (sc != sc) sc = -INFINITY;
            best = max(best, ranked(order_key(sc), i));
        };
        const bool any = lead == -INFINITY || (first_i >= 0 && may_win(first));
        if (__syncthreads_or(any && (lead == -INFINITY || may_win(second)))) {
            for (int c = tid; c < row.chunks; c += kSaThreads) {   // two of one thread's tokens, or nothing to go by
                float v[E];
                const unsigned kept = kept_of(c, set, v);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if ((kept >> e) & 1) {
                        const float z = __ldg(noise + row.first(c) + e);
                        if (may_win(estimate(v[e], z))) exact(v[e], z, row.first(c) + e);
                    }
            }
        } else if (any) {
            exact(row.value(first_i), __ldg(noise + first_i), first_i);
        }
        return index_of(cluster_max(best));
    };

    // ---------------------------------------------------------------- the winner, if it is kept
    // Sums over the cluster of two sets' tokens: their number or, for top-p, their weight.
    auto weigh = [&](float l) { return by_p ? weight(below(l)) : 1ull; };
    auto sums = [&](const Above& a0, const Above& a1, bool bins, bool whole, u64& s0, u64& s1) {
        unsigned x_high = 0, y_high = 0;
        int x_low = 0, y_low = 0;
        const float edge = key_value(order_key(-(float)f.bin) + 1);        // the least number above -f.bin
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            float v[E];
            row.load(c, v);
            const int i0 = row.first(c);
            const float l0 = bins ? edge : a0.least(i0, E), l1 = a1.least(i0, E);
            if (!whole) {                              // few chunks have tokens of either
                float most = v[0];
#pragma unroll
                for (int e = 1; e < E; ++e) most = fmaxf(most, v[e]);
                if (!(most >= fminf(l0, l1))) continue;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool in0 = (bins ? -(below(v[e]) * scale) : v[e]) >= l0, in1 = v[e] >= l1;
                const WeightParts w = by_p ? weight.parts(below(v[e])) : WeightParts{0u, 1};
                x_high += in0 ? w.high : 0u;
                x_low += in0 ? w.low : 0;
                y_high += in1 ? w.high : 0u;
                y_low += in1 ? w.low : 0;
            }
        }
        u64 x = Weigher::sum(x_high, x_low), y = Weigher::sum(y_high, y_low);
        // equal values below the index in the chunk that the index falls in, if it is one of this slice's (the next
        // slice may share it, and an index between two tokens' ranks may be any number)
        auto rest = [&](const Above& a) {
            u64 n = 0;
            if (a.index > row.first(0) && a.index < row.first(row.chunks)) {
                const int c = (a.index - row.first(0)) / E;
                if (c % kSaThreads == tid)
                    for (int i = max(row.first(c), row.begin); i < min(a.index, row.end); ++i) n += row.value(i) == a.at ? 1 : 0;
            }
            return n * weigh(a.at);
        };
        if (!bins) x += rest(a0);
        y += rest(a1);
        block_scan(x, y, s0, s1, s);
        if (C > 1) {
            exchange(s0, s1);
            s0 = s1 = 0;
            for (int i = 0; i < C; ++i) {
                s0 += s.part[turn][i];
                s1 += s.part_w[turn][i];
            }
        }
    };
    // Ranks from s.kept up are kept, ranks up to `from` are not. With both cuts top-k's is known at
    // first by its bin only (`loose`), which bounds the weight of its tokens from both sides; a token
    // between the bounds, one in thousands, makes all blocks look for the cut itself.
    bool loose = !f.none;
    if (tid == 0) {
        s.kept = ((u64)top << 32) | 0xFFFFFFFFu;
        s.target = s.target_hi = by_p ? 0 : (u64)k;
    }
    int winner;
    for (int round = 0;; ++round) {
        winner = race();
        if (!by_k && !by_p) break;
        const u64 won = ranked(order_key(as_float(row.base[winner])), winner), hi = s.kept;
        u64 target = s.target, target_hi = s.target_hi;
        if (won >= hi) break;
        u64 mid = won + (hi - won) / 2, before_mid, before;
        if ((mid >> 32) == 0x7FFFFFFFu) mid = 0x7FFFFFFEFFFFFFFFull;       // as a value that key equals 0
        // the first round has no use for mid: top-p's set, or the part of it in the bins before top-k's
        sums(Above(round == 0 ? from : mid), Above(won), round == 0 && loose, round == 0, before_mid, before);
        if (round == 0 && by_p) {
            u64 most = 0, fewest = 0;
            if (loose) {
                const u64 w0 = f.bin > 0 ? weight(f.bin / scale * 0.999999f) : kSaWhole;
                const u64 w1 = weight((f.bin + 1) / scale * 1.000001f);
                most = (u64)(k - f.before) * (w0 + (w0 >> 13) + 1);
                fewest = f.bin < kSaBins - 1 && w1 > 0 ? (u64)(k - f.before) * (w1 - (w1 >> 13) - 1) : 0;
            }
            target = share_of(p, before_mid + fewest);
            target_hi = share_of(p, before_mid + most);
        }
        // 1: kept, 0: not kept, -1: not known
        auto judge = [&](u64 rank, u64 sum) {
            if (!loose) return sum < target ? 1 : 0;
            const float at = place(below(key_value((uint32_t)(rank >> 32))));
            if (sum >= target_hi || at >= (float)(f.bin + 1)) return 0;
            return sum < target && at < (float)f.bin ? 1 : -1;
        };
        const int is_kept = judge(won, before), mid_kept = round > 0 ? judge(mid, before_mid) : 0;
        if (is_kept == 1) break;
        from = won;
        // past the far edge of top-k's bin nothing is kept
        if (loose && f.bin < kSaBins - 1)
            from = max(from, (u64)order_key(m - (f.bin + 1) / scale * 1.00001f - 1e-6f * fabsf(m)) << 32);
        if (is_kept < 0 || mid_kept < 0) {
            const u64 last = f.count <= kSaList ? sort_bin(f) : refine_bin(f);
            u64 mass, unused;
            sums(Above(last - 1), Above(last - 1), false, true, mass, unused);
            target = target_hi = share_of(p, mass);
            loose = false;
            if (won >= last && before < target) break;
            from = max(from, last - 1);
        } else if (round > 0 && mid_kept == 0) {
            from = max(from, mid);
        }
        if (tid == 0) {                                // read again after the race's barriers
            if (round > 0 && mid_kept == 1) s.kept = mid;
            s.target = target;
            s.target_hi = target_hi;
        }
    }
    if (rank == 0 && tid == 0) a.tokens[r] = winner;
}

template <typename T, int PerSm>
nq_status sample_launch(const SampleArgs& a, int B, int C, size_t bytes, const StepDevice& d, cudaStream_t stream) {
    auto kern = sample_kernel<T, PerSm>;
    static thread_local int set_for_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (set_for_device != dev) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSaSliceBytes) != cudaSuccess)
            return NQ_ERR_CUDA;
        set_for_device = dev;
    }
    return step_launch(kern, dim3((unsigned)(B * C)), dim3(kSaThreads), a.resident ? bytes : 0, stream, d.pdl, C, a) ==
                   cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

template <typename T>
nq_status sample_rows(SampleArgs a, int B, const StepDevice& d, cudaStream_t stream) {
    // Eight blocks a row while every block of the call can be resident at once (two an SM); past
    // that fewer and larger slices, up to 40000 tokens (fp32: what fits shared memory), which saves
    // cluster barriers. Measured, mixed settings: 64 rows of 152064 bf16 51 us at 8, 47 at 4; 256
    // rows of 128257 fp32 157 at 8, 124 at 4, 267 at 2; top-k 50 on 256 rows of 32001 25 at 2, 16 at 1. 16-bit slices
    // up to 65000, which would fit too: 256 rows of 200000 150 us against 215, 64 of them 64 against 69, but 256 of
    // 128256 with top-k 50 and top-p 0.9 66 against 59; 152064, 160000 and 262144 the same within 3 %.
    int C = kSaMaxCluster;
    while (C > 1 && (long long)B * C > 2 * d.sms && a.V / (C / 2) <= 40000) C /= 2;
    a.slice = ((a.V + C - 1) / C + 15) / 16 * 16;
    const size_t bytes = ((size_t)a.slice * sizeof(T) + 15) / 16 * 16 + 16;
    a.resident = bytes <= (size_t)kSaSliceBytes;
    // Slices of which only one fits an SM leave a thread 128 registers (256 rows of 128257 fp32 137 -> 124 us).
    if (a.resident && bytes > (size_t)kSaTwoBytes) return sample_launch<T, 1>(a, B, C, bytes, d, stream);
    return sample_launch<T, 2>(a, B, C, bytes, d, stream);
}

bool meet(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace

}  // namespace nq

using namespace nq;

extern "C" nq_status nq_sample(const void* logits, int dtype, long long stride, const float* noise,
                               long long noise_stride, int B, int V, const float* temperature, const int* top_k,
                               const float* top_p, const float* min_p, int* tokens, void* stream) {
    if (B < 0 || B > (1 << 20) || V < 1 || V > kSaMaxVocab || stride < V || noise_stride < V) return NQ_ERR_SHAPE;
    if (dtype != NQ_BF16 && dtype != NQ_FP16 && dtype != NQ_FP32) return NQ_ERR_SHAPE;
    if (B == 0) return NQ_OK;
    const long long logits_span = step_span(B, stride, V), noise_span = step_span(B, noise_stride, V);
    if (logits_span < 0 || noise_span < 0) return NQ_ERR_SHAPE;
    if (!logits || !noise || !tokens) return NQ_ERR_NULL;
    const int size = dtype == NQ_FP32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % size) return NQ_ERR_ALIGN;
    for (const void* p : {(const void*)noise, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                          (const void*)min_p, (const void*)tokens})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return NQ_ERR_ALIGN;
    const long long tb = B * 4ll;
    if (meet(tokens, tb, logits, logits_span * size) || meet(tokens, tb, noise, noise_span * 4) ||
        meet(tokens, tb, temperature, tb) || meet(tokens, tb, top_k, tb) || meet(tokens, tb, top_p, tb) ||
        meet(tokens, tb, min_p, tb))
        return NQ_ERR_ALIAS;
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    SampleArgs a = {logits, stride, noise, noise_stride, temperature, top_k, top_p, min_p, tokens, V, 0, 0};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == NQ_BF16) return sample_rows<__nv_bfloat16>(a, B, d, s);
    if (dtype == NQ_FP16) return sample_rows<__half>(a, B, d, s);
    return sample_rows<float>(a, B, d, s);
}
