// nq_sample.cu -- the choice of the next token (nq_sample): temperature, top-k, top-p and min-p,
// with the random numbers given as one Exp(1) variate per token. Among the kept tokens, the
// argmax of d_i - log(noise_i), d_i = (l_i - max) / T, is token i with probability proportional
// to exp(d_i) (the first of independent exponential clocks of rates exp(d_i) to ring): no
// cumulative sum decides the token, so rounding moves the choice only where two scores are
// within an ulp of each other.
//
// Kept tokens are a prefix of the row's order (logit descending, index ascending), so a row needs
// a cut, not a sort: a histogram of the distance to the maximum finds the bin that holds the
// cut. If few tokens lie up to that bin they are gathered, sorted and settled by one block; else
// the cut is refined over the bits of the logits' ordered integers (at most three more
// histograms) and a last pass over the row takes the argmax.
//
// Weights are summed as 2^-30 fixed point in integers (two 32-bit halves in the histogram): sums
// are exact and do not depend on the order of the atomics.
//
// A row is a thread-block cluster, a slice of the row a block, kept in shared memory when it fits
// (one read of the logits from memory); histograms and results cross through distributed shared
// memory. Bound by the latency of these few steps for few rows, by the logits' (and, unfiltered,
// the noise's) bytes for many.
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
constexpr int kSaList = 2 * kSaThreads;        // tokens the gathering block can sort
constexpr int kSaMaxCluster = 8;
constexpr int kSaMaxSlice = 65535;             // 16-bit halves of the weights sum below 2^32
constexpr int kSaMaxVocab = kSaMaxSlice / 16 * 16 * kSaMaxCluster;
constexpr int kSaSliceBytes = 160 * 1024;      // most shared memory for a slice
constexpr float kSaRange = 32.f;               // distance to the maximum covered by the bins
constexpr float kSaLeastT = 0.75f;             // in units of max(T, this)
constexpr float kSaOne = 1073741824.f;         // 2^30: the weight of the maximum
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

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

struct Found {             // the bin of a cut: counts and weights of the tokens before it and in it
    int bin, before, count, total;
    u64 before_w, total_w;
    int by_count;          // the cut was looked for by count (else by weight)
    int none;              // no cut
};

struct SaShared {
    unsigned hist[3][kSaBins];                 // count, low and high halves of the weights
    u64 list[kSaList];
    u64 part[2][kSaMaxCluster];                // cluster exchange, alternating
    u64 part_w[2][kSaMaxCluster];
    u64 warp[kSaWarps];
    u64 warp_w[kSaWarps];
    Found found;
    unsigned listed;
    u64 scalar;
};

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
    __device__ __forceinline__ void from_global(int c, T (&x)[E]) const {
        const int i0 = first(c);
        if (i0 >= begin && i0 + E <= end) {
            *reinterpret_cast<uint4*>(x) = __ldg(reinterpret_cast<const uint4*>(base + i0));
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = i0 + e >= begin && i0 + e < end ? base[i0 + e] : T(-INFINITY);
        }
    }
    __device__ __forceinline__ void load(int c, uint32_t (&key)[E]) const {
        alignas(16) T x[E];
        if (smem)
            *reinterpret_cast<uint4*>(x) = reinterpret_cast<const uint4*>(smem)[c];
        else
            from_global(c, x);
#pragma unroll
        for (int e = 0; e < E; ++e) key[e] = order_key(as_float(x[e]));
    }
};

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
    v = s.warp[0];
#pragma unroll
    for (int i = 1; i < kSaWarps; ++i) v = s.warp[i] > v ? s.warp[i] : v;
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

template <typename T>
__global__ void __launch_bounds__(kSaThreads) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t sa_slice[];
    __shared__ SaShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int tid = threadIdx.x;
    const int r = blockIdx.x / C;
    constexpr int E = Row<T>::E;

    if (tid == 0) s.listed = 0;
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
    const float floor_d = least > 0.f ? logf(fminf(least, 1.f)) : -INFINITY;

    // exchange: every block's value to every block of the cluster
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

    // The maximum, its lowest index; the slice goes to shared memory on the way.
    u64 best = 0;
    if (a.resident) {
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            alignas(16) T x[E];
            row.from_global(c, x);
            reinterpret_cast<uint4*>(sa_slice)[c] = *reinterpret_cast<const uint4*>(x);
        }
        row.smem = sa_slice;    // each thread reads back its own chunks until the next barrier
    }
    for (int c = tid; c < row.chunks; c += kSaThreads) {
        uint32_t key[E];
        row.load(c, key);
        const int i0 = row.first(c);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const u64 v = ((u64)key[e] << 32) | (0xFFFFFFFFu - (uint32_t)(i0 + e));
            best = v > best ? v : best;
        }
    }
    best = cluster_max(best);
    const uint32_t top = (uint32_t)(best >> 32);
    const int first = (int)(0xFFFFFFFFu - (uint32_t)best);
    if (top <= kSaNone || !(temp > 0.f)) {     // nothing to choose from, or greedy
        if (rank == 0 && tid == 0) a.tokens[r] = top <= kSaNone ? -1 : first;
        return;
    }
    const float m = key_value(top);
    auto dist = [&](uint32_t key) { return key == top ? 0.f : (key_value(key) - m) / temp; };
    auto weight = [&](uint32_t key) { return (unsigned)rintf(expf(dist(key)) * kSaOne); };
    // (token score, lowest index) as one ordered integer
    auto race = [&](float d, int i) {
        return ((u64)order_key(d - logf(noise[i])) << 32) | (0xFFFFFFFFu - (uint32_t)i);
    };

    // ---------------------------------------------------------------- the cut
    // tokens whose weight rounds to nothing need no exponential
    const float tiny = temp * 25.f;
    auto add = [&](unsigned bin, uint32_t key) {
        atomicAdd(&s.hist[0][bin], 1u);
        if (!(m - key_value(key) > tiny)) {
            const unsigned w = weight(key);
            if (w & 0xFFFFu) atomicAdd(&s.hist[1][bin], w & 0xFFFFu);
            if (w >> 16) atomicAdd(&s.hist[2][bin], w >> 16);
        }
    };
    auto clear = [&]() {
        __syncthreads();
        for (int i = tid; i < 3 * kSaBins; i += kSaThreads) (&s.hist[0][0])[i] = 0;
        __syncthreads();
    };
    // The bin where the count (before `base` tokens) reaches kk, or where the weight (after
    // `base_w`) reaches the share p of `mass` (0: of the total found here). kk <= 0: by weight. A
    // count that is not reached turns into the search by weight.
    auto find = [&](int kk, int base, u64 base_w, u64 mass) {
        if (tid == 0) s.found.none = 1;
        cl.sync();
        const int sec = kSaBins / C, per = sec > kSaThreads ? sec / kSaThreads : 1;
        const int b0 = rank * sec + tid * per;
        const bool mine = tid * per < sec;
        unsigned cnt[kSaBins / kSaThreads];
        u64 wt[kSaBins / kSaThreads];
        u64 x = 0, y = 0, tx, ty;
#pragma unroll
        for (int i = 0; i < kSaBins / kSaThreads; ++i) {
            cnt[i] = 0;
            wt[i] = 0;
            if (mine && i < per) {
                for (int c = 0; c < C; ++c) {
                    const unsigned* h = C > 1 ? cl.map_shared_rank(&s.hist[0][0], c) : &s.hist[0][0];
                    cnt[i] += h[b0 + i];
                    wt[i] += ((u64)h[2 * kSaBins + b0 + i] << 16) + h[kSaBins + b0 + i];
                }
                x += cnt[i];
                y += wt[i];
            }
        }
        const u64 ox = x, oy = y;
        block_scan(x, y, tx, ty, s);
        x -= ox;
        y -= oy;
        u64 total = tx, total_w = ty;
        if (C > 1) {
            exchange(tx, ty);
            total = total_w = 0;
            for (int i = 0; i < C; ++i) {
                if (i < rank) {
                    x += s.part[turn][i];
                    y += s.part_w[turn][i];
                }
                total += s.part[turn][i];
                total_w += s.part_w[turn][i];
            }
        }
        x += base;
        y += base_w;
        const bool by_count = kk > 0 && (u64)kk <= base + total;
        double target = (double)p * (double)(mass ? mass : base_w + total_w);
        if (!(target >= 0.5)) target = 0.5;     // the first token is always kept
        if (by_count || p < 1.f) {
#pragma unroll
            for (int i = 0; i < kSaBins / kSaThreads; ++i) {
                if (mine && i < per && cnt[i] > 0 &&
                    (by_count ? x < (u64)kk && x + cnt[i] >= (u64)kk
                              : (double)y < target && (double)(y + wt[i]) >= target)) {
                    const Found f = {b0 + i, (int)x, (int)cnt[i], (int)(base + total), y, base_w + total_w, by_count, 0};
                    for (int c = 0; c < C; ++c) *cl.map_shared_rank(&s.found, c) = f;
                }
                x += cnt[i];
                y += wt[i];
            }
        }
        cl.sync();
        return s.found;
    };
    const float scale = (kSaBins / kSaRange) / fmaxf(temp, kSaLeastT);
    auto bin_of = [&](uint32_t key) {
        return key == top ? 0 : (int)fminf((m - key_value(key)) * scale, (float)(kSaBins - 1));
    };

    uint32_t cut = kSaNone + 1;    // kept: keys above `cut`, and the first `ties` tokens at it
    u64 ties = ~0ull;
    if ((k > 0 && k < a.V) || p < 1.f) {
        clear();
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            uint32_t key[E];
            row.load(c, key);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (key[e] > kSaNone) add(bin_of(key[e]), key[e]);
        }
        const Found f = find(k, 0, 0, 0);
        if (!f.none && f.before + f.count <= kSaList) {
            // ------------------------------------------------------------ few: one block settles the row
            for (int c = tid; c < row.chunks; c += kSaThreads) {
                uint32_t key[E];
                row.load(c, key);
                const int i0 = row.first(c);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (key[e] > kSaNone && bin_of(key[e]) <= f.bin) {
                        const unsigned at = atomicAdd(cl.map_shared_rank(&s.listed, 0), 1u);
                        cl.map_shared_rank(&s.list[0], 0)[at] = ((u64)key[e] << 32) | (0xFFFFFFFFu - (uint32_t)(i0 + e));
                    }
            }
            cl.sync();
            if (rank != 0) return;
            const int n = f.before + f.count;
            int size = 2;
            while (size < n) size *= 2;
            for (int i = tid; i < size; i += kSaThreads)
                if (i >= n) s.list[i] = 0;
            __syncthreads();
            for (int len = 2; len <= size; len *= 2)          // descending
                for (int d = len / 2; d > 0; d /= 2) {
                    for (int i = tid; i < size / 2; i += kSaThreads) {
                        const int lo = (i / d) * 2 * d + i % d, hi = lo + d;
                        const u64 u = s.list[lo], v = s.list[hi];
                        if ((u < v) == ((lo & len) == 0)) {
                            s.list[lo] = v;
                            s.list[hi] = u;
                        }
                    }
                    __syncthreads();
                }
            u64 v[2], w[2], x = 0, y = 0, tx, ty;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = 2 * tid + i;
                v[i] = at < n ? s.list[at] : 0;
                w[i] = at < n && (!f.by_count || at < k) ? weight((uint32_t)(v[i] >> 32)) : 0;
                y += w[i];
            }
            const u64 own = y;
            block_scan(x, y, tx, ty, s);
            y -= own;
            const double target = (double)p * (double)(f.by_count ? ty : f.total_w);
            best = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = 2 * tid + i;
                if (at < n) {
                    const float d = dist((uint32_t)(v[i] >> 32));
                    const bool kept = (!f.by_count || at < k) && (!(p < 1.f) || (double)y < target) && d >= floor_d;
                    if (kept || at == 0) {
                        const u64 c = race(d, (int)(0xFFFFFFFFu - (uint32_t)v[i]));
                        best = c > best ? c : best;
                    }
                }
                y += w[i];
            }
            best = block_max(best, s);
            if (tid == 0) a.tokens[r] = (int)(0xFFFFFFFFu - (uint32_t)best);
            return;
        }
        // ------------------------------------------------------------ many: refine the cut by the keys' bits
        // From the interval [lo, hi] of keys (tokens above: base, base_w) to one key.
        struct Cut {
            uint32_t key;
            int before, count;
            u64 before_w;
        };
        auto refine = [&](uint32_t lo, uint32_t hi, int kk, int base, u64 base_w, u64 mass, int count) {
            while (lo < hi) {
                const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
                clear();
                for (int c = tid; c < row.chunks; c += kSaThreads) {
                    uint32_t key[E];
                    row.load(c, key);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (key[e] >= lo && key[e] <= hi) add((hi - key[e]) >> shift, key[e]);
                }
                const Found g = find(kk, base, base_w, mass);
                if (g.none) break;             // cannot be: the interval holds the cut
                base = g.before;
                base_w = g.before_w;
                count = g.count;
                hi -= (uint32_t)g.bin << shift;
                const uint32_t low = hi - ((1u << shift) - 1);
                lo = low > lo && low <= hi ? low : lo;
            }
            return Cut{hi, base, count, base_w};
        };
        if (!f.none) {
            // the keys of the bin
            u64 high = 0, low = 0;
            for (int c = tid; c < row.chunks; c += kSaThreads) {
                uint32_t key[E];
                row.load(c, key);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (key[e] > kSaNone && bin_of(key[e]) == f.bin) {
                        high = key[e] > high ? key[e] : high;
                        low = (0xFFFFFFFFu - key[e]) > low ? (0xFFFFFFFFu - key[e]) : low;
                    }
            }
            high = cluster_max(high);
            low = cluster_max(low);
            u64 mass = f.by_count ? 0 : f.total_w;
            Cut g = refine(0xFFFFFFFFu - (uint32_t)low, (uint32_t)high, f.by_count ? k : 0, f.before, f.before_w, mass, f.count);
            cut = g.key;
            u64 w = weight(cut);
            if (f.by_count) {
                ties = (u64)(k - g.before);
                mass = g.before_w + ties * w;
                if (p < 1.f) g = refine(cut, top, 0, 0, 0, mass, 0);
            }
            if (p < 1.f) {
                // tokens at the key whose mass before is below the share
                double target = (double)p * (double)mass;
                if (!(target >= 0.5)) target = 0.5;
                w = weight(g.key);
                u64 t = 0;
                if (w > 0 && (double)g.before_w < target) {
                    t = (u64)((target - (double)g.before_w) / (double)w);
                    while (t > 0 && (double)(g.before_w + (t - 1) * w) >= target) --t;
                    while ((double)(g.before_w + t * w) < target) ++t;
                }
                if (g.key != cut || t < ties) ties = t;
                cut = g.key;
            }
        }
    }

    // ---------------------------------------------------------------- the race over the row
    // Tokens at the cut are counted in index order only if some of them fall out.
    best = 0;
    u64 seen = 0;
    bool ranked = false;
    if (ties != ~0ull) {
        u64 x = 0, y = 0, tx, ty;
        for (int c = tid; c < row.chunks; c += kSaThreads) {
            uint32_t key[E];
            row.load(c, key);
#pragma unroll
            for (int e = 0; e < E; ++e) x += key[e] == cut ? 1 : 0;
        }
        block_scan(x, y, tx, ty, s);
        if (C > 1) {
            exchange(tx, 0);
            tx = 0;
            for (int i = 0; i < C; ++i) {
                if (i < rank) seen += s.part[turn][i];
                tx += s.part[turn][i];
            }
        }
        ranked = tx > ties;
    }
    for (int c0 = 0; c0 < row.chunks; c0 += kSaThreads) {
        const int c = c0 + tid;
        uint32_t key[E];
        u64 x = 0, y = 0, tx, ty, own = 0;
        if (c < row.chunks) {
            row.load(c, key);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) key[e] = 0;
        }
        if (ranked) {
#pragma unroll
            for (int e = 0; e < E; ++e) own += key[e] == cut ? 1 : 0;
            x = own;
            block_scan(x, y, tx, ty, s);
            x += seen - own;                   // tokens at the cut before this chunk
            seen += tx;
        }
        const int i0 = row.first(c);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            bool kept = key[e] >= cut;
            if (ranked && key[e] == cut) kept = x++ < ties;
            if (kept) {
                const float d = dist(key[e]);
                if (d >= floor_d || i0 + e == first) {
                    const u64 v = race(d, i0 + e);
                    best = v > best ? v : best;
                }
            }
        }
    }
    best = cluster_max(best);
    if (rank == 0 && tid == 0) a.tokens[r] = (int)(0xFFFFFFFFu - (uint32_t)best);
}

template <typename T>
nq_status sample_launch(SampleArgs a, int B, const StepDevice& d, cudaStream_t stream) {
    auto kern = sample_kernel<T>;
    static thread_local int set_for_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (set_for_device != dev) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSaSliceBytes) != cudaSuccess)
            return NQ_ERR_CUDA;
        set_for_device = dev;
    }
    int C = kSaMaxCluster;
    a.slice = ((a.V + C - 1) / C + 15) / 16 * 16;
    const size_t bytes = ((size_t)a.slice * sizeof(T) + 15) / 16 * 16 + 16;
    a.resident = bytes <= (size_t)kSaSliceBytes;
    return step_launch(kern, dim3((unsigned)(B * C)), dim3(kSaThreads), a.resident ? bytes : 0, stream, d.pdl, C, a) ==
                   cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
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
    if (!logits || !noise || !tokens) return NQ_ERR_NULL;
    const int size = dtype == NQ_FP32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % size) return NQ_ERR_ALIGN;
    for (const void* p : {(const void*)noise, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                          (const void*)min_p, (const void*)tokens})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return NQ_ERR_ALIGN;
    const long long tb = B * 4ll;
    if (meet(tokens, tb, logits, ((B - 1) * stride + V) * size) || meet(tokens, tb, noise, ((B - 1) * noise_stride + V) * 4) ||
        meet(tokens, tb, temperature, tb) || meet(tokens, tb, top_k, tb) || meet(tokens, tb, top_p, tb) ||
        meet(tokens, tb, min_p, tb))
        return NQ_ERR_ALIAS;
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    SampleArgs a = {logits, stride, noise, noise_stride, temperature, top_k, top_p, min_p, tokens, V, 0, 0};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == NQ_BF16) return sample_launch<__nv_bfloat16>(a, B, d, s);
    if (dtype == NQ_FP16) return sample_launch<__half>(a, B, d, s);
    return sample_launch<float>(a, B, d, s);
}
