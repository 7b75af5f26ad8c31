// nq_moe.cu -- around the experts of a layer: which experts a token takes and where its rows lie (nq_moe_route), and
// the sum of their results (nq_moe_combine).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_fp8.h"
#include "nq_step.h"

namespace nq {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------- router

// Choice of experts: a warp a token, expert 32 v + lane in the lane's register v. Logits become whole numbers of
// the same order. The k-th largest of the lanes' largest is a bound below which nothing is chosen; what is not below it, a
// few more than k, goes to a lane each, which counts those before it. (A round a choice, each a search of all registers and two
// reductions, took 18 us for 16384 tokens x 256.) Where more than 32 are left (equal logits), rounds.
//
// With a bias the order is that of sigmoid(l) + b in 64 bits, which this GPU has few units for (an exponential takes a warp
// some 2 us). Values in 32 bits are off by less than half of kRtTol (1 + |value|): the fast exponential by 2^-22 and |l|
// 2^-23 of itself, which reach the sigmoid times s (1 - s) <= 1/4 and |l| s (1 - s) < 1/4, the quotient by 2^-22, the bias's
// addition by 2^-24 of the value: 2^-21 (1 + |value|) together. Only where neighbours among the chosen and the best of the others
// are nearer than kRtTol (1 + |value|) are the candidates settled in 64 bits; those near the bound are among them.
//
// Places: a stable counting sort by expert, by one cluster of blocks, each with a share of the tokens in order, cut
// into a run for each warp. Warps count their runs' choices, the blocks exchange their counts, and each warp goes through its
// run again, 32 choices at a time: a choice's place is its expert's next, plus those of the lanes before it with the same
// expert. No order of atomics shows. (Bit sets of tokens for each expert instead took 36 us for 16384 x 8 of 256.)
// Calls of few tokens choose and place in one launch.

constexpr int kRtThreads = 1024;
constexpr int kRtWarps = kRtThreads / 32;
// Blocks of the placing cluster: as many as are always there, or, for many tokens, 16 where the GPU takes such clusters
// (16384 x 8 of 256: 35.5 us with 8 blocks, 27.6 with 16).
constexpr int kRtCluster = 8, kRtClusterMany = 16;
constexpr int kRtMany = 4096;                    // tokens from which on
constexpr int kRtFew = 64;                       // tokens up to which one launch chooses and places
constexpr int kRtChooseThreads = 256;            // of a choosing block of a large call
constexpr int kRtMostChosen = 32;
constexpr int kRtMostTokens = 1 << 20;
constexpr float kRtTol = 0x1p-20f;

struct RouteArgs {
    const void* logits;
    long long stride;
    const float* bias;                           // sigmoid only; may be NULL
    int* ids;
    float* weights;
    int* offsets;
    int* rows;
    int* slots;
    int T, E, k;
    float scale;
    int dtype;
    bool sigmoid, normalize;
    int share;                                   // tokens of a block of the placing cluster
};

__device__ __forceinline__ float route_load(const void* p, long long i, int dtype) {
    if (dtype == NQ_FP32) return __ldg(static_cast<const float*>(p) + i);
    const uint16_t h = __ldg(static_cast<const unsigned short*>(p) + i);
    return dtype == NQ_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// A number that orders as f does (both zeros equal); 0, below all, for NaN and -inf.
__device__ __forceinline__ uint32_t route_key(float f) {
    if (!(f > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(f + 0.f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float route_value(uint32_t key) {
    return __uint_as_float((key >> 31) ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// sigmoid(l) + b in 64 bits as a whole number of the same order (0: not above -inf).
__device__ __noinline__ uint64_t route_key_64(float l, float b) {
    const double v = 1.0 / (1.0 + exp(-(double)l)) + (double)b;
    if (!(l > -INFINITY) || !(v > -INFINITY)) return 0;
    const uint64_t bits = (uint64_t)__double_as_longlong(v + 0.0);
    return (bits >> 63) ? ~bits : bits | (1ull << 63);
}

// The choice of one token in 64 bits among one candidate a lane (-1: none): lane j gets the j-th, or -1.
__device__ __forceinline__ int route_settle(const RouteArgs& a, long long row, int candidate) {
    const int lane = threadIdx.x & 31;
    uint64_t key = 0;
    if (candidate >= 0) key = route_key_64(route_load(a.logits, row + candidate, a.dtype), __ldg(a.bias + candidate));
    int rank = key ? 0 : 32;
    for (int i = 0; i < 32; ++i) {
        const uint64_t other = __shfl_sync(0xFFFFFFFFu, key, i);
        const int e = __shfl_sync(0xFFFFFFFFu, candidate, i);
        if (key && other && (other > key || (other == key && e < candidate))) ++rank;
    }
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        const unsigned who = __ballot_sync(0xFFFFFFFFu, rank == j);
        if (!who) break;
        const int e = __shfl_sync(0xFFFFFFFFu, candidate, __ffs(who) - 1);
        if (lane == j) mine = e;
    }
    return mine;
}

// The same among all experts, a round a choice: where more than 32 are near (with a bias: in 64 bits throughout).
template <int V>
__device__ __noinline__ int route_rounds(const RouteArgs& a, long long row) {
    const int lane = threadIdx.x & 31;
    uint32_t taken = 0;
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0;
        int at = -1;
        for (int v = 0; v < V; ++v) {
            const int e = 32 * v + lane;
            if (e >= a.E || ((taken >> v) & 1)) continue;
            const float l = route_load(a.logits, row + e, a.dtype);
            const uint64_t key = a.bias ? route_key_64(l, __ldg(a.bias + e)) : route_key(l);
            if (key > best) {
                best = key;
                at = e;
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const uint64_t key = __shfl_xor_sync(0xFFFFFFFFu, best, d);
            const int e = __shfl_xor_sync(0xFFFFFFFFu, at, d);
            if (e >= 0 && (at < 0 || key > best || (key == best && e < at))) {
                best = key;
                at = e;
            }
        }
        if (at < 0) break;
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        if (lane == j) mine = at;
    }
    return mine;
}

// A warp's shared memory: the lanes' largest, the candidates (key, expert), and in order.
struct RouteWarp {
    uint32_t largest[32];
    uint2 near[32], order[32];
};

// Chooses token t's experts and writes them with their weights.
template <int V>
__device__ __forceinline__ void route_choose(const RouteArgs& a, int t, RouteWarp& sm) {
    const int lane = threadIdx.x & 31;
    const long long row = (long long)t * a.stride;
    float l[V];
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 32 * v + lane;
        l[v] = e < a.E ? route_load(a.logits, row + e, a.dtype) : -INFINITY;
    }
    const bool biased = a.bias != nullptr;
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = 32 * v + lane;
        float f = l[v];
        if (biased && e < a.E && f > -INFINITY) f = __fdividef(1.f, 1.f + __expf(-f)) + __ldg(a.bias + e);
        key[v] = route_key(f);
        m = max(m, key[v]);
    }
    // the bound: as many lanes as are chosen (with a bias, one more) have something that is not below it
    const int want = biased ? a.k + 1 : a.k;
    sm.largest[lane] = m;
    __syncwarp();
    int before = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const uint4 o = *reinterpret_cast<const uint4*>(sm.largest + i);
        before += (o.x > m) + (o.y > m) + (o.z > m) + (o.w > m);
    }
    // (lanes with equal values count alike: the smallest of those with fewer than `want` before them)
    uint32_t bound = __reduce_min_sync(0xFFFFFFFFu, before < want ? m : 0xFFFFFFFFu);
    if (want > 32) bound = 0;
    if (biased && bound) {
        const float f = route_value(bound);
        bound = route_key(f - 2.f * kRtTol * (1.f + fabsf(f)));
    }
    bound = max(bound, 1u);
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const unsigned who = __ballot_sync(0xFFFFFFFFu, key[v] >= bound);
        const int at = n + __popc(who & ((1u << lane) - 1));
        if (key[v] >= bound && at < 32) sm.near[at] = make_uint2(key[v], 32 * v + lane);
        n += __popc(who);
    }
    __syncwarp();
    int mine = -1;                               // lane j: the j-th choice
    if (n <= 32) {
        const uint2 c = lane < n ? sm.near[lane] : make_uint2(0, 0);
        int rank = 0;
        for (int i = 0; i < n; ++i) {
            const uint2 o = sm.near[i];
            rank += o.x > c.x || (o.x == c.x && o.y < c.y);
        }
        if (lane < n) sm.order[rank] = c;
        __syncwarp();
        mine = lane < min(n, a.k) ? (int)sm.order[lane].y : -1;
        if (biased) {
            bool unsure = false;
            if (lane < a.k && lane + 1 < n) {
                const float hi = route_value(sm.order[lane].x), lo = route_value(sm.order[lane + 1].x);
                unsure = !(hi - lo > kRtTol * (1.f + fabsf(hi)));
            }
            if (__any_sync(0xFFFFFFFFu, unsure)) mine = route_settle(a, row, lane < n ? (int)c.y : -1);
        }
    } else {
        mine = route_rounds<V>(a, row);
    }
    __syncwarp();                                // the warp's next token uses the same memory
    // weights of the chosen
    const float c = mine >= 0 ? route_load(a.logits, row + mine, a.dtype) : -INFINITY;
    float w;
    if (a.sigmoid) {
        float top = c;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        // e^c / (1 + e^c) of a score below one half. Where only ratios count, all scores without the factor that the largest
        // has in e^c, so that those which fp32 cannot hold do not vanish.
        const float m = a.normalize ? fminf(top, 0.f) : 0.f;
        w = mine < 0 ? 0.f : (c > 0.f ? 1.f : expf(c - m)) / (1.f + expf(-fabsf(c)));
        if (a.normalize) {
            const float sum = warp_sum(w);
            if (mine >= 0) w = w / sum;
        }
    } else {
        const float top = __shfl_sync(0xFFFFFFFFu, c, 0);
        w = mine < 0 ? 0.f : (c == top ? 1.f : expf(c - top));
        float sum;
        if (a.normalize) {
            sum = warp_sum(w);
        } else {
            float part = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (l[v] > -INFINITY) part += l[v] == top ? 1.f : expf(l[v] - top);
            sum = warp_sum(part);
        }
        if (mine >= 0) w = w / sum;
    }
    if (lane < a.k) {
        a.ids[(long long)t * a.k + lane] = mine;
        a.weights[(long long)t * a.k + lane] = w * a.scale;
    }
}

// Places of the tokens' rows, by a cluster of blocks (see above). Shared memory: the block's counts [E], and of each
// warp its counts and then next places [warps][E].
constexpr int kRtOnce = 8;                       // choices of a lane that are loaded at once
__device__ __forceinline__ void route_place(const RouteArgs& a, int* sm) {
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), blocks = (int)cl.num_blocks(), tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    int* const count = sm;
    int* const next = sm + a.E;
    int* const my_next = next + warp * a.E;
    __shared__ int warp_total[kRtWarps];
    const int t0 = min(a.T, rank * a.share), t1 = min(a.T, t0 + a.share);
    // the warp's run of tokens
    const int run = (a.share + kRtWarps - 1) / kRtWarps;
    const int r0 = min(t1, t0 + warp * run) * a.k, r1 = min(t1, t0 + (warp + 1) * run) * a.k;
    for (int i = tid; i < kRtWarps * a.E; i += kRtThreads) next[i] = 0;
    __syncthreads();
    int e[kRtOnce];
    for (int b0 = r0; b0 < r1; b0 += 32 * kRtOnce) {
#pragma unroll
        for (int j = 0; j < kRtOnce; ++j) e[j] = b0 + 32 * j + lane < r1 ? a.ids[b0 + 32 * j + lane] : -1;
#pragma unroll
        for (int j = 0; j < kRtOnce; ++j)
            if (e[j] >= 0) atomicAdd(my_next + e[j], 1);
    }
    const bool once = r1 - r0 <= 32 * kRtOnce;   // then e still has them below
    __syncthreads();
    // (at most 512 experts, one a thread)
    if (tid < a.E) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < kRtWarps; ++w) sum += next[w * a.E + tid];
        count[tid] = sum;
    }
    cl.sync();
    // experts' totals and the rows of the blocks before this one
    int mine = 0, ahead = 0;
    if (tid < a.E)
        for (int b0 = 0; b0 < blocks; b0 += 8) {
            int c[8];                            // (loads in flight together)
#pragma unroll
            for (int b = 0; b < 8; ++b) c[b] = b0 + b < blocks ? *cl.map_shared_rank(count + tid, b0 + b) : 0;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (b0 + b < rank) ahead += c[b];
                mine += c[b];
            }
        }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, d);
        if (lane >= d) upto += u;
    }
    if (lane == 31) warp_total[warp] = upto;
    __syncthreads();
    int base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kRtWarps; ++w) {
        const int c = warp_total[w];
        if (w < warp) base += c;
        all += c;
    }
    if (tid < a.E) {
        int at = base + upto - mine;
        if (rank == 0) {
            a.offsets[tid] = at;
            if (tid == a.E - 1) a.offsets[a.E] = all;
        }
        at += ahead;
#pragma unroll 8
        for (int w = 0; w < kRtWarps; ++w) {
            const int c = next[w * a.E + tid];
            next[w * a.E + tid] = at;
            at += c;
        }
    }
    // the entries behind the last row
    for (int i = all + rank * kRtThreads + tid; i < a.T * a.k; i += blocks * kRtThreads) a.rows[i] = -1;
    __syncthreads();
    for (int b0 = r0; b0 < r1; b0 += 32 * kRtOnce) {
        if (!once)
#pragma unroll
            for (int j = 0; j < kRtOnce; ++j) e[j] = b0 + 32 * j + lane < r1 ? a.ids[b0 + 32 * j + lane] : -1;
#pragma unroll
        for (int j = 0; j < kRtOnce; ++j) {
            const int i = b0 + 32 * j + lane;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, e[j]);
            int at = -1;
            if (e[j] >= 0) at = my_next[e[j]] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (e[j] >= 0) {
                if ((same >> lane) == 1) my_next[e[j]] = at + 1;     // the last of the same
                a.rows[at] = i / a.k;
            }
            __syncwarp();
            if (i < r1) a.slots[i] = at;
        }
    }
    cl.sync();                                   // no block leaves while another reads its counts
}

template <int V>
__global__ void __launch_bounds__(kRtChooseThreads) route_choose_kernel(const RouteArgs a) {
    __shared__ __align__(16) RouteWarp sm[kRtChooseThreads / 32];
    const int warp = threadIdx.x >> 5, t = blockIdx.x * (kRtChooseThreads / 32) + warp;
    grid_launch_dependents();
    grid_dependency_wait();
    if (t < a.T) route_choose<V>(a, t, sm[warp]);
}

template <int V>
__global__ void __launch_bounds__(kRtThreads, 1) route_few_kernel(const RouteArgs a) {
    extern __shared__ int route_smem[];
    __shared__ __align__(16) RouteWarp sm[kRtWarps];
    const int rank = (int)cluster_rank(), warp = threadIdx.x >> 5;
    grid_launch_dependents();
    grid_dependency_wait();
    const int t0 = min(a.T, rank * a.share), t1 = min(a.T, t0 + a.share);
    for (int t = t0 + warp; t < t1; t += kRtWarps) route_choose<V>(a, t, sm[warp]);
    __syncthreads();
    route_place(a, route_smem);
}

__global__ void __launch_bounds__(kRtThreads, 1) route_place_kernel(const RouteArgs a) {
    extern __shared__ int route_smem[];
    grid_launch_dependents();
    grid_dependency_wait();
    route_place(a, route_smem);
}

// Whether a cluster of kRtClusterMany blocks can run (queried once a device, which allows them there).
constexpr int kDevices = 64;
bool route_wide_clusters() {
    static std::once_flag once[kDevices];
    static int most[kDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return false;
    int& n = most[dev];
    std::call_once(once[dev], [&n] {
        if (cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (kRtWarps + 1) * kMostExperts * 4) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kRtClusterMany);
        cfg.blockDim = dim3(kRtThreads);
        cfg.dynamicSmemBytes = (kRtWarps + 1) * kMostExperts * 4;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kRtClusterMany;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, route_place_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    });
    return n > 0;
}

template <int V>
cudaError_t route_launch(RouteArgs a, cudaStream_t stream, bool pdl) {
    const bool few = a.T <= kRtFew;
    int blocks = few ? (a.T + kRtWarps - 1) / kRtWarps : min(kRtCluster, (a.T + kRtWarps - 1) / kRtWarps);
    if (a.T >= kRtMany && route_wide_clusters()) blocks = kRtClusterMany;
    a.share = (a.T + blocks - 1) / blocks;
    const size_t smem = (size_t)(kRtWarps + 1) * a.E * 4;
    const void* kern = few ? (const void*)route_few_kernel<V> : (const void*)route_place_kernel;
    if (smem > 24 * 1024) {
        static thread_local int set_for_device[2] = {-1, -1};
        int dev = 0;
        cudaGetDevice(&dev);
        if (set_for_device[few] != dev) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (kRtWarps + 1) * kMostExperts * 4);
            if (e != cudaSuccess) return e;
            set_for_device[few] = dev;
        }
    }
    if (few) return step_launch(route_few_kernel<V>, dim3(blocks), dim3(kRtThreads), smem, stream, pdl, blocks, a);
    const int per = kRtChooseThreads / 32;
    const cudaError_t e = step_launch(route_choose_kernel<V>, dim3((a.T + per - 1) / per), dim3(kRtChooseThreads), 0, stream,
                                      pdl, 1, a);
    if (e != cudaSuccess) return e;
    return step_launch(route_place_kernel, dim3(blocks), dim3(kRtThreads), smem, stream, pdl, blocks, a);
}

// ---------------------------------------------------------------- combination

// A thread a token's 8 columns: its k rows' loads are in flight together; the sum is fp32, in the order of the choices.
// Bound by memory: each row of y once.

constexpr int kCbThreads = 128;
constexpr int kCbRows = 4;                       // rows whose loads are in flight together

struct CombineArgs {
    const uint8_t* y;
    const int* slots;
    const float* weights;
    const uint8_t* base;
    uint8_t* out;
    long long y_stride, base_stride, out_stride; // bytes
    int M, T, k, N;
    uint32_t segments;                           // blocks of kCbThreads x 8 columns in a row
};

template <bool BF16>
__device__ __forceinline__ void add_eight(float (&sum)[8], uint4 v, float w) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 p;
        if constexpr (BF16) {
            p.x = __uint_as_float(x[i] << 16);
            p.y = __uint_as_float(x[i] & 0xFFFF0000u);
        } else {
            p = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
        }
        sum[2 * i] = fmaf(w, p.x, sum[2 * i]);
        sum[2 * i + 1] = fmaf(w, p.y, sum[2 * i + 1]);
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kCbThreads) combine_kernel(const CombineArgs a) {
    const int t = (int)(blockIdx.x / a.segments);
    const int col = ((int)(blockIdx.x - (uint32_t)t * a.segments) * kCbThreads + threadIdx.x) * 8;
    grid_launch_dependents();
    grid_dependency_wait();
    if (col >= a.N) return;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4 base;
    if (a.base) base = *reinterpret_cast<const uint4*>(a.base + t * a.base_stride + col * 2);
    for (int j0 = 0; j0 < a.k; j0 += kCbRows) {
        uint4 v[kCbRows];
        float w[kCbRows];
#pragma unroll
        for (int j = 0; j < kCbRows; ++j) {
            w[j] = 0.f;
            v[j] = make_uint4(0, 0, 0, 0);
            if (j0 + j < a.k) {
                const int slot = __ldg(a.slots + (long long)t * a.k + j0 + j);
                if (slot >= 0 && slot < a.M) {
                    w[j] = __ldg(a.weights + (long long)t * a.k + j0 + j);
                    v[j] = __ldg(reinterpret_cast<const uint4*>(a.y + slot * a.y_stride + col * 2));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kCbRows; ++j) add_eight<BF16>(sum, v[j], w[j]);
    }
    if (a.base) add_eight<BF16>(sum, base, 1.f);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(sum[2 * i], sum[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __half2 p = __floats2half2_rn(sum[2 * i], sum[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    *reinterpret_cast<uint4*>(a.out + t * a.out_stride + col * 2) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace
}  // namespace nq

using namespace nq;

extern "C" {

nq_status nq_moe_route(const void* logits, int dtype, long long stride, const float* bias, int T, int E, int k,
                       int score, int normalize, float scale, int* ids, float* weights, int* offsets, int* rows,
                       int* slots, void* stream) {
    if (dtype != NQ_BF16 && dtype != NQ_FP16 && dtype != NQ_FP32) return NQ_ERR_SHAPE;
    if (T < 0 || T > kRtMostTokens || E < 1 || E > kMostExperts || k < 1 || k > E || k > kRtMostChosen) return NQ_ERR_SHAPE;
    if ((score != NQ_SOFTMAX && score != NQ_SIGMOID) || (bias && score != NQ_SIGMOID)) return NQ_ERR_SHAPE;
    if (stride < E || !(scale > 0.f) || !(scale < INFINITY)) return NQ_ERR_SHAPE;
    if (T == 1) stride = E;
    const int el = dtype == NQ_FP32 ? 4 : 2;
    const long long lb = step_span(T, stride, E) * el, n = (long long)T * k * 4;
    if (lb < 0) return NQ_ERR_SHAPE;
    if (!offsets) return NQ_ERR_NULL;
    if (mis(offsets, 4)) return NQ_ERR_ALIGN;
    if (T > 0) {
        if (!logits || !ids || !weights || !rows || !slots) return NQ_ERR_NULL;
        if (mis(logits, el) || mis(bias, 4) || mis(ids, 4) || mis(weights, 4) || mis(rows, 4) || mis(slots, 4))
            return NQ_ERR_ALIGN;
    }
    const struct {
        const void* p;
        long long n;
    } out[] = {{ids, n}, {weights, n}, {rows, n}, {slots, n}, {offsets, (E + 1) * 4ll}};
    for (int i = 0; i < 5; ++i) {
        if (meet(out[i].p, out[i].n, logits, lb) || meet(out[i].p, out[i].n, bias, E * 4ll)) return NQ_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return NQ_ERR_ALIAS;
    }
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) return cudaMemsetAsync(offsets, 0, (E + 1) * 4, s) == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
    RouteArgs a;
    a.logits = logits;
    a.stride = stride;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    a.T = T;
    a.E = E;
    a.k = k;
    a.scale = scale;
    a.dtype = dtype;
    a.sigmoid = score == NQ_SIGMOID;
    a.normalize = normalize != 0;
    const cudaError_t e = E <= 32    ? route_launch<1>(a, s, d.pdl)
                          : E <= 64  ? route_launch<2>(a, s, d.pdl)
                          : E <= 128 ? route_launch<4>(a, s, d.pdl)
                          : E <= 256 ? route_launch<8>(a, s, d.pdl)
                                     : route_launch<16>(a, s, d.pdl);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

nq_status nq_moe_combine(const void* y, int dtype, long long y_stride, int M, const int* slots, const float* weights,
                         int T, int k, int N, const void* base, long long base_stride, void* out, long long out_stride,
                         void* stream) {
    if (dtype != NQ_BF16 && dtype != NQ_FP16) return NQ_ERR_SHAPE;
    if (M < 0 || M > kFp8MostRows || T < 0 || T > kRtMostTokens || k < 1 || k > kRtMostChosen) return NQ_ERR_SHAPE;
    if (N < 8 || N % 8 || N > kFp8MostCols || y_stride < N || out_stride < N || (base && base_stride < N)) return NQ_ERR_SHAPE;
    if (M <= 1) y_stride = N;                    // between rows: nothing
    if (T == 1) base_stride = out_stride = N;
    const long long yb = 2 * step_span(M, y_stride, N), bb = base ? 2 * step_span(T, base_stride, N) : 0;
    const long long ob = 2 * step_span(T, out_stride, N), n = (long long)T * k * 4;
    if (yb < 0 || bb < 0 || ob < 0) return NQ_ERR_SHAPE;
    if (T == 0) return NQ_OK;
    if ((M > 0 && !y) || !slots || !weights || !out) return NQ_ERR_NULL;
    if (mis(y, 16) || mis(base, 16) || mis(out, 16) || y_stride % 8 || out_stride % 8 || (base && base_stride % 8) ||
        mis(slots, 4) || mis(weights, 4))
        return NQ_ERR_ALIGN;
    // out may be base itself: each of its elements is read by the thread that writes it
    const bool same = base == out && base_stride == out_stride;
    if (meet(out, ob, y, yb) || meet(out, ob, slots, n) || meet(out, ob, weights, n) || (!same && meet(out, ob, base, bb)))
        return NQ_ERR_ALIAS;
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    CombineArgs a;
    a.y = static_cast<const uint8_t*>(y);
    a.slots = slots;
    a.weights = weights;
    a.base = static_cast<const uint8_t*>(base);
    a.out = static_cast<uint8_t*>(out);
    a.y_stride = y_stride * 2;
    a.base_stride = base_stride * 2;
    a.out_stride = out_stride * 2;
    a.M = M;
    a.T = T;
    a.k = k;
    a.N = N;
    a.segments = (uint32_t)((N / 8 + kCbThreads - 1) / kCbThreads);
    const long long blocks = (long long)T * a.segments;
    if (blocks > 0x7FFFFFFFll) return NQ_ERR_SHAPE;
    auto kern = dtype == NQ_BF16 ? combine_kernel<true> : combine_kernel<false>;
    return step_launch(kern, dim3((unsigned)blocks), dim3(kCbThreads), 0, reinterpret_cast<cudaStream_t>(stream), d.pdl, 1,
                       a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // extern "C"
