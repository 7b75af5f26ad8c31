// nq_pages.cu -- the paged KV cache's bookkeeping: block tables and slot maps built on the GPU
// from request lengths (nq_page_tables), and the store of new keys and values through the slot
// map (nq_kv_append).
#include <cuda_runtime.h>

#include <cstdint>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_launch.h"
#include "nq_step.h"

namespace nq {

namespace {

constexpr int kPtThreads = 1024;
constexpr int kPtTokensPerBlock = 1024;   // one token a thread until the grid is full
constexpr int kPtMaxRequests = 8192;      // two scans of 4 bytes a request stay in shared memory

struct PageArgs {
    const int* lens;
    const int* new_lens;
    const int* free_blocks;
    const int* num_free;
    int* table;
    long long table_stride;
    int* q_start;
    int* kv_lens;
    int* positions;
    long long* slots;
    int* counts;
    int R, free_capacity, page_shift, max_blocks, max_tokens;
};

// One request's share, from its lengths: whether they are usable, its clipped token count and
// the blocks it needs beyond those it owns.
struct PageNeed {
    int old, n, owned, need;
    bool valid;
};

__device__ __forceinline__ PageNeed page_need(const PageArgs& a, int r) {
    PageNeed p;
    p.old = a.lens[r];
    const int n = a.new_lens[r];
    p.n = n > 0 ? n : 0;
    const int mask = (1 << a.page_shift) - 1;
    const long long end = (long long)p.old + p.n;
    // (positions are 32-bit: a table may be wide enough for more)
    p.valid = p.old >= 0 && n >= 0 && end <= min((long long)a.max_blocks << a.page_shift, 0x7FFFFFFFll);
    p.owned = p.valid ? (int)(((long long)p.old + mask) >> a.page_shift) : 0;
    p.need = p.valid ? (int)((end + mask) >> a.page_shift) - p.owned : 0;
    return p;
}

// Inclusive scan of two values over the block (kPtThreads threads).
__device__ __forceinline__ void block_scan2(long long& x, int& y, long long* wx, int* wy) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long ux = __shfl_up_sync(0xFFFFFFFFu, x, d);
        const int uy = __shfl_up_sync(0xFFFFFFFFu, y, d);
        if (lane >= d) {
            x += ux;
            y += uy;
        }
    }
    if (lane == 31) {
        wx[warp] = x;
        wy[warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
        long long sx = wx[lane];
        int sy = wy[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const long long ux = __shfl_up_sync(0xFFFFFFFFu, sx, d);
            const int uy = __shfl_up_sync(0xFFFFFFFFu, sy, d);
            if (lane >= d) {
                sx += ux;
                sy += uy;
            }
        }
        wx[lane] = sx;
        wy[lane] = sy;
    }
    __syncthreads();
    if (warp > 0) {
        x += wx[warp - 1];
        y += wy[warp - 1];
    }
}

// Every block scans all requests by itself (a few thousand lengths at most: cheaper than a
// second launch or a wait between blocks) and then writes its own share of the tokens and of
// the per-request outputs. No block reads what another writes: a token that lies in a block the
// request owned before reads that entry of the table, which nobody changes; the entries added
// now are computed from the free list by every reader, and written by the thread of the token
// that begins the block.
__global__ void __launch_bounds__(kPtThreads) page_tables_kernel(const PageArgs a) {
    extern __shared__ int pt_smem[];
    __shared__ long long wx[32];
    __shared__ int wy[32];
    __shared__ long long carry_x;
    __shared__ int carry_y;
    int* const t_end = pt_smem;            // tokens up to and with request r, clipped
    int* const b_end = pt_smem + a.R;      // blocks asked for up to and with request r
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x;
    const int num_free = min(*a.num_free, a.free_capacity);
    long long base_x = 0;
    int base_y = 0;
    for (int r0 = 0; r0 < a.R; r0 += kPtThreads) {
        const int r = r0 + tid;
        PageNeed p = {0, 0, 0, 0, false};
        if (r < a.R) p = page_need(a, r);
        long long x = p.n;
        int y = 0;
        block_scan2(x, y, wx, wy);
        x += base_x;
        // a request whose last token would lie past the token buffers asks for nothing
        const bool valid = p.valid && x <= a.max_tokens;
        __syncthreads();
        long long dummy = 0;
        y = valid ? p.need : 0;
        block_scan2(dummy, y, wx, wy);
        y += base_y;                       // <= tokens / 16 + requests: far from overflow
        if (r < a.R) {
            t_end[r] = (int)(x < a.max_tokens ? x : a.max_tokens);
            // the top bit marks a request that is not valid
            b_end[r] = valid ? y : (y | (int)0x80000000);
        }
        if (tid == kPtThreads - 1) {
            carry_x = x;
            carry_y = y;
        }
        __syncthreads();
        base_x = carry_x;
        base_y = carry_y;
    }
    __syncthreads();

    // Per request: admitted when its blocks, counted in order, are within the free list.
    auto asked = [&](int r) { return r < 0 ? 0 : b_end[r] & 0x7FFFFFFF; };
    auto admitted = [&](int r) {
        return b_end[r] >= 0 && (b_end[r] == asked(r - 1) || b_end[r] <= num_free);
    };
    const int stride = gridDim.x * kPtThreads;
    for (int r = blockIdx.x * kPtThreads + tid; r < a.R; r += stride) {
        a.q_start[r + 1] = t_end[r];
        a.kv_lens[r] = admitted(r) ? a.lens[r] + a.new_lens[r] : 0;
        if (r == 0) a.q_start[0] = 0;
    }
    if (blockIdx.x == 0) {
        // totals: the admitted requests that take blocks are those of a prefix of the counts
        int refused = 0, taken = 0;
        for (int r = tid; r < a.R; r += kPtThreads) {
            const bool ok = admitted(r);
            refused += ok ? 0 : 1;
            if (ok && b_end[r] > asked(r - 1)) taken = b_end[r];
        }
        taken = __reduce_max_sync(0xFFFFFFFFu, taken);
        refused = __reduce_add_sync(0xFFFFFFFFu, refused);
        __syncthreads();
        if ((tid & 31) == 0) {
            wx[tid >> 5] = taken;
            wy[tid >> 5] = refused;
        }
        __syncthreads();
        if (tid < 32) {
            const int tk = __reduce_max_sync(0xFFFFFFFFu, (int)wx[tid]);
            const int rf = __reduce_add_sync(0xFFFFFFFFu, wy[tid]);
            if (tid == 0) {
                a.counts[0] = t_end[a.R - 1];
                a.counts[1] = tk;
                a.counts[2] = rf;
            }
        }
    }

    // Tokens: each finds its request by bisection of the scan.
    const int total = t_end[a.R - 1], mask = (1 << a.page_shift) - 1;
    for (int t = blockIdx.x * kPtThreads + tid; t < a.max_tokens; t += stride) {
        int pos = -1;
        long long slot = -1;
        if (t < total) {
            int lo = 0, hi = a.R - 1;      // the first request whose end passes t
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (t_end[mid] > t)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            const int r = lo;
            if (admitted(r)) {
                const int old = a.lens[r];
                const int owned = (int)(((long long)old + mask) >> a.page_shift);
                pos = old + t - (r > 0 ? t_end[r - 1] : 0);
                const int b = pos >> a.page_shift;
                int* entry = a.table + r * a.table_stride + b;
                int id;
                if (b < owned) {
                    id = *entry;
                } else {
                    id = a.free_blocks[asked(r - 1) + b - owned];
                    if ((pos & mask) == 0) *entry = id;
                }
                slot = ((long long)id << a.page_shift) + (pos & mask);
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
}

// ---------------------------------------------------------------- KV append

struct AppendArgs {
    const uint4* k;
    const uint4* v;
    long long k_stride, v_stride;          // between tokens, in 16-byte chunks
    const long long* slots;
    uint4* kc;
    uint4* vc;
    long long block_stride, row_stride, head_stride;   // of the caches, in 16-byte chunks
    long long num_slots;
    int tokens, page_shift, head_shift;    // head_shift: log2 of a head's 16-byte chunks
    int row_chunks;                        // a token's 16-byte chunks of K (or of V)
};

constexpr int kApThreads = 256;
constexpr int kApChunks = 4;               // loads in flight a thread

// A pure copy, bound by memory: a warp takes the K or the V row of a token, kApChunks 16-byte loads a
// lane before the first store. (Chunks numbered over the whole call cost a division each and kept
// the issue slots busy: 16381 tokens of 8 x 128 22.5 us, so 19.5: 6.75 TB/s.)
__global__ void __launch_bounds__(kApThreads) kv_append_kernel(const AppendArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long row = (long long)blockIdx.x * (kApThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long t = row >> 1;
    if (t >= a.tokens) return;
    const bool is_v = row & 1;
    const long long slot = a.slots[t];
    if (slot < 0 || slot >= a.num_slots) return;
    const uint4* const src = is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride;
    uint4* const dst = (is_v ? a.vc : a.kc) + (slot >> a.page_shift) * a.block_stride +
                       (slot & ((1 << a.page_shift) - 1)) * a.row_stride;
    for (int c0 = lane; c0 < a.row_chunks; c0 += 32 * kApChunks) {
        uint4 val[kApChunks];
#pragma unroll
        for (int i = 0; i < kApChunks; ++i)
            if (c0 + 32 * i < a.row_chunks) val[i] = __ldg(src + c0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kApChunks; ++i) {
            const int c = c0 + 32 * i;
            if (c < a.row_chunks) dst[(c >> a.head_shift) * a.head_stride + (c & ((1 << a.head_shift) - 1))] = val[i];
        }
    }
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

bool meet(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace

int check_kv_cache(const nq_kv_cache* c) {
    if (!c) return NQ_ERR_NULL;
    if (c->num_blocks < 0 || c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) != 0) return NQ_ERR_SHAPE;
    if ((c->dim != 64 && c->dim != 128 && c->dim != 256) || c->heads < 1 || c->heads > 1024) return NQ_ERR_SHAPE;
    if (c->num_blocks > (1 << 28)) return NQ_ERR_SHAPE;
    if (c->block_stride < c->dim || c->row_stride < c->dim || c->head_stride < c->dim ||
        c->block_stride >= (1ll << 38) || c->row_stride >= (1ll << 38) || c->head_stride >= (1ll << 38))
        return NQ_ERR_SHAPE;
    if (c->num_blocks == 0) return NQ_OK;
    if (step_span(c->num_blocks, c->block_stride,
                  step_span(c->page, c->row_stride, step_span(c->heads, c->head_stride, c->dim))) < 0)
        return NQ_ERR_SHAPE;
    if (!c->K || !c->V) return NQ_ERR_NULL;
    if (mis16(c->K) || mis16(c->V) || c->block_stride % 8 || c->row_stride % 8 || c->head_stride % 8)
        return NQ_ERR_ALIGN;
    return NQ_OK;
}

long long kv_cache_span(const nq_kv_cache* c) {
    return 2 * step_span(c->num_blocks, c->block_stride,
                         step_span(c->page, c->row_stride, step_span(c->heads, c->head_stride, c->dim)));
}

}  // namespace nq

using namespace nq;

extern "C" {

nq_status nq_page_tables(const int* lens, const int* new_lens, int R, const int* free_blocks, int free_capacity,
                         const int* num_free, int page, int* block_table, long long table_stride, int max_blocks, int* q_start,
                         int* kv_lens, int* positions, int64_t* slots, int max_tokens, int* counts, void* stream) {
    if (R < 0 || R > kPtMaxRequests || free_capacity < 0 || max_tokens < 0 || max_tokens > (1 << 28) || max_blocks < 0 ||
        max_blocks > (1 << 24) || table_stride < max_blocks || page < 16 || page > 256 || (page & (page - 1)) != 0)
        return NQ_ERR_SHAPE;
    if (R == 0 && max_tokens == 0) return NQ_OK;
    if (R == 0) return NQ_ERR_SHAPE;   // tokens without requests
    const long long table_span = max_blocks > 0 ? step_span(R, table_stride, max_blocks) : 0;
    if (table_span < 0) return NQ_ERR_SHAPE;
    if (!lens || !new_lens || (free_capacity > 0 && !free_blocks) || !num_free || !q_start || !kv_lens || !counts ||
        (max_blocks > 0 && !block_table) || (max_tokens > 0 && (!positions || !slots)))
        return NQ_ERR_NULL;
    const void* ptrs[] = {lens, new_lens, free_blocks, num_free, block_table, q_start, kv_lens, positions, slots, counts};
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % (p == slots ? 8 : 4) != 0) return NQ_ERR_ALIGN;
    struct {
        const void* p;
        long long n;
    } out[] = {{block_table, table_span * 4},
               {q_start, (R + 1) * 4ll},
               {kv_lens, R * 4ll},
               {positions, max_tokens * 4ll},
               {slots, max_tokens * 8ll},
               {counts, 12}},
      in[] = {{lens, R * 4ll}, {new_lens, R * 4ll}, {free_blocks, free_capacity * 4ll}, {num_free, 4}};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 4; ++j)
            if (meet(out[i].p, out[i].n, in[j].p, in[j].n)) return NQ_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return NQ_ERR_ALIAS;
    }
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    PageArgs a;
    a.lens = lens;
    a.new_lens = new_lens;
    a.free_blocks = free_blocks;
    a.num_free = num_free;
    a.free_capacity = free_capacity;
    a.table = block_table;
    a.table_stride = table_stride;
    a.q_start = q_start;
    a.kv_lens = kv_lens;
    a.positions = positions;
    a.slots = reinterpret_cast<long long*>(slots);
    a.counts = counts;
    a.R = R;
    a.page_shift = log2_of(page);
    a.max_blocks = max_blocks;
    a.max_tokens = max_tokens;
    const int want = (max_tokens + kPtTokensPerBlock - 1) / kPtTokensPerBlock;
    const int grid = want < 1 ? 1 : (want < d.sms ? want : d.sms);
    const size_t smem = (size_t)R * 8;
    if (smem > 40 * 1024) {
        static thread_local int set_for_device = -1;
        int dev = 0;
        cudaGetDevice(&dev);
        if (set_for_device != dev) {
            if (cudaFuncSetAttribute(page_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kPtMaxRequests * 8) != cudaSuccess)
                return NQ_ERR_CUDA;
            set_for_device = dev;
        }
    }
    return step_launch(page_tables_kernel, dim3(grid), dim3(kPtThreads), smem, reinterpret_cast<cudaStream_t>(stream),
                       d.pdl, 1, a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

nq_status nq_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const int64_t* slots,
                       int tokens, const nq_kv_cache* cache, void* stream) {
    int st = check_kv_cache(cache);
    if (st != NQ_OK) return st;
    const long long row = (long long)cache->heads * cache->dim;
    if (tokens < 0 || tokens > (1 << 28) || k_stride < row || v_stride < row) return NQ_ERR_SHAPE;
    const long long kb = 2 * step_span(tokens, k_stride, row), vb = 2 * step_span(tokens, v_stride, row);
    if (kb < 0 || vb < 0) return NQ_ERR_SHAPE;
    if (tokens == 0 || cache->num_blocks == 0) return NQ_OK;
    if (!k || !v || !slots) return NQ_ERR_NULL;
    if (mis16(k) || mis16(v) || k_stride % 8 || v_stride % 8 || (reinterpret_cast<uintptr_t>(slots) & 7u))
        return NQ_ERR_ALIGN;
    const long long span = kv_cache_span(cache);
    for (const void* c : {(const void*)cache->K, (const void*)cache->V})
        if (meet(c, span, k, kb) || meet(c, span, v, vb) || meet(c, span, slots, tokens * 8ll)) return NQ_ERR_ALIAS;
    StepDevice d;
    st = step_device(&d);
    if (st != NQ_OK) return st;
    AppendArgs a;
    a.k = static_cast<const uint4*>(k);
    a.v = static_cast<const uint4*>(v);
    a.k_stride = k_stride / 8;
    a.v_stride = v_stride / 8;
    a.slots = reinterpret_cast<const long long*>(slots);
    a.kc = static_cast<uint4*>(cache->K);
    a.vc = static_cast<uint4*>(cache->V);
    a.block_stride = cache->block_stride / 8;
    a.row_stride = cache->row_stride / 8;
    a.head_stride = cache->head_stride / 8;
    a.page_shift = log2_of(cache->page);
    a.num_slots = (long long)cache->num_blocks << a.page_shift;
    a.tokens = tokens;
    a.head_shift = log2_of(cache->dim / 8);
    a.row_chunks = (int)(row / 8);
    const long long grid = (2ll * tokens + kApThreads / 32 - 1) / (kApThreads / 32);
    return step_launch(kv_append_kernel, dim3((unsigned)grid), dim3(kApThreads), 0,
                       reinterpret_cast<cudaStream_t>(stream), d.pdl, 1, a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // extern "C"
