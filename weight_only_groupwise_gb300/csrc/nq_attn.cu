// Instantiations and host side of the paged attention call (nq_attn.cuh): argument checks, the
// caches' tensor maps and the two launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "nq.h"
#include "nq_attn.cuh"
#include "nq_launch.h"

namespace nq {

int check_kv_cache(const nq_kv_cache* c);
long long kv_cache_span(const nq_kv_cache* c);

namespace {

template <int D, bool BF16, bool PAIR>
cudaError_t attn_launch(const AttnArgs& a, int blocks, bool splits, cudaStream_t stream, bool pdl) {
    auto kern = attn_kernel<D, BF16, PAIR>;
    static thread_local int set_for_device = -1;
    int dev = 0;
    cudaGetDevice(&dev);
    if (set_for_device != dev) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, AttnGeo<D, PAIR>::kSmem);
        if (e != cudaSuccess) return e;
        set_for_device = dev;
    }
    cudaError_t e = step_launch(kern, dim3(blocks), dim3(kAttnThreads), AttnGeo<D, PAIR>::kSmem, stream, pdl && !PAIR,
                                PAIR ? 2 : 1, a);
    if (e != cudaSuccess || !splits) return e;
    // a block takes 32 items of a split with many parts. Its launch follows the exit of the attention
    // kernel's blocks, which do not ask for it themselves: join blocks that wait beside working ones slow them. One
    // token over 4100 keys, in a stream and in a graph: 15.5 and 15.2 us so, 18.0 and 15.4 as an ordinary launch, 19.0 and
    // 18.5 if the blocks ask at their end, 21.3 and 21.0 at their start.
    const int rows = (a.tokens < a.block_tokens ? a.tokens : a.block_tokens) * a.group;
    const int y = (rows * (D / 8) + 31) / 32;
    return step_launch(attn_join_kernel<D, BF16>, dim3(blocks, y < kJoinBlocksY ? y : kJoinBlocksY), dim3(kJoinThreads), 0,
                       stream, pdl && !PAIR, 1, a);
}

template <bool BF16>
cudaError_t attn_launch_dim(int dim, bool pair, const AttnArgs& a, int blocks, bool splits, cudaStream_t stream, bool pdl) {
    switch (dim) {
        case 64: return attn_launch<64, BF16, false>(a, blocks, splits, stream, pdl);
        case 128: return attn_launch<128, BF16, false>(a, blocks, splits, stream, pdl);
        default:
            return pair ? attn_launch<256, BF16, true>(a, blocks, splits, stream, pdl)
                        : attn_launch<256, BF16, false>(a, blocks, splits, stream, pdl);
    }
}

// Pairs of blocks that can be resident at once (queried once).
int pair_capacity(int sms) {
    static std::atomic<int> known{-1};
    int n = known.load();
    if (n >= 0) return n;
    auto kern = attn_kernel<256, true, true>;
    constexpr int smem = AttnGeo<256, true>::kSmem;
    n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(sms / 2 * 2);
        cfg.blockDim = dim3(kAttnThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
    }
    if (n > sms / 2) n = sms / 2;
    known.store(n);
    return n;
}

// Whether a call of 256 columns runs on pairs of blocks: where its requests bring on average rows
// for two pairs' query tiles or more, all its heads enough to fill the SMs, and no window makes the tiles
// short (the lengths are on the device; any split of the tokens is right either way). Measured,
// pairs against single blocks, 24 query and 4 KV heads: 2048 tokens over 16384 keys 531 us
// against 572 (page 16: 535, 717), 8 x 128 over up to 8000 165 against 200, 4 x 1000 without a cache 114, 119; but
// 512 over 4096 68, 69, 86 over 16000 62, 59, and 700 in a window of 1024 56, 50.
bool attn_uses_pairs(int tokens, int R, int group, int q_heads, int window) {
    return (long long)tokens * group >= 512ll * R && (long long)tokens * q_heads >= 16384 && (window == 0 || window >= 4096);
}

bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

bool meet(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace

}  // namespace nq

using namespace nq;

extern "C" {

nq_status nq_attn_reserve(void) {
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    uint8_t* ws = nullptr;
    if (!tensor_maps_available()) return NQ_ERR_CUDA;
    return attn_workspace(&ws);
}

nq_status nq_attn_paged(const void* q, long long q_stride, const nq_kv_cache* cache, const int* block_table,
                        long long table_stride, int max_blocks, const int* q_start, const int* kv_lens, int R,
                        int tokens, int q_heads, float scale, int window, int sinks, int dtype, void* out,
                        long long out_stride, void* stream) {
    int st = check_kv_cache(cache);
    if (st != NQ_OK) return st;
    if (R < 0 || R > kAttnMaxRequests || tokens < 0 || tokens > (1 << 23) || max_blocks < 0 || table_stride < max_blocks)
        return NQ_ERR_SHAPE;
    if (q_heads < 1 || q_heads % cache->heads != 0 || q_heads / cache->heads > kAttnRows) return NQ_ERR_SHAPE;
    if ((long long)max_blocks * cache->page > (1 << 30)) return NQ_ERR_SHAPE;
    if (window < 0 || window > (1 << 30) || sinks < 0 || sinks > (1 << 30) || (sinks > 0 && window == 0))
        return NQ_ERR_SHAPE;
    if (dtype != NQ_BF16 && dtype != NQ_FP16) return NQ_ERR_SHAPE;
    if (!(scale > 0.f) || !std::isfinite(scale)) return NQ_ERR_SHAPE;
    const long long row = (long long)q_heads * cache->dim;
    if (q_stride < row || out_stride < row) return NQ_ERR_SHAPE;
    if (tokens == 1) q_stride = out_stride = row;       // between rows: nothing
    const long long qb = 2 * step_span(tokens, q_stride, row), ob = 2 * step_span(tokens, out_stride, row);
    const long long tb = max_blocks > 0 ? 4 * step_span(R, table_stride, max_blocks) : 0;
    if (qb < 0 || ob < 0 || tb < 0) return NQ_ERR_SHAPE;
    if (tokens == 0) return NQ_OK;
    if (!q || !out || !q_start || (R > 0 && (!kv_lens || (max_blocks > 0 && !block_table)))) return NQ_ERR_NULL;
    if (mis16(q) || mis16(out) || q_stride % 8 || out_stride % 8) return NQ_ERR_ALIGN;
    for (const void* p : {(const void*)block_table, (const void*)q_start, (const void*)kv_lens})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return NQ_ERR_ALIGN;
    const long long span = kv_cache_span(cache);
    if (meet(out, ob, q, qb) || meet(out, ob, cache->K, span) ||
        meet(out, ob, cache->V, span) || meet(out, ob, q_start, (R + 1) * 4ll) || meet(out, ob, kv_lens, R * 4ll) ||
        meet(out, ob, block_table, tb))
        return NQ_ERR_ALIAS;
    StepDevice d;
    st = step_device(&d);
    if (st != NQ_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (R == 0 || cache->num_blocks == 0 || max_blocks == 0)   // no key anywhere
        return cudaMemset2DAsync(out, out_stride * 2, 0, row * 2, tokens, s) == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
    uint8_t* ws = nullptr;
    st = attn_workspace(&ws);
    if (st != NQ_OK) return st;

    alignas(64) AttnArgs a;
    const bool bf16 = dtype == NQ_BF16;
    a.heads = cache->heads;
    a.group = q_heads / cache->heads;
    a.block_tokens = kAttnRows / a.group;
    const int pairs = cache->dim == 256 && attn_uses_pairs(tokens, R, a.group, q_heads, window) ? pair_capacity(d.sms) : 0;
    const bool pair = pairs > 0;
    const int units = pair ? pairs : d.sms;
    a.tile_tokens = pair ? 2 * a.block_tokens : a.block_tokens;
    a.gang = 1;
    for (int g = 2; g <= a.heads && g <= units; ++g)
        if (a.heads % g == 0 && units / g * g >= units - units / 16) a.gang = g;
    a.stride = pair ? 2 * a.gang : a.gang;
    a.gangs = units / a.gang;
    a.turns = a.heads / a.gang;
    const int blocks = a.gangs * a.stride;
    a.few_tokens = 1;
    while (a.few_tokens * a.group % 8 != 0) a.few_tokens *= 2;
    if (a.few_tokens > a.block_tokens) a.few_tokens = a.block_tokens;
    if (!encode_q_map(&a.qmap, q, q_stride, cache->dim, q_heads, tokens, a.group, a.block_tokens, bf16) ||
        !encode_q_map(&a.qfew, q, q_stride, cache->dim, q_heads, tokens, a.group, a.few_tokens, bf16) ||
        !encode_kv_map(&a.kmap, cache->K, cache, bf16, pair ? 64 : kAttnKeys) ||
        !encode_kv_map(&a.vmap, cache->V, cache, bf16, cache->dim == 256 && !pair ? 64 : kAttnKeys))
        return NQ_ERR_CUDA;
    a.out = static_cast<uint16_t*>(out);
    a.out_stride = out_stride;
    a.wide = reinterpret_cast<uintptr_t>(out) % 32 == 0 && out_stride % 16 == 0;
    a.table = block_table;
    a.table_stride = table_stride;
    a.q_start = q_start;
    a.kv_lens = kv_lens;
    a.R = R;
    a.tokens = tokens;
    a.page_shift = 0;
    while ((1 << a.page_shift) < cache->page) ++a.page_shift;
    a.max_keys = max_blocks * cache->page;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.dev_err = reinterpret_cast<int*>(ws);
    a.splits = reinterpret_cast<int4*>(ws + kAttnErrBytes);
    a.ml = reinterpret_cast<float2*>(ws + kAttnErrBytes + (size_t)d.sms * kAttnSplitBytes);
    a.part = reinterpret_cast<float*>(a.ml + (size_t)d.sms * 2 * kAttnRows);
    a.wait_ns = d.wait_ns;
    // whether any query tile can be long enough to be split: the keys a token can see, and the window's
    // drift over a tile's tokens
    long long keys = a.max_keys;
    if (window > 0 && keys > (long long)window + a.tile_tokens + 2 * kAttnKeys + sinks)
        keys = (long long)window + a.tile_tokens + 2 * kAttnKeys + sinks;
    const bool splits = (keys + kAttnKeys - 1) / kAttnKeys > kAttnWhole;
    const cudaError_t e = bf16 ? attn_launch_dim<true>(cache->dim, pair, a, blocks, splits, s, d.pdl)
                               : attn_launch_dim<false>(cache->dim, pair, a, blocks, splits, s, d.pdl);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // extern "C"
