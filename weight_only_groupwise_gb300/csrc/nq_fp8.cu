// nq_fp8.cu -- host side of the products of 8-bit codes with block scales (nq_fp8.cuh), dense and by expert, plain and
// SwiGLU: argument checks, tensor maps, the choice of kernel.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "nq.h"
#include "nq_fp8.cuh"
#include "nq_step.h"

namespace nq {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_tiled() {
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// Rows of codes as a 2-D map {K, rows}: boxes of 128 codes (a 128-byte swizzled row, zeros past K) of `box` rows.
bool encode_rows(CUtensorMap* map, const void* codes, long long stride, int K, int rows, int box) {
    const EncodeFn fn = encode_tiled();
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t boxes[2] = {kFp8Block, (cuuint32_t)box}, each[2] = {1, 1};
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, boxes, each,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Weights as a 3-D map {K, N, E}; a box is 128 codes of `box` rows of one expert.
bool encode_weights(CUtensorMap* map, const nq_fp8_weight& w, int K, int N, int E, int box) {
    const EncodeFn fn = encode_tiled();
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)E};
    const cuuint64_t strides[2] = {(cuuint64_t)w.row_stride, (cuuint64_t)w.expert_stride};
    const cuuint32_t boxes[3] = {kFp8Block, (cuuint32_t)box, 1}, each[3] = {1, 1, 1};
    return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(w.codes), dims, strides, boxes, each,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The error word of bounded waits: one in the memory of each device that the library is loaded on.
__device__ int g_error;
constexpr int kDevices = 64;
std::mutex g_lock;
int* g_error_at[kDevices] = {};

int* error_word(int dev) {
    if (dev < 0 || dev >= kDevices) return nullptr;
    std::lock_guard<std::mutex> lk(g_lock);
    if (!g_error_at[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_error) == cudaSuccess) g_error_at[dev] = static_cast<int*>(p);
    }
    return g_error_at[dev];
}

// A launch with as much shared memory as the kernel asks for (allowed once a device and thread).
template <typename Kern>
cudaError_t fp8_launch(Kern kern, int& set_for_device, int dev, int blocks, int threads, int smem, cudaStream_t stream,
                       bool pdl, int cluster, const Fp8Args& a) {
    if (set_for_device != dev) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
        set_for_device = dev;
    }
    return step_launch(kern, dim3(blocks), dim3(threads), (size_t)smem, stream, pdl, cluster, a);
}
template <bool GLU, bool BULK>
cudaError_t launch_rows(const Fp8Args& a, int dev, int blocks, cudaStream_t stream, bool pdl) {
    using Geo = Fp8RowsGeo<GLU, BULK>;
    static thread_local int set = -1;
    return fp8_launch(fp8_rows_kernel<GLU, BULK>, set, dev, blocks, Geo::kThreads, Geo::smem(a.c.E), stream, pdl, 1, a);
}
template <int BN, bool GLU>
cudaError_t launch_cols(const Fp8Args& a, int dev, int blocks, cudaStream_t stream, bool pdl) {
    using Geo = Fp8ColsGeo<BN, GLU>;
    static thread_local int set = -1;
    return fp8_launch(fp8_cols_kernel<BN, GLU>, set, dev, blocks, Geo::kThreads, Geo::smem(a.c.E), stream, pdl, a.c.split, a);
}
template <bool GLU>
cudaError_t launch_cols_of(int bn, const Fp8Args& a, int dev, int blocks, cudaStream_t stream, bool pdl) {
    switch (bn) {
        case 16: return launch_cols<16, GLU>(a, dev, blocks, stream, pdl);
        case 32: return launch_cols<32, GLU>(a, dev, blocks, stream, pdl);
        case 64: return launch_cols<64, GLU>(a, dev, blocks, stream, pdl);
        default: return launch_cols<GLU ? 64 : 128, GLU>(a, dev, blocks, stream, pdl);
    }
}

// Rows of x in the order of their experts: a warp a row, codes and scales, zeros for a row that x has not. Bound by memory.
struct GatherArgs {
    const uint8_t* x;
    const float* xs;
    const int* rows;
    uint8_t* to;
    float* to_scales;
    long long x_stride, xs_stride;
    int M, x_rows, K, blocks, stride, scale_stride;
};
constexpr int kGatherThreads = 256;

__global__ void __launch_bounds__(kGatherThreads) fp8_gather_kernel(const GatherArgs a) {
    const int i = blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    grid_launch_dependents();
    grid_dependency_wait();
    if (i >= a.M) return;
    const int r = __ldg(a.rows + i);
    const bool there = r >= 0 && r < a.x_rows;
    const uint4* const from = reinterpret_cast<const uint4*>(a.x + (there ? r : 0) * a.x_stride);
    uint4* const to = reinterpret_cast<uint4*>(a.to + (long long)i * a.stride);
    for (int k = lane; k < a.K / 16; k += 4 * 32) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = there && k + 32 * j < a.K / 16 ? __ldg(from + k + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + 32 * j < a.K / 16) to[k + 32 * j] = v[j];
    }
    for (int b = lane; b < a.blocks; b += 32)
        a.to_scales[(long long)i * a.scale_stride + b] = there ? __ldg(a.xs + r * a.xs_stride + b) : 0.f;
}

// Clusters of n blocks that can run at once, by n (queried once a device, which is the current one; none of a device past the
// last that is counted).
const int* fp8_clusters(int dev, int sms) {
    static std::once_flag once[kDevices];
    static int most[kDevices][kF8MostSplit + 1] = {};
    static const int none[kF8MostSplit + 1] = {};
    if (dev < 0 || dev >= kDevices) return none;
    std::call_once(once[dev], [sms, n_of = most[dev]] {
        using Geo = Fp8ColsGeo<16, false>;
        auto kern = fp8_cols_kernel<16, false>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) != cudaSuccess) {
            cudaGetLastError();
            return;
        }
        for (int n = 2; n <= kF8MostSplit; ++n) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(sms / n * n);
            cfg.blockDim = dim3(Geo::kThreads);
            cfg.dynamicSmemBytes = (size_t)Geo::smem(1);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = (unsigned)n;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n_of[n], kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n_of[n] = 0;
            }
        }
    });
    return most[dev];
}

// Which kernel takes a call, and how. rows: of x in a tile of fp8_cols_kernel, or 0 for fp8_rows_kernel; split: blocks that
// share a tile's K.
struct Fp8Plan {
    int rows, split;
};

// Rows a group on average up to which calls by expert go in small tiles. Where weights of many experts are read for few rows
// each, these need fewer copies. SwiGLU, 128 experts of 2048 -> 768, us with tiles of 16, 32 rows and fp8_rows_kernel: 12
// rows an expert 67.4, 70.8, 79.8; 24 rows 76.4, 70.8, 81.0; 32 rows 97, 88, 83. Plain, tiles of 16, 32, 64 rows and
// fp8_rows_kernel: 128 experts of 768 -> 2048, 6 rows 35.2, 39.9, -, 38.4; 12 rows 42.2, 43.2, 40.3, 40.5; 28 rows 67, 56.1,
// 41.9, 41.7; 64 experts, 24 rows -, 28.9, 22.9, 25.7; 56 rows -, 47.5, 30.2, 28.0; 256 of 2048 -> 4096, 20 rows -, 389, 321,
// 332. Tiles of 64 rows that the copy engine gathers take it longer than their weights, so that calls with `gathered` rows,
// which have not been copied together, leave them out.
int fp8_experts_rows(int M, int E, bool glu, bool gathered) {
    const int each = (M + E - 1) / E;
    if (glu) return each <= 16 ? 16 : each <= 28 ? 32 : 0;
    return each <= 10 ? 16 : each <= 32 && !gathered ? 64 : 0;
}

// A dense call: the fewest microseconds by a count of the blocks of K that the busiest SM goes through, at what one of them
// takes each kernel (measured at K = 4096 and 5120; a tile's blocks of K, 128 columns or 256, are one after
// another): few tiles leave SMs idle, large ones are cheaper a row. A launch takes 4 us, the exchange of a split sum 1.5.
// 333 x 4112 x 2501, us: tiles of 64 rows 15.0, of 128 shared by two blocks 14.2, fp8_rows_kernel 28.4; 256 x 4096 x 5120:
// 23.6, 16.5, 20.4; 512 x 5120 x 17408: 111, 67, 48.
Fp8Plan fp8_dense_plan(int M, int K, int N, bool glu, int sms, const int* clusters) {
    static const struct {
        int rows;
        float us[2];                             // a block of K: plain, SwiGLU
    } kinds[] = {{16, {0.25f, 0.35f}}, {32, {0.30f, 0.50f}}, {64, {0.35f, 0.70f}}, {128, {0.43f, 0.f}}, {0, {0.48f, 0.62f}}};
    const long long blocks = (K + kFp8Block - 1) / kFp8Block;
    Fp8Plan best = {0, 1};
    float least = 1e30f;
    for (const auto& k : kinds) {
        if (k.us[glu] == 0.f) continue;
        const int high = k.rows ? k.rows : kF8Tile, wide = k.rows || glu ? 128 : 256;
        const long long tiles = (long long)((M + high - 1) / high) * ((N + wide - 1) / wide), rounds = (tiles + sms - 1) / sms;
        long long split = 1;                     // as many as can run at once
        for (int n = 2; k.rows && n <= kF8MostSplit && n <= blocks / 2; ++n)
            if (tiles <= clusters[n]) split = n;
        const float us = 4.f + (split > 1 ? 1.5f : 0.f) + k.us[glu] * rounds * ((blocks + split - 1) / split);
        if (us < least) {
            least = us;
            best = {k.rows, (int)split};
        }
    }
    return best;
}

// Whether gathered rows are copied together first, where there is scratch memory: for tiles of 64 rows and more, whose rows
// take the copy engine longer to gather than to multiply (4096 tokens x 8 of 64 experts: 1014 us, 497 so).
bool fp8_gathers(int M, int E, bool glu) { return fp8_experts_rows(M, E, glu, true) == 0; }
long long scratch_stride(int K) { return (K + 15) / 16 * 16; }
int scratch_scales(int K) { return ((K + kFp8Block - 1) / kFp8Block + 3) / 4 * 4; }

// Bytes that a weight's codes and floats that its scales span; -1: more than a tensor can have.
long long weight_span(const nq_fp8_weight* w, int E, int N, int K) {
    const long long rows = step_span(N, w->row_stride, K);
    return rows < 0 ? -1 : step_span(E, w->expert_stride, rows);
}
long long weight_scale_span(const nq_fp8_weight* w, int E, int N, int K) {
    const long long rows = step_span((N + kFp8Block - 1) / kFp8Block, w->scale_row_stride, (K + kFp8Block - 1) / kFp8Block);
    return rows < 0 ? -1 : step_span(E, w->scale_expert_stride, rows);
}

// All of the four products. experts: rows and offsets count, else they are not given.
int fp8_call(const nq_fp8_rows* x, bool experts, const int* rows, int M, const int* offsets, int E,
             const nq_fp8_weight* w0, const nq_fp8_weight* w1, bool glu, const nq_fp8_out* y, int K, int N, void* scratch,
             void* stream) {
    if (!x || !w0 || (glu && !w1) || !y) return NQ_ERR_NULL;
    if (x->rows < 0 || x->rows > kFp8MostRows || M < 0 || M > kFp8MostRows || E < 1 || E > kMostExperts) return NQ_ERR_SHAPE;
    if (K < 16 || K > kFp8MostCols || K % 16 || N < 1 || N > kFp8MostCols) return NQ_ERR_SHAPE;
    if (experts && !rows && M > x->rows) return NQ_ERR_SHAPE;
    const bool codes = y->dtype == NQ_E4M3;
    if (y->dtype != NQ_BF16 && y->dtype != NQ_FP16 && !(codes && glu && N % 16 == 0)) return NQ_ERR_SHAPE;
    const int kb = (K + kFp8Block - 1) / kFp8Block, nb = (N + kFp8Block - 1) / kFp8Block, el = codes ? 1 : 2;
    long long xst = x->stride, xss = x->scale_stride, yst = y->stride, yss = y->scale_stride;
    if (x->rows <= 1) {                          // between rows: nothing
        xst = K;
        xss = kb;
    }
    if (M <= 1) {
        yst = N;
        yss = nb;
    }
    if (xst < K || xss < kb || yst < N || (codes && yss < nb)) return NQ_ERR_SHAPE;
    const long long xb = step_span(x->rows, xst, K), xsb = 4 * step_span(x->rows, xss, kb);
    const long long yb = el * step_span(M, yst, N), ysb = codes ? 4 * step_span(M, yss, nb) : 0;
    if (xb < 0 || xsb < 0 || yb < 0 || ysb < 0) return NQ_ERR_SHAPE;
    const nq_fp8_weight* w[2] = {w0, glu ? w1 : w0};
    long long wb[2], wsb[2];
    nq_fp8_weight v[2];
    for (int g = 0; g < 2; ++g) {
        v[g] = *w[g];
        if (N == 1) v[g].row_stride = K;         // between one row and the next: nothing
        if (nb == 1) v[g].scale_row_stride = kb;
        if (E == 1) {
            v[g].expert_stride = (K + 15) / 16 * 16;
            v[g].scale_expert_stride = kb;
        }
        if (v[g].row_stride < K || v[g].scale_row_stride < kb || v[g].expert_stride < 0 || v[g].scale_expert_stride < 0)
            return NQ_ERR_SHAPE;
        wb[g] = weight_span(&v[g], E, N, K);
        wsb[g] = 4 * weight_scale_span(&v[g], E, N, K);
        if (wb[g] < 0 || wsb[g] < 0) return NQ_ERR_SHAPE;
    }
    if (M == 0) return NQ_OK;
    if ((x->rows > 0 && (!x->codes || !x->scales)) || !y->data || (codes && !y->scales) || (experts && !offsets))
        return NQ_ERR_NULL;
    for (int g = 0; g < 2; ++g)
        if (!v[g].codes || !v[g].scales) return NQ_ERR_NULL;
    if (mis(x->codes, 16) || xst % 16 || mis(x->scales, 4) || mis(y->data, codes ? 16 : 2) || (codes && yst % 16) ||
        (codes && mis(y->scales, 4)) || mis(rows, 4) || mis(offsets, 4) || mis(scratch, 16))
        return NQ_ERR_ALIGN;
    for (int g = 0; g < 2; ++g)
        if (mis(v[g].codes, 16) || v[g].row_stride % 16 || v[g].expert_stride % 16 || mis(v[g].scales, 4)) return NQ_ERR_ALIGN;
    const struct {
        const void* p;
        long long n;
    } in[] = {{x->codes, xb}, {x->scales, xsb}, {rows, M * 4ll}, {offsets, (E + 1) * 4ll},
              {v[0].codes, wb[0]}, {v[0].scales, wsb[0]}, {v[1].codes, wb[1]}, {v[1].scales, wsb[1]}};
    for (const auto& i : in)
        if (meet(y->data, yb, i.p, i.n) || (codes && meet(y->scales, ysb, i.p, i.n))) return NQ_ERR_ALIAS;
    if (codes && meet(y->data, yb, y->scales, ysb)) return NQ_ERR_ALIAS;
    const bool gathers = rows && scratch && fp8_gathers(M, E, glu);
    if (gathers) {
        const long long sb = M * (scratch_stride(K) + 4ll * scratch_scales(K));
        for (const auto& i : in)
            if (meet(scratch, sb, i.p, i.n)) return NQ_ERR_ALIAS;
        if (meet(scratch, sb, y->data, yb) || (codes && meet(scratch, sb, y->scales, ysb))) return NQ_ERR_ALIAS;
    }
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NQ_ERR_CUDA;
    Fp8Args a;
    Fp8Call& c = a.c;
    c.err = error_word(dev);
    if (!c.err) return NQ_ERR_CUDA;
    c.xs = x->scales;
    c.rows = rows;
    c.offsets = offsets;
    for (int g = 0; g < 2; ++g) {
        c.ws[g] = v[g].scales;
        c.ws_row[g] = v[g].scale_row_stride;
        c.ws_expert[g] = v[g].scale_expert_stride;
    }
    c.xs_stride = xss;
    c.y = static_cast<uint8_t*>(y->data);
    c.ys = y->scales;
    c.y_stride = yst;
    c.ys_stride = yss;
    c.x_rows = x->rows;
    c.E = E;
    c.M = M;
    c.K = K;
    c.N = N;
    c.dtype = y->dtype;
    c.wide = !mis(y->data, 16) && yst % 8 == 0;
    c.quads = !mis(x->scales, 16) && xss % 4 == 0;
    c.wait_ns = d.wait_ns;
    const Fp8Plan plan = experts ? Fp8Plan{fp8_experts_rows(M, E, glu, rows && !gathers), 1} : fp8_dense_plan(M, K, N, glu, d.sms, fp8_clusters(dev, d.sms));
    const int bn = plan.rows;
    const bool few = bn > 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const void* codes_at = x->codes;
    int x_rows = x->rows;
    if (gathers) {
        GatherArgs g;
        g.x = static_cast<const uint8_t*>(x->rows > 0 ? x->codes : v[0].codes);
        g.xs = x->scales;
        g.rows = rows;
        g.to = static_cast<uint8_t*>(scratch);
        g.to_scales = reinterpret_cast<float*>(g.to + M * scratch_stride(K));
        g.x_stride = xst;
        g.xs_stride = xss;
        g.M = M;
        g.x_rows = x->rows;
        g.K = K;
        g.blocks = kb;
        g.stride = (int)scratch_stride(K);
        g.scale_stride = scratch_scales(K);
        const int per = kGatherThreads / 32;
        if (step_launch(fp8_gather_kernel, dim3((M + per - 1) / per), dim3(kGatherThreads), 0, s, d.pdl, 1, g) != cudaSuccess)
            return NQ_ERR_CUDA;
        codes_at = scratch;
        x_rows = M;
        xst = g.stride;
        c.rows = rows = nullptr;
        c.xs = g.to_scales;
        c.xs_stride = g.scale_stride;
        c.x_rows = M;
        c.quads = true;                          // (M codes rows are a multiple of 16 bytes)
    }
    // a map needs a row; of none, any memory that is there
    c.x_past = x_rows > 0 ? x_rows : 1;
    if (x_rows == 0) codes_at = v[0].codes;
    if (!encode_rows(&a.xmap, codes_at, x_rows > 1 ? xst : K, K, c.x_past, rows ? 1 : (few ? bn : kF8Tile))) return NQ_ERR_CUDA;
    for (int g = 0; g <= (int)glu; ++g)
        if (!encode_weights(&a.wmap[g], v[g], K, N, E, few || glu ? kF8Tile : 256)) return NQ_ERR_CUDA;
    if (!glu) a.wmap[1] = a.wmap[0];
    // a block an SM, or one a tile where the tiles cannot be more
    const int wide = few || glu ? kF8Tile : 256, high = few ? bn : kF8Tile;
    const long long most = (long long)((N + wide - 1) / wide) * (experts ? (M + high - 1) / high + (E < M ? E : M) : (M + high - 1) / high);
    c.split = plan.split;
    // results of sums of up to so many blocks of K go by bulk copies, at the price of a stage (us, stored by the threads and so:
    // 24570 rows of 128 experts x 2048, K = 256 52.6, 45.3; 768 83.0, 74.3; 2304 166.8, 166.0; 4096 281.4, 273.8; 4096 x 5120 x
    // 17408 327.1, 329.3; 2048 x 17408 x 5120 204.3, 209.8)
    const bool bulk = c.wide && N % 8 == 0 && K <= 32 * kFp8Block;
    const int blocks = c.split > 1 ? (int)(most * c.split) : (int)(most < d.sms ? most : d.sms);
    const cudaError_t e = few ? (glu ? launch_cols_of<true>(bn, a, dev, blocks, s, d.pdl) : launch_cols_of<false>(bn, a, dev, blocks, s, d.pdl))
                              : glu  ? launch_rows<true, false>(a, dev, blocks, s, d.pdl)
                          : bulk ? launch_rows<false, true>(a, dev, blocks, s, d.pdl)
                                 : launch_rows<false, false>(a, dev, blocks, s, d.pdl);
    return e == cudaSuccess ? NQ_OK : NQ_ERR_CUDA;
}

}  // namespace
}  // namespace nq

using namespace nq;

int nq::fp8_take_error(int dev) {
    int* at = nullptr;
    {
        if (dev < 0 || dev >= kDevices) return NQ_OK;
        std::lock_guard<std::mutex> lk(g_lock);
        at = g_error_at[dev];
    }
    if (!at) return NQ_OK;                       // nothing has run there
    int err = 0;
    if (cudaMemcpy(&err, at, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return NQ_ERR_CUDA;
    if (err == 0) return NQ_OK;
    if (cudaMemset(at, 0, sizeof(int)) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return NQ_ERR_CUDA;
    return NQ_ERR_TIMEOUT;
}

extern "C" {

size_t nq_fp8_scratch_bytes(int M, int E, int K, int swiglu) {
    if (M <= 0 || M > kFp8MostRows || E < 1 || E > kMostExperts || K < 16 || K > kFp8MostCols || !fp8_gathers(M, E, swiglu != 0)) return 0;
    return (size_t)M * (scratch_stride(K) + 4 * scratch_scales(K));
}

nq_status nq_gemm_fp8(const nq_fp8_rows* x, const nq_fp8_weight* w, const nq_fp8_out* y, int K, int N, void* stream) {
    return fp8_call(x, false, nullptr, x ? x->rows : 0, nullptr, 1, w, nullptr, false, y, K, N, nullptr, stream);
}

nq_status nq_swiglu_fp8(const nq_fp8_rows* x, const nq_fp8_weight* wg, const nq_fp8_weight* wu, const nq_fp8_out* h,
                        int K, int N, void* stream) {
    return fp8_call(x, false, nullptr, x ? x->rows : 0, nullptr, 1, wg, wu, true, h, K, N, nullptr, stream);
}

nq_status nq_gemm_fp8_experts(const nq_fp8_rows* x, const int* rows, int M, const int* offsets, int E,
                              const nq_fp8_weight* w, const nq_fp8_out* y, int K, int N, void* scratch, void* stream) {
    return fp8_call(x, true, rows, M, offsets, E, w, nullptr, false, y, K, N, scratch, stream);
}

nq_status nq_swiglu_fp8_experts(const nq_fp8_rows* x, const int* rows, int M, const int* offsets, int E,
                                const nq_fp8_weight* wg, const nq_fp8_weight* wu, const nq_fp8_out* h, int K, int N,
                                void* scratch, void* stream) {
    return fp8_call(x, true, rows, M, offsets, E, wg, wu, true, h, K, N, scratch, stream);
}

}  // extern "C"
