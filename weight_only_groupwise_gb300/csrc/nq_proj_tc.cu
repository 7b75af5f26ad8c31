// Instantiations (4- and 5-bit codes) and host side of the large-batch tensor-core projection
// kernel (nq_tc.cuh): the tensor maps and the launch.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "nq.h"
#include "nq_launch.h"

namespace nq {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

}  // namespace

bool tensor_maps_available() { return encode_fn() != nullptr; }

// X (bf16 [T][K], row-major) as a 3-D tensor [K/64][T][64]: a box {64, TP, BG} (BG = the
// stage's groups) lands in shared memory as one [TP][64] block per group, 128-byte rows with
// the 128-byte swizzle (16-byte chunk c of token t at chunk c ^ (t % 8)), which is the tensor
// core's K-major swizzled layout; tokens T..TP-1 are outside the tensor and read as zeros.
// 128-byte rows keep the copy engine's request count at TP per group.
bool encode_x_map(CUtensorMap* map, const void* X, int T, int K, int TP) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kGroup, (cuuint64_t)T, (cuuint64_t)(K / kGroup)};
    const cuuint64_t strides[2] = {(cuuint64_t)K * 2, (cuuint64_t)kGroup * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kGroup, (cuuint32_t)TP, (cuuint32_t)tc_stage_groups(TP)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(X), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The packed codes and scales of a matrix as 3-D tensors of 8-byte elements [RT][G][bytes / 8]
// (16-row tiles, 64-wide K groups, one tile-group block): a box {bytes / 8, BG, kTcTiles} (BG =
// the stage's groups for TP padded tokens) is one stage's codes (or scales) of a 128-row
// block, laid out tile-major as the kernel reads them; tiles past RT and groups past G read as
// zeros.
bool encode_weight_maps(CUtensorMap* wmap, CUtensorMap* smap, const void* W, const void* S, int bits, int K, int N,
                        int TP) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int G = K / kGroup, RT = N / kTileRows;
    const cuuint32_t estr[3] = {1, 1, 1};
    const int tb = code_tile_bytes(bits);
    const cuuint64_t wdims[3] = {(cuuint64_t)(tb / 8), (cuuint64_t)G, (cuuint64_t)RT};
    const cuuint64_t wstr[2] = {(cuuint64_t)tb, (cuuint64_t)G * tb};
    const cuuint32_t bg = (cuuint32_t)tc_stage_groups(TP);
    const cuuint32_t wbox[3] = {(cuuint32_t)(tb / 8), bg, (cuuint32_t)kTcTiles};
    const int stb = scale_tile_bytes(bits);
    const cuuint64_t sdims[3] = {(cuuint64_t)(stb / 8), (cuuint64_t)G, (cuuint64_t)RT};
    const cuuint64_t sstr[2] = {(cuuint64_t)stb, (cuuint64_t)G * stb};
    const cuuint32_t sbox[3] = {(cuuint32_t)(stb / 8), bg, (cuuint32_t)kTcTiles};
    return fn(wmap, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<void*>(W), wdims, wstr, wbox, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
           fn(smap, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<void*>(S), sdims, sstr, sbox, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One of a paged cache's two tensors as a 4-D map {dim, page rows, heads, blocks} with the
// cache's own strides; a box is 64 columns (a 128-byte swizzled row) of min(page, rows) keys of
// one head and block. A block id outside the cache reads as zeros.
bool encode_kv_map(CUtensorMap* map, void* base, const nq_kv_cache* c, bool bf16, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c->dim, (cuuint64_t)c->page, (cuuint64_t)c->heads, (cuuint64_t)c->num_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)c->row_stride * 2, (cuuint64_t)c->head_stride * 2,
                                   (cuuint64_t)c->block_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(c->page < rows ? c->page : rows), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [tokens][heads][dim] as a 3-D map {dim, heads, tokens}: a box is 64 columns (a 128-byte
// swizzled row) of `group` heads of `box_tokens` tokens; tokens past the last read as zeros.
bool encode_q_map(CUtensorMap* map, const void* q, long long stride, int dim, int heads, int tokens, int group,
                  int box_tokens, bool bf16) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)box_tokens};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(q),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_tc_proj(int bits, const TcArgs& a, cudaStream_t stream, bool pdl) {
    if (bits == kFp4) return launch_tc_proj_fp4(a, stream, pdl);
    switch (a.p.TP) {
        case 16: return bits == 4 ? tc_launch<4, 16>(a, stream, pdl) : tc_launch<5, 16>(a, stream, pdl);
        case 32: return bits == 4 ? tc_launch<4, 32>(a, stream, pdl) : tc_launch<5, 32>(a, stream, pdl);
        default: return bits == 4 ? tc_launch<4, 64>(a, stream, pdl) : tc_launch<5, 64>(a, stream, pdl);
    }
}

}  // namespace nq
