// nq_step.h -- internal interface of the serving-step calls (page tables, KV append, paged
// attention, sampling) to the runtime in nq_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace nq {

// The current device as a step call sees it: its SM count, whether dependent launches are on
// and the bound of device-side waits. Returns an nq_status (NQ_ERR_DEVICE off a GB300).
struct StepDevice {
    int sms;
    bool pdl;
    unsigned long long wait_ns;
};
int step_device(StepDevice* out);

// The attention workspace of the current device (allocated on first use, never moved until
// nq_shutdown): 256 bytes whose first int is the device error word, then `kAttnWsBytes(sms)`
// bytes of scratch.
int attn_workspace(uint8_t** ws);

// Elements from the first of `rows` rows, `stride` apart, to the end of the last; -1 from 2^38 on, which no tensor
// of this GPU can have (the limit keeps spans and offsets in 64 bits, and strides in a tensor map's range).
inline long long step_span(long long rows, long long stride, long long row) {
    if (rows <= 0) return 0;
    constexpr long long most = 1ll << 38;
    if (row < 0 || row >= most || (rows > 1 && stride > (most - 1 - row) / (rows - 1))) return -1;
    return (rows - 1) * stride + row;
}

constexpr size_t kAttnErrBytes = 256;
constexpr int kAttnRows = 128;      // query rows of an attention tile
constexpr int kAttnMaxDim = 256;
// Per block: one split record, two partial tiles (fp32 rows x dim), their (maximum, sum) rows.
constexpr size_t kAttnSplitBytes = 32;
inline size_t attn_ws_bytes(int sms) {
    return kAttnErrBytes + (size_t)sms * (kAttnSplitBytes + 2 * kAttnRows * (kAttnMaxDim * 4 + 8));
}

// Launch with programmatic dependent launch when `pdl` (the kernel then waits for the
// preceding kernel of the stream itself before it touches memory).
template <typename K, typename... A>
inline cudaError_t step_launch(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl, int cluster,
                               const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace nq
