// nq_fp8.h -- what the 8-bit calls share (quantisation, products, experts): limits, the rule of scales and codes,
// host checks.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace nq {

constexpr int kFp8Block = 128;              // columns (and rows of a weight) of a scale
constexpr int kFp8MostRows = 1 << 24;
constexpr int kFp8MostCols = 1 << 20;       // K and N
constexpr int kMostExperts = 512;

inline bool mis(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

inline bool meet(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// The error word of the products' bounded waits on device `dev`, reported and cleared for nq_device_error, whose
// caller has synchronised: NQ_OK, NQ_ERR_TIMEOUT or NQ_ERR_CUDA.
int fp8_take_error(int dev);

#ifdef __CUDACC__
// The scale of a block whose largest magnitude is m (NaN if one of its values is).
__device__ __forceinline__ float fp8_scale(float m) {
    const float s = m / 448.f;
    return s < 0x1p-126f ? 0x1p-126f : s;
}

// Four e4m3 codes, the first in the lowest byte: round to nearest even, at most 448, NaN for NaN.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
#endif

}  // namespace nq
