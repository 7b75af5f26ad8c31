// nq_quant.cu -- activations into 8-bit codes with a scale for each 128 columns of a row (nq_quant_fp8):
//
//   s[r, b] = max(max over the block of |x| / 448, 2^-126),   c[r, k] = e4m3(x[r, k] / s[r, k / 128])
//
// 448 is e4m3's largest value; the floor keeps s normal, so that x / s is at most 448 for any x and a block of zeros
// needs no case of its own. Bound by memory: x once, a byte an element and 4 / 128 for the scales (8191 x 17408 in
// 16 bits: 69 us, 6.2 TB/s; issue slots, which the arithmetic fills to some 70 %, come next). Nothing is reused, so a
// warp takes 1024 columns of a row straight from memory: its lanes have 8 columns of four pairs of blocks, all loads in
// flight at once, and 16 lanes find a block's largest by shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_fp8.h"
#include "nq_step.h"

namespace nq {
namespace {

constexpr int kQtThreads = 64;                   // (8191 x 17408, us: 64 69.2, 128 70.5, 256 72.2, 512 83.6)
constexpr int kQtSteps = 4;                      // loads of 8 columns a lane (with 256 threads: 2 83.1, 4 72.2, 8 72.7)
constexpr int kQtCols = 32 * 8 * kQtSteps;       // columns of a warp

struct QuantArgs {
    const uint8_t* x;
    uint8_t* codes;
    float* scales;
    long long x_stride, codes_stride, scale_stride;   // between rows: bytes, bytes, floats
    int K;
    uint32_t segments;                           // of kQtCols columns in a row
    long long total;                             // rows x segments
};

// 8 columns as floats.
template <int DTYPE>
struct Eight {
    uint4 lo, hi;                                // hi: fp32 only
    __device__ __forceinline__ void load(const uint8_t* p) {
        lo = __ldg(reinterpret_cast<const uint4*>(p));
        if (DTYPE == NQ_FP32) hi = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { lo = hi = make_uint4(0, 0, 0, 0); }
    // The largest magnitude of the 16 lanes' columns, by the order of bits: a NaN is the largest of all, so that it reaches
    // the scale. 16-bit values two at a time.
    __device__ __forceinline__ float largest() const {
        if constexpr (DTYPE == NQ_FP32) {
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            return __uint_as_float(m);
        } else {
            const uint32_t sign = 0x7FFF7FFFu;
            uint32_t m = __vmaxu2(__vmaxu2(lo.x & sign, lo.y & sign), __vmaxu2(lo.z & sign, lo.w & sign));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
            m = max(m & 0xFFFFu, m >> 16);
            return DTYPE == NQ_BF16 ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
        }
    }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DTYPE == NQ_FP32) {
                f[i] = __uint_as_float(w[i]);
                f[4 + i] = __uint_as_float(w[4 + i]);
            } else if constexpr (DTYPE == NQ_BF16) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        }
    }
};

// x / s for two, with r = 1 / s rounded: the product and one correction by its residual, which is exact in an fma. Rounding
// the residual down makes no difference to it but for its sign where it is zero: -0, which added to a quotient of either zero
// leaves that as it is (+0 turns -0 into +0).
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990: rounded as the quotient
// is. A division each took 92 us for 8191 x 17408 in 16 bits, single ones of this 74, two at a time and the largest of two
// at a time 72.)
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void quotients(float& a, float& b, uint64_t minus_s, uint64_t r) {
    const uint64_t x = two(a, b);
    uint64_t q, e;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q), "l"(minus_s), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(r), "l"(q));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(q));
}

template <int DTYPE>
__global__ void __launch_bounds__(kQtThreads) quant_kernel(const QuantArgs a) {
    const long long at = (long long)blockIdx.x * (kQtThreads / 32) + (threadIdx.x >> 5);
    // (the next kernel is not let start early: a product reads its weights' codes without waiting for what has been)
    grid_dependency_wait();
    if (at >= a.total) return;
    const int lane = threadIdx.x & 31;
    const long long r = a.segments == 1 ? at : at / a.segments;
    const int col0 = (int)(at - r * a.segments) * kQtCols + lane * 8;
    const uint8_t* x = a.x + r * a.x_stride + (long long)col0 * (DTYPE == NQ_FP32 ? 4 : 2);
    Eight<DTYPE> v[kQtSteps];
#pragma unroll
    for (int i = 0; i < kQtSteps; ++i) {
        if (col0 + i * 256 < a.K)
            v[i].load(x + i * 256 * (DTYPE == NQ_FP32 ? 4 : 2));
        else
            v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kQtSteps; ++i) {
        float f[8];
        v[i].floats(f);
        const float s = fp8_scale(v[i].largest());
        const int col = col0 + i * 256;
        if (col < a.K) {
            if (s > 0x1p-60f && s < 0x1p60f) {
                const float r = 1.f / s;
                const uint64_t minus_s = two(-s, -s), rr = two(r, r);
#pragma unroll
                for (int j = 0; j < 8; j += 2) quotients(f[j], f[j + 1], minus_s, rr);
            } else {                             // residuals out of range, an infinite scale
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] /= s;
            }
            uint2 c;
            c.x = fp8_codes(f[0], f[1], f[2], f[3]);
            c.y = fp8_codes(f[4], f[5], f[6], f[7]);
            *reinterpret_cast<uint2*>(a.codes + r * a.codes_stride + col) = c;
            if ((lane & 15) == 0) a.scales[r * a.scale_stride + col / kFp8Block] = s;
        }
    }
}

}  // namespace
}  // namespace nq

using namespace nq;

extern "C" nq_status nq_quant_fp8(const void* x, int dtype, long long x_stride, int rows, int K, void* codes,
                                  long long codes_stride, float* scales, long long scale_stride, void* stream) {
    if (dtype != NQ_BF16 && dtype != NQ_FP16 && dtype != NQ_FP32) return NQ_ERR_SHAPE;
    if (rows < 0 || rows > kFp8MostRows || K < 16 || K > kFp8MostCols || K % 16) return NQ_ERR_SHAPE;
    const int el = dtype == NQ_FP32 ? 4 : 2, blocks = (K + kFp8Block - 1) / kFp8Block;
    if (x_stride < K || codes_stride < K || scale_stride < blocks) return NQ_ERR_SHAPE;
    if (rows == 1) {                             // between rows: nothing
        x_stride = codes_stride = K;
        scale_stride = blocks;
    }
    const long long xb = step_span(rows, x_stride, K), cb = step_span(rows, codes_stride, K);
    const long long sb = step_span(rows, scale_stride, blocks);
    if (xb < 0 || cb < 0 || sb < 0) return NQ_ERR_SHAPE;
    if (rows == 0) return NQ_OK;
    if (!x || !codes || !scales) return NQ_ERR_NULL;
    if (mis(x, 16) || mis(codes, 16) || mis(scales, 4) || x_stride * el % 16 || codes_stride % 16) return NQ_ERR_ALIGN;
    if (meet(codes, cb, x, xb * el) || meet(scales, sb * 4, x, xb * el) || meet(codes, cb, scales, sb * 4))
        return NQ_ERR_ALIAS;
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    QuantArgs a;
    a.x = static_cast<const uint8_t*>(x);
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.x_stride = x_stride * el;
    a.codes_stride = codes_stride;
    a.scale_stride = scale_stride;
    a.K = K;
    a.segments = (uint32_t)((K + kQtCols - 1) / kQtCols);
    a.total = (long long)rows * a.segments;
    const dim3 grid((unsigned)((a.total + kQtThreads / 32 - 1) / (kQtThreads / 32)));
    auto kern = dtype == NQ_BF16 ? quant_kernel<NQ_BF16> : (dtype == NQ_FP16 ? quant_kernel<NQ_FP16> : quant_kernel<NQ_FP32>);
    return step_launch(kern, grid, dim3(kQtThreads), 0, reinterpret_cast<cudaStream_t>(stream), d.pdl, 1, a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}
