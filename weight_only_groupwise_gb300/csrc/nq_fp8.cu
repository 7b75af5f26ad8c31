// nq_fp8.cu -- products of 8-bit codes with block scales: dense and by expert, plain and SwiGLU.
#include <cuda.h>
#include <cuda_runtime.h>

#include "nq.h"
#include "nq_common.cuh"
#include "nq_fp8.h"
#include "nq_step.h"

namespace nq {
namespace {

constexpr int kSimpleRows = 32, kSimpleThreads = 256, kSimpleK = 32;

struct Fp8Args {
    const uint8_t* x;
    const float* xs;
    long long x_stride, xs_stride;
    int x_rows;
    const int* rows;                             // NULL: row i
    const int* offsets;                          // NULL: one group of M rows
    int E, M, K, N;
    const uint8_t* w[2];
    const float* ws[2];
    long long w_row[2], w_expert[2], ws_row[2], ws_expert[2];
    uint8_t* y;
    float* ys;
    long long y_stride, ys_stride;               // elements
    int dtype;
    bool glu;
};

__device__ __forceinline__ float e4m3_float(uint8_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
    return __half2float(__ushort_as_half((uint16_t)h));
}

// A block 32 rows x 128 columns; a thread a row's 16 columns.
__global__ void __launch_bounds__(kSimpleThreads) fp8_simple_kernel(const Fp8Args a) {
    __shared__ float sx[kSimpleRows][kSimpleK + 1], sw[2][128][kSimpleK + 1];
    grid_launch_dependents();
    grid_dependency_wait();
    int tile = blockIdx.y, e = 0, r0 = 0, r1 = a.M;
    if (a.offsets) {
        for (;; ++e) {
            if (e == a.E) return;
            r0 = min(max(a.offsets[e], 0), a.M);
            r1 = min(max(a.offsets[e + 1], r0), a.M);
            const int n = (r1 - r0 + kSimpleRows - 1) / kSimpleRows;
            if (tile < n) break;
            tile -= n;
        }
    }
    r0 += tile * kSimpleRows;
    const int n0 = blockIdx.x * 128, tid = threadIdx.x, row = tid >> 3, c0 = tid & 7;
    const int live = min(kSimpleRows, r1 - r0);
    float acc[2][16] = {};
    auto source = [&](int r) { return r < live ? (a.rows ? a.rows[r0 + r] : r0 + r) : -1; };
    const int mine = source(row);
    const bool there = mine >= 0 && mine < a.x_rows;
    for (int b0 = 0; b0 < a.K; b0 += 128) {
        const float s = there ? a.xs[mine * a.xs_stride + b0 / 128] : 0.f;
        float part[2][16] = {};
        for (int k0 = b0; k0 < min(a.K, b0 + 128); k0 += kSimpleK) {
            __syncthreads();
            for (int i = tid; i < kSimpleRows * kSimpleK; i += kSimpleThreads) {
                const int r = i / kSimpleK, k = k0 + i % kSimpleK, at = source(r);
                sx[r][i % kSimpleK] = at >= 0 && at < a.x_rows && k < a.K ? e4m3_float(a.x[at * a.x_stride + k]) : 0.f;
            }
            for (int g = 0; g <= (int)a.glu; ++g)
                for (int i = tid; i < 128 * kSimpleK; i += kSimpleThreads) {
                    const int n = i / kSimpleK, k = k0 + i % kSimpleK;
                    sw[g][n][i % kSimpleK] = n0 + n < a.N && k < a.K
                                                 ? e4m3_float(a.w[g][e * a.w_expert[g] + (n0 + n) * a.w_row[g] + k])
                                                 : 0.f;
                }
            __syncthreads();
            for (int k = 0; k < kSimpleK; ++k)
                for (int g = 0; g <= (int)a.glu; ++g)
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[g][i] = fmaf(sx[row][k], sw[g][c0 + 8 * i][k], part[g][i]);
        }
        for (int g = 0; g <= (int)a.glu; ++g) {
            const float f = s * a.ws[g][e * a.ws_expert[g] + (n0 / 128) * a.ws_row[g] + b0 / 128];
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[g][i] = fmaf(f, part[g][i], acc[g][i]);
        }
    }
    float m = 0.f;
    if (a.glu)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            acc[0][i] = silu_mul(acc[0][i], acc[1][i]);
            if (n0 + c0 + 8 * i < a.N)
                m = __uint_as_float(max(__float_as_uint(m), __float_as_uint(acc[0][i]) & 0x7FFFFFFFu));
        }
    float q = 1.f;
    if (a.dtype == NQ_E4M3) {
        for (int d = 4; d > 0; d >>= 1)
            m = __uint_as_float(max(__float_as_uint(m), __shfl_xor_sync(0xFFFFFFFFu, __float_as_uint(m), d)));
        q = fp8_scale(m);
        if (row < live && c0 == 0) a.ys[(r0 + row) * a.ys_stride + n0 / 128] = q;
    }
    if (row >= live) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int n = n0 + c0 + 8 * i;
        if (n >= a.N) continue;
        const long long at = (r0 + row) * a.y_stride + n;
        if (a.dtype == NQ_E4M3)
            a.y[at] = (uint8_t)fp8_codes(acc[0][i] / q, 0.f, 0.f, 0.f);
        else
            reinterpret_cast<uint16_t*>(a.y)[at] =
                a.dtype == NQ_BF16 ? bf16_bits_rn(acc[0][i]) : __half_as_ushort(__float2half_rn(acc[0][i]));
    }
}

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
             const nq_fp8_weight* w0, const nq_fp8_weight* w1, bool glu, const nq_fp8_out* y, int K, int N, void* stream) {
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
            v[g].expert_stride = (long long)K;
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
        mis(y->scales, 4) || mis(rows, 4) || mis(offsets, 4))
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
    StepDevice d;
    const int st = step_device(&d);
    if (st != NQ_OK) return st;
    Fp8Args a;
    a.x = static_cast<const uint8_t*>(x->codes);
    a.xs = x->scales;
    a.x_stride = xst;
    a.xs_stride = xss;
    a.x_rows = x->rows;
    a.rows = rows;
    a.offsets = offsets;
    a.E = E;
    a.M = M;
    a.K = K;
    a.N = N;
    for (int g = 0; g < 2; ++g) {
        a.w[g] = static_cast<const uint8_t*>(v[g].codes);
        a.ws[g] = v[g].scales;
        a.w_row[g] = v[g].row_stride;
        a.w_expert[g] = v[g].expert_stride;
        a.ws_row[g] = v[g].scale_row_stride;
        a.ws_expert[g] = v[g].scale_expert_stride;
    }
    a.y = static_cast<uint8_t*>(y->data);
    a.ys = y->scales;
    a.y_stride = yst;
    a.ys_stride = yss;
    a.dtype = y->dtype;
    a.glu = glu;
    const dim3 grid((N + 127) / 128, (M + kSimpleRows - 1) / kSimpleRows + (experts ? E : 0));
    if (grid.y > 65535) return NQ_ERR_SHAPE;
    return step_launch(fp8_simple_kernel, grid, dim3(kSimpleThreads), 0, reinterpret_cast<cudaStream_t>(stream), d.pdl, 1,
                       a) == cudaSuccess
               ? NQ_OK
               : NQ_ERR_CUDA;
}

}  // namespace
}  // namespace nq

using namespace nq;

extern "C" {

nq_status nq_gemm_fp8(const nq_fp8_rows* x, const nq_fp8_weight* w, const nq_fp8_out* y, int K, int N, void* stream) {
    return fp8_call(x, false, nullptr, x ? x->rows : 0, nullptr, 1, w, nullptr, false, y, K, N, stream);
}

nq_status nq_swiglu_fp8(const nq_fp8_rows* x, const nq_fp8_weight* wg, const nq_fp8_weight* wu, const nq_fp8_out* h,
                        int K, int N, void* stream) {
    return fp8_call(x, false, nullptr, x ? x->rows : 0, nullptr, 1, wg, wu, true, h, K, N, stream);
}

nq_status nq_gemm_fp8_experts(const nq_fp8_rows* x, const int* rows, int M, const int* offsets, int E,
                              const nq_fp8_weight* w, const nq_fp8_out* y, int K, int N, void* stream) {
    return fp8_call(x, true, rows, M, offsets, E, w, nullptr, false, y, K, N, stream);
}

nq_status nq_swiglu_fp8_experts(const nq_fp8_rows* x, const int* rows, int M, const int* offsets, int E,
                                const nq_fp8_weight* wg, const nq_fp8_weight* wu, const nq_fp8_out* h, int K, int N,
                                void* stream) {
    return fp8_call(x, true, rows, M, offsets, E, wg, wu, true, h, K, N, stream);
}

}  // extern "C"
