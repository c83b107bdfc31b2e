// The projections (ssd_linear_*): what the entry points and kernels share.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "ssd_common.cuh"

namespace ssd {

// out = act(acc + bias) + residual for element (m, n) of an [M, N] product
struct LinearEpilogue {
    const float *bias = nullptr;       // [N] or null
    const void *residual = nullptr;    // [M, N] in the output's type, or null
    void *out = nullptr;               // [M, N]
    void *preact = nullptr;            // [M, N] in the operands' type, or null
    int act = SSD_ACT_NONE;
    int pre_f32 = 0;                   // preact is fp32 (fp32 operands)
};

// Launches a kernel that may start before the one of this library ahead of it in
// the stream has ended (pdl), and waits for it (pdl_wait_prerequisites) before
// it reads or writes what is shared.
template <typename... P, typename... A>
cudaError_t linear_launch(void (*kern)(P...), unsigned blocks, unsigned threads, size_t smem, bool pdl, cudaStream_t s, A... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&c, kern, P(args)...);
}

// The activations and their slopes, for a result of type T.  float32: to a few
// roundings of the result over the whole range, by the library's exponential, and
// sigmoids from e^-|z|, so that neither side overflows or cancels (what is divided
// by is in [1, 2], where the fast division is within 2 units in the last place; the
// other's branches held the loads of dz back: 333 x 1001 x 771 backward 63 and 67 us).
// bf16: by the fast exponential, which is off by the rounding of its argument
// (6e-6 of the result at |z| = 100, 1e-6 below 16) where the store rounds by up to
// 2^-8; the library's took 8192 x 5120 x 2560 with silu from 135 to 188 us.
template <typename T> __device__ __forceinline__ float linear_act(float z, int act) {
    if (act == SSD_ACT_SILU) {
        if constexpr (sizeof(T) == 2) return silu_f(z);
        const float e = expf(-fabsf(z));
        return __fdividef(z < 0.0f ? z * e : z, 1.0f + e);
    }
    if (act == SSD_ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z;
}

// act'(z)
template <typename T> __device__ __forceinline__ float linear_act_slope(float z, int act) {
    if constexpr (sizeof(T) == 2) {
        if (act == SSD_ACT_SILU) {
            const float q = __fdividef(1.0f, 1.0f + __expf(-z));
            return q * fmaf(z, 1.0f - q, 1.0f);
        }
        if (act == SSD_ACT_GELU)
            return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z), 0.5f + 0.5f * erff(z * 0.70710678118654752f));
        return 1.0f;
    } else {
        if (act == SSD_ACT_SILU) {   // s + z s (1 - s)
            const float e = expf(-fabsf(z)), q = __fdividef(1.0f, 1.0f + e), p = e * q;
            return (z < 0.0f ? p : q) * fmaf(z, z < 0.0f ? q : p, 1.0f);
        }
        if (act == SSD_ACT_GELU)
            return fmaf(z * 0.39894228040143268f, expf(-0.5f * z * z), 0.5f + 0.5f * erff(z * 0.70710678118654752f));
        return 1.0f;
    }
}

// ---- bf16 products on the tensor cores (ssd_linear_tc.cu)
// D[m, n] = sum_k A(m, k) B(n, k), then the epilogue.  An operand runs along k
// (rows of k, ld apart) or, with *_mn, along its own index (rows of m or n,
// one per k).  ld a multiple of 8 elements, 16-byte aligned.  terms 2 (b_mn): A is
// the sum of two matrices, the second `plane` of its rows in memory after the first; `plane` is a
// multiple of 64, and with a_mn the rows between are zeros.  `part`: scratch of
// linear_tc_part_bytes(M, N, K, b_mn, terms); out_f32: out and residual are fp32; clear:
// *status is set to 0 first.
size_t linear_tc_part_bytes(int64_t M, int64_t N, int64_t K, bool b_mn, int terms = 1);
cudaError_t linear_tc(const void *A, int64_t lda, bool a_mn, const void *B, int64_t ldb, bool b_mn,
                      const LinearEpilogue &ep, int out_f32, int64_t M, int64_t N, int64_t K, void *part, unsigned *status,
                      bool clear, cudaStream_t s, int terms = 1, int64_t plane = 0);
// ---- fp32 products on the tensor cores, in bf16 parts (ssd_linear_tc.cu)
// Whether they beat `other_cycles`; an operand's parts (linear_parts_bytes of
// its rows and columns in memory, either matrix may be null) serve it along k
// and along its own rows.
bool linear_parts_pay(int64_t M, int64_t N, int64_t K, bool b_mn, double other_cycles);
size_t linear_parts_bytes(int64_t rows, int64_t cols);
size_t linear_parts_sum_bytes(int64_t M, int64_t N, int64_t K, bool b_mn);
cudaError_t linear_parts(const float *a, int64_t a_rows, int64_t a_cols, void *a_parts, const float *b, int64_t b_rows, int64_t b_cols,
                         void *b_parts, cudaStream_t st);
cudaError_t linear_tc_parts(const void *A, bool a_mn, const void *B, bool b_mn, const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K,
                            void *part, unsigned *status, bool clear, cudaStream_t st);
// ---- few bf16 rows, forward (ssd_linear_rows.cu); any K.  Clears *status.
constexpr int64_t kLrMost = 32;
cudaError_t linear_rows(const void *x, const void *W, const LinearEpilogue &ep, int out_f32, int64_t M, int64_t N, int64_t K,
                        unsigned *status, cudaStream_t s);
// ---- fp32 products on the CUDA cores (ssd_linear_f32.cu): as linear_tc, any
// strides, one of each operand's being 1; status, if any, is cleared.
double linear_f32_cycles(int64_t M, int64_t N, int64_t K);   // its estimate
cudaError_t linear_f32(const float *A, int64_t lda, bool a_mn, const float *B, int64_t ldb, bool b_mn,
                       const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K, unsigned *status, cudaStream_t s);
// The parts of k, [splits, M, N], added in order, then the epilogue.
template <typename TO>
cudaError_t linear_join(const float *part, const LinearEpilogue &ep, int64_t M, int64_t N, int splits, cudaStream_t s);
// Rows of `cols` bf16 copied to rows of a multiple of 8, zeros behind.
cudaError_t linear_pad(const void *src, void *dst, int64_t rows, int64_t cols, cudaStream_t s);

template <typename T> __device__ __forceinline__ T linear_from_f(float v);
template <> __device__ __forceinline__ float linear_from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 linear_from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

}  // namespace ssd
