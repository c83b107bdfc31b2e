// The projections into and out of a layer, out = act(x W^T + bias) +
// residual, and their backward: entry points, the fp32 product on CUDA cores
// and the elementwise pass of the backward.
#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kSgBM = 64, kSgBN = 64, kSgBK = 16, kSgThreads = 256;

// Element (m, n) of the product sum_k A(m, k) B(n, k), both operands with
// strides of their own (one of each is 1): the tile is staged transposed,
// k-major, so that the inner product reads whole vectors.
template <typename T, typename TO, bool kAContigK, bool kBContigK>
__global__ void __launch_bounds__(kSgThreads)
linear_simt_kernel(const T *__restrict__ A, const T *__restrict__ B, LinearEpilogue ep, int64_t M, int64_t N, int64_t K,
                   int64_t lda, int64_t ldb) {
    __shared__ float sA[kSgBK][kSgBM + 4];
    __shared__ float sB[kSgBK][kSgBN + 4];
    const int tid = threadIdx.x;
    const int64_t m0 = (int64_t)blockIdx.y * kSgBM, n0 = (int64_t)blockIdx.x * kSgBN;
    const int tm = (tid / 16) * 4, tn = (tid % 16) * 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kSgBK) {
        for (int i = tid; i < kSgBM * kSgBK; i += kSgThreads) {
            const int k = kAContigK ? i % kSgBK : i / kSgBM, m = kAContigK ? i / kSgBK : i % kSgBM;
            const bool in = m0 + m < M && k0 + k < K;
            sA[k][m] = in ? to_f(A[kAContigK ? (m0 + m) * lda + k0 + k : (k0 + k) * lda + m0 + m]) : 0.0f;
        }
        for (int i = tid; i < kSgBN * kSgBK; i += kSgThreads) {
            const int k = kBContigK ? i % kSgBK : i / kSgBN, n = kBContigK ? i / kSgBK : i % kSgBN;
            const bool in = n0 + n < N && k0 + k < K;
            sB[k][n] = in ? to_f(B[kBContigK ? (n0 + n) * ldb + k0 + k : (k0 + k) * ldb + n0 + n]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSgBK; ++k) {
            const float4 a = *reinterpret_cast<const float4 *>(&sA[k][tm]);
            const float4 b = *reinterpret_cast<const float4 *>(&sB[k][tn]);
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + tm + i;
        if (m >= M) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tn + j;
            if (n >= N) break;
            float z = acc[i][j] + (ep.bias ? ep.bias[n] : 0.0f);
            if (ep.preact) static_cast<T *>(ep.preact)[m * N + n] = linear_from_f<T>(z);
            z = linear_act(z, ep.act);
            if (ep.residual) z += to_f(static_cast<const TO *>(ep.residual)[m * N + n]);
            static_cast<TO *>(ep.out)[m * N + n] = linear_from_f<TO>(z);
        }
    }
}

template <typename T, typename TO>
cudaError_t simt_product(const void *A, const void *B, const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K,
                         int64_t lda, int64_t ldb, bool a_contig_k, bool b_contig_k, cudaStream_t s) {
    TraceScope tr(s, kTrLinear);
    const dim3 grid((unsigned)((N + kSgBN - 1) / kSgBN), (unsigned)((M + kSgBM - 1) / kSgBM));
    auto kern = a_contig_k ? (b_contig_k ? linear_simt_kernel<T, TO, true, true> : linear_simt_kernel<T, TO, true, false>)
                           : (b_contig_k ? linear_simt_kernel<T, TO, false, true> : linear_simt_kernel<T, TO, false, false>);
    kern<<<grid, kSgThreads, 0, s>>>((const T *)A, (const T *)B, ep, M, N, K, lda, ldb);
    return cudaGetLastError();
}

// dz = dy act'(preact), rows ld apart with zeros behind N, and its column
// sums over 64 rows.  A thread walks 64 rows of one column.
constexpr int kDzRows = 64;

template <typename T>
__global__ void __launch_bounds__(128)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, T *__restrict__ dz, float *__restrict__ part,
                 int64_t M, int64_t N, int64_t ld, int act) {
    const int64_t n = (int64_t)blockIdx.x * 128 + threadIdx.x, m0 = (int64_t)blockIdx.y * kDzRows;
    if (n >= ld) return;
    const int64_t m1 = m0 + kDzRows < M ? m0 + kDzRows : M;
    if (n >= N) {
        if (dz)
            for (int64_t m = m0; m < m1; ++m) dz[m * ld + n] = linear_from_f<T>(0.0f);
        return;
    }
    float sum = 0.0f;
    for (int64_t m = m0; m < m1; ++m) {
        float d = to_f(dy[m * N + n]);
        // rounded before it is added, so that the sum is the same whether dz is stored or not
        if (act != SSD_ACT_NONE) d = __fmul_rn(d, linear_act_slope(to_f(z[m * N + n]), act));
        sum += d;
        if (dz) dz[m * ld + n] = linear_from_f<T>(d);
    }
    if (part) part[blockIdx.y * N + n] = sum;
}

bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ssd_status check_sizes(int64_t M, int64_t N, int64_t K, int in_dtype) {
    if (M < 0 || N <= 0 || K <= 0) return SSD_ERR_INVALID_ARG;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    const int64_t most = 1ll << 31;
    if (M >= most || N >= most || K >= most || M * N >= (1ll << 38) || M * K >= (1ll << 38) || N * K >= (1ll << 38))
        return SSD_ERR_UNSUPPORTED;
    // grid rows of 64
    if (M > 65535ll * 64 || N > 65535ll * 64) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

size_t elem(int in_dtype) { return in_dtype == SSD_BF16 ? 2 : 4; }

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }

// Workspace regions after the status word, each 256-byte aligned.  bf16 rows
// that are not a multiple of 16 bytes are copied to rows that are (TMA's
// strides); dz is stored where it differs from dy.
struct Regions {
    size_t x = 0, w = 0, dz = 0, sums = 0, part = 0, total = 0;
};

Regions regions_of(int64_t M, int64_t N, int64_t K, int in_dtype, int backward) {
    Regions r;
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    const bool bf = in_dtype == SSD_BF16;
    if (bf && K % 8) {
        r.x = take((size_t)(M * up8(K)) * 2);
        r.w = take((size_t)(N * up8(K)) * 2);
    }
    if (backward) {
        r.dz = take((size_t)(M * (bf ? up8(N) : N)) * elem(in_dtype));
        r.sums = take((size_t)((M + kDzRows - 1) / kDzRows * N) * sizeof(float));
    }
    if (bf && M > 0) {
        size_t part = backward ? linear_tc_part_bytes(M, K, N) : linear_tc_part_bytes(M, N, K);
        if (backward && linear_tc_part_bytes(N, K, M) > part) part = linear_tc_part_bytes(N, K, M);
        r.part = take(part);
    }
    r.total = at;
    return r;
}

size_t ws_bytes(int64_t M, int64_t N, int64_t K, int in_dtype, int backward) {
    return regions_of(M, N, K, in_dtype, backward).total;
}

bool act_ok(int act) { return act == SSD_ACT_NONE || act == SSD_ACT_SILU || act == SSD_ACT_GELU; }

}  // namespace
}  // namespace ssd

extern "C" {

SSD_API ssd_status ssd_linear_workspace_size(int64_t rows, int64_t n_out, int64_t n_in, int in_dtype, int backward,
                                             size_t *bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return SSD_ERR_INVALID_ARG;
    const ssd_status st = ssd::check_sizes(rows, n_out, n_in, in_dtype);
    if (st == SSD_OK) *bytes = ssd::ws_bytes(rows, n_out, n_in, in_dtype, backward);
    return st;
}

SSD_API ssd_status ssd_linear_fwd(const void *x, const void *weight, const float *bias, const void *residual, void *out,
                                  void *preact, int64_t rows, int64_t n_out, int64_t n_in, int activation, int in_dtype,
                                  int out_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const ssd_status st = ssd::check_sizes(rows, n_out, n_in, in_dtype);
    if (st != SSD_OK) return st;
    if (!ssd::act_ok(activation)) return SSD_ERR_INVALID_ARG;
    if (out_dtype != in_dtype && out_dtype != SSD_F32) return SSD_ERR_UNSUPPORTED;
    if (!weight || (rows > 0 && (!x || !out))) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, weight, (const void *)bias, residual, (const void *)out, (const void *)preact})
        if (!ssd::a16(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::ws_bytes(rows, n_out, n_in, in_dtype, 0)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
    if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
    if (rows == 0) return SSD_OK;
    ssd::LinearEpilogue ep;
    ep.bias = bias; ep.residual = residual; ep.out = out; ep.preact = preact; ep.act = activation;
    if (in_dtype == SSD_F32) {
        e = ssd::simt_product<float, float>(x, weight, ep, rows, n_out, n_in, n_in, n_in, true, true, s);
    } else {
        char *ws = static_cast<char *>(workspace);
        const ssd::Regions r = ssd::regions_of(rows, n_out, n_in, in_dtype, 0);
        if (n_in % 8) {
            e = ssd::linear_pad(x, ws + r.x, rows, n_in, s);
            if (e == cudaSuccess) e = ssd::linear_pad(weight, ws + r.w, n_out, n_in, s);
            x = ws + r.x;
            weight = ws + r.w;
        }
        if (e == cudaSuccess)
            e = ssd::linear_tc(x, ssd::up8(n_in), false, weight, ssd::up8(n_in), false, ep, out_dtype == SSD_F32, rows,
                               n_out, n_in, ws + r.part, static_cast<unsigned *>(workspace), s);
    }
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

SSD_API ssd_status ssd_linear_bwd(const void *x, const void *weight, const void *dy, const void *preact, void *dx,
                                  void *dweight, float *dbias, int64_t rows, int64_t n_out, int64_t n_in, int activation,
                                  int in_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const ssd_status st = ssd::check_sizes(rows, n_out, n_in, in_dtype);
    if (st != SSD_OK) return st;
    if (!ssd::act_ok(activation)) return SSD_ERR_INVALID_ARG;
    const bool acts = activation != SSD_ACT_NONE;
    if (rows > 0 && (!dy || (acts && !preact) || (dx && !weight) || (dweight && !x))) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, weight, dy, preact, (const void *)dx, (const void *)dweight, (const void *)dbias})
        if (!ssd::a16(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::ws_bytes(rows, n_out, n_in, in_dtype, 1)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
    if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
    const size_t es = ssd::elem(in_dtype);
    if (rows == 0) {
        // no rows: the sums over them are zero
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)(n_out * n_in) * es, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)n_out * sizeof(float), s);
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    char *ws = static_cast<char *>(workspace);
    const bool bf = in_dtype == SSD_BF16;
    const ssd::Regions r = ssd::regions_of(rows, n_out, n_in, in_dtype, 1);
    void *dz = ws + r.dz;
    float *sums = reinterpret_cast<float *>(ws + r.sums);
    const int64_t ld = bf ? ssd::up8(n_out) : n_out;
    const bool store = (acts || ld != n_out) && (dx || dweight);
    if (store || dbias) {
        ssd::TraceScope tr(s, ssd::kTrLinearDz);
        const dim3 grid((unsigned)((ld + 127) / 128), (unsigned)((rows + ssd::kDzRows - 1) / ssd::kDzRows));
        if (bf)
            ssd::linear_dz_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(
                (const __nv_bfloat16 *)dy, (const __nv_bfloat16 *)preact, (__nv_bfloat16 *)(store ? dz : nullptr),
                dbias ? sums : nullptr, rows, n_out, ld, activation);
        else
            ssd::linear_dz_kernel<float><<<grid, 128, 0, s>>>((const float *)dy, (const float *)preact,
                                                              (float *)(store ? dz : nullptr), dbias ? sums : nullptr,
                                                              rows, n_out, ld, activation);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && dbias)
        e = ssd::column_sum(sums, dbias, nullptr, (rows + ssd::kDzRows - 1) / ssd::kDzRows, n_out, n_out, s);
    const void *d = store ? dz : dy;
    if (bf && n_in % 8) {
        if (e == cudaSuccess && dx) e = ssd::linear_pad(weight, ws + r.w, n_out, n_in, s);
        if (e == cudaSuccess && dweight) e = ssd::linear_pad(x, ws + r.x, rows, n_in, s);
        weight = ws + r.w;
        x = ws + r.x;
    }
    unsigned *status = static_cast<unsigned *>(workspace);
    ssd::LinearEpilogue ex, ew;
    ex.out = dx;
    ew.out = dweight;
    if (e == cudaSuccess && dx)
        e = bf ? ssd::linear_tc(d, ld, false, weight, ssd::up8(n_in), true, ex, 0, rows, n_in, n_out, ws + r.part, status, s)
               : ssd::simt_product<float, float>(d, weight, ex, rows, n_in, n_out, n_out, n_in, true, false, s);
    if (e == cudaSuccess && dweight)
        e = bf ? ssd::linear_tc(d, ld, true, x, ssd::up8(n_in), true, ew, 0, n_out, n_in, rows, ws + r.part, status, s)
               : ssd::simt_product<float, float>(d, x, ew, n_out, n_in, rows, n_out, n_in, false, false, s);
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

}  // extern "C"
