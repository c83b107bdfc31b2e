// The projections into and out of a layer, out = act(x W^T + bias) +
// residual, and their backward: entry points, the join of parts of k and the
// elementwise pass of the backward.
#include <initializer_list>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_tc.cuh"
#include "ssd_trace.h"

namespace ssd {
namespace {

template <typename TO>
__global__ void __launch_bounds__(256)
linear_join_kernel(const float *__restrict__ part, LinearEpilogue ep, int64_t MN, int N, int splits) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    tc::pdl_wait_prerequisites();   // the parts' sums
    if (i >= MN) return;
    float z = 0.0f;
#pragma unroll 4
    for (int k = 0; k < splits; ++k) z += part[k * MN + i];
    if (ep.bias) z += ep.bias[MN >> 32 ? (int)(i % N) : (int)((uint32_t)i % (uint32_t)N)];
    if (ep.preact) {
        if (ep.pre_f32) static_cast<float *>(ep.preact)[i] = z;
        else static_cast<__nv_bfloat16 *>(ep.preact)[i] = __float2bfloat16_rn(z);
    }
    z = linear_act<TO>(z, ep.act);
    if (ep.residual) z += to_f(static_cast<const TO *>(ep.residual)[i]);
    static_cast<TO *>(ep.out)[i] = linear_from_f<TO>(z);
}

// dz = dy act'(preact), rows ld apart with zeros behind N, and its column
// sums over 64 rows (of the float32 values).  A bf16 dz is rounded once, where it
// becomes an operand of the two products: by up to 2^-8 of a value, next to the
// roundings that dy and x carry already.  Its gradients are 1.4 times as far from 64 bits as with dz
// whole (8192 x 5120 x 2560: 0.0023 and 0.0017 of their size, bf16 stores included); a
// caller who wants that asks for kWide, which stores what the rounding leaves as a second
// matrix `low` behind (with zeros in the rows up to a multiple of 64) and
// takes twice the products (695 us for 345).  A block takes 64 rows of 256 columns: a thread 8 columns
// (16 bytes of bf16, where kVec) of every eighth row; its sums of 8 rows are added in
// order.  Bound by HBM: 6 bytes a value of bf16 with an activation.
constexpr int kDzRows = 64, kDzCols = 256;

template <typename T> struct Eight;
template <> struct Eight<float> {
    static __device__ __forceinline__ void get(const float *p, float (&v)[8]) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void put(float *p, const float (&v)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    static __device__ __forceinline__ void get(const __nv_bfloat16 *p, float (&v)[8]) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// What bf16's rounding leaves of v (nothing of an infinity).
__device__ __forceinline__ float rest_of(float v) {
    const float hi = __bfloat162float(__float2bfloat16_rn(v));
    return fabsf(hi) <= 3.402823466e38f ? v - hi : 0.0f;
}

// kVec: rows of dy and preact start on 8 elements
template <typename T, bool kVec, bool kWide>
__global__ void __launch_bounds__(256)
linear_dz_kernel(const T *__restrict__ dy, const T *__restrict__ z, T *__restrict__ dz, float *__restrict__ part,
                 int64_t M, int64_t N, int64_t ld, int act, int64_t low) {
    __shared__ float s_sum[8][kDzCols + 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned by = blockIdx.z * 65535u + blockIdx.y;   // (rows may be more than a grid's second axis takes)
    const int64_t n = (int64_t)blockIdx.x * kDzCols + lane * 8, m0 = (int64_t)by * kDzRows + warp;
    if ((int64_t)by * kDzRows >= M) return;
    float sum[8] = {};
    if (n < ld) {
#pragma unroll 4
        for (int i = 0; i < kDzRows / 8; ++i) {
            const int64_t m = m0 + 8 * i;
            float d[8], q[8];
            if (m >= M) {
                if (!kWide) break;
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = 0.0f;
            } else if (kVec) {
                Eight<T>::get(dy + m * N + n, d);
                if (act != SSD_ACT_NONE) Eight<T>::get(z + m * N + n, q);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[j] = n + j < N ? to_f(dy[m * N + n + j]) : 0.0f;
                    q[j] = act != SSD_ACT_NONE && n + j < N ? to_f(z[m * N + n + j]) : 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // rounded before it is added, so that the sum is the same whether dz is stored or not
                if (act != SSD_ACT_NONE && (kVec || n + j < N) && (!kWide || m < M)) d[j] = __fmul_rn(d[j], linear_act_slope<T>(q[j], act));
                sum[j] += d[j];
            }
            if (dz) {
                if (kVec) {
                    Eight<T>::put(dz + m * ld + n, d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < ld) dz[m * ld + n + j] = linear_from_f<T>(d[j]);
                }
            }
            if constexpr (kWide) {
                T *rest = dz + low;
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = rest_of(d[j]);
                if (kVec) {
                    Eight<T>::put(rest + m * ld + n, d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < ld) rest[m * ld + n + j] = linear_from_f<T>(d[j]);
                }
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) s_sum[warp][lane * 8 + j] = sum[j];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kDzCols + threadIdx.x;
    if (c < N) {
        float t = s_sum[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < 8; ++k) t += s_sum[k][threadIdx.x];
        part[by * N + c] = t;
    }
}

template <typename T, bool kWide = false>
cudaError_t dz_launch(const void *dy, const void *z, void *dz, float *part, int64_t M, int64_t N, int64_t ld, int act,
                      int64_t low, cudaStream_t s) {
    TraceScope tr(s, kTrLinearDz);
    const unsigned cols = (unsigned)((ld + kDzCols - 1) / kDzCols), rows = (unsigned)((M + kDzRows - 1) / kDzRows);
    const dim3 grid(cols, rows < 65535u ? rows : 65535u, (rows + 65534u) / 65535u);
    (N % 8 == 0 ? linear_dz_kernel<T, true, kWide> : linear_dz_kernel<T, false, kWide>)<<<grid, 256, 0, s>>>(
        (const T *)dy, (const T *)z, (T *)dz, part, M, N, ld, act, low);
    return cudaGetLastError();
}

bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ssd_status check_sizes(int64_t M, int64_t N, int64_t K, int in_dtype, bool wide = false) {
    if (M < 0 || N <= 0 || K <= 0) return SSD_ERR_INVALID_ARG;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    const int64_t most = (1ll << 31) - 512;   // (a tile's last coordinate fits 31 bits)
    if (M >= most || N >= most || K >= most || M * N >= (1ll << 38) || M * K >= (1ll << 38) || N * K >= (1ll << 38))
        return SSD_ERR_UNSUPPORTED;
    if (wide && M >= (1ll << 30) - 512) return SSD_ERR_UNSUPPORTED;   // both parts' rows in one map
    return SSD_OK;
}

size_t elem(int in_dtype) { return in_dtype == SSD_BF16 ? 2 : 4; }

int64_t up8(int64_t v) { return (v + 7) / 8 * 8; }
int64_t dz_plane(int64_t M) { return (M + kDzRows - 1) / kDzRows * kDzRows; }   // rows of one part of a wide dz

// Workspace regions after the status word, each 256-byte aligned.  bf16 rows
// that are not a multiple of 16 bytes are copied to rows that are (TMA's
// strides); dz is stored where it differs from dy.
struct Regions {
    size_t x = 0, w = 0, dz = 0, sums = 0, part = 0, dz_parts = 0, total = 0;
    bool parts = false;   // fp32 products on the tensor cores: x, w and dz_parts hold the operands' parts
};

// fp32: the tensor cores where they are estimated faster, both products of a
// backward alike.  2048 x 2560 x 2560 takes 190 us there and 603 on the CUDA cores,
// 333 x 1001 x 771 19 and 27; 128 x 2000 x 500 stays on the CUDA cores (14).
bool use_parts(int64_t M, int64_t N, int64_t K, int backward) {
    if (M == 0) return false;
    if (!backward) return linear_parts_pay(M, N, K, false, linear_f32_cycles(M, N, K));
    return linear_parts_pay(M, K, N, true, linear_f32_cycles(M, K, N)) && linear_parts_pay(N, K, M, true, linear_f32_cycles(N, K, M));
}

// backward 2: dz in two parts
Regions regions_of(int64_t M, int64_t N, int64_t K, int in_dtype, int backward) {
    Regions r;
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    const bool bf = in_dtype == SSD_BF16;
    if (bf && K % 8 && (backward || M > kLrMost)) {
        r.x = take((size_t)(M * up8(K)) * 2);
        r.w = take((size_t)(N * up8(K)) * 2);
    }
    if (backward) {
        r.dz = take((size_t)((bf && backward == 2 ? 2 * dz_plane(M) : M) * (bf ? up8(N) : N)) * elem(in_dtype));
        r.sums = take((size_t)((M + kDzRows - 1) / kDzRows * N) * sizeof(float));
    }
    if (bf && M > 0) {
        size_t part = !backward && M > kLrMost ? linear_tc_part_bytes(M, N, K, false) : 0;
        for (int terms = 1; terms <= backward; ++terms)
            for (const size_t p : {linear_tc_part_bytes(M, K, N, true, terms), linear_tc_part_bytes(N, K, M, true, terms)})
                if (p > part) part = p;
        r.part = take(part);
    }
    if (!bf && use_parts(M, N, K, backward)) {
        r.parts = true;
        r.x = take(linear_parts_bytes(M, K));
        r.w = take(linear_parts_bytes(N, K));
        size_t part = backward ? linear_parts_sum_bytes(M, K, N, true) : linear_parts_sum_bytes(M, N, K, false);
        if (backward) {
            r.dz_parts = take(linear_parts_bytes(M, N));
            if (linear_parts_sum_bytes(N, K, M, true) > part) part = linear_parts_sum_bytes(N, K, M, true);
        }
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

template <typename TO>
cudaError_t linear_join(const float *part, const LinearEpilogue &ep, int64_t M, int64_t N, int splits, cudaStream_t s) {
    return linear_launch(linear_join_kernel<TO>, (unsigned)((M * N + 255) / 256), 256, 0, true, s, part, ep, M * N, (int)N, splits);
}
template cudaError_t linear_join<float>(const float *, const LinearEpilogue &, int64_t, int64_t, int, cudaStream_t);
template cudaError_t linear_join<__nv_bfloat16>(const float *, const LinearEpilogue &, int64_t, int64_t, int, cudaStream_t);

}  // namespace ssd

extern "C" {

SSD_API ssd_status ssd_linear_workspace_size(int64_t rows, int64_t n_out, int64_t n_in, int in_dtype, int backward,
                                             size_t *bytes) {
    if (!bytes || backward < 0 || backward > 2) return SSD_ERR_INVALID_ARG;
    const ssd_status st = ssd::check_sizes(rows, n_out, n_in, in_dtype, backward == 2);
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
    ssd::LinearEpilogue ep;
    ep.bias = bias; ep.residual = residual; ep.out = out; ep.preact = preact; ep.act = activation;
    cudaError_t e = cudaSuccess;
    if (in_dtype == SSD_BF16 && rows > 0 && rows <= ssd::kLrMost) {
        e = ssd::linear_rows(x, weight, ep, out_dtype == SSD_F32, rows, n_out, n_in, static_cast<unsigned *>(workspace), s);
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    // the kernels clear the status word themselves
    if (rows == 0) e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
    if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
    if (rows == 0) return SSD_OK;
    char *ws = static_cast<char *>(workspace);
    const ssd::Regions r = ssd::regions_of(rows, n_out, n_in, in_dtype, 0);
    ep.pre_f32 = in_dtype == SSD_F32;
    if (r.parts) {
        e = ssd::linear_parts((const float *)x, rows, n_in, ws + r.x, (const float *)weight, n_out, n_in, ws + r.w, s);
        if (e == cudaSuccess)
            e = ssd::linear_tc_parts(ws + r.x, false, ws + r.w, false, ep, rows, n_out, n_in, ws + r.part,
                                     static_cast<unsigned *>(workspace), true, s);
    } else if (in_dtype == SSD_F32) {
        e = ssd::linear_f32((const float *)x, n_in, false, (const float *)weight, n_in, false, ep, rows, n_out, n_in,
                            static_cast<unsigned *>(workspace), s);
    } else {
        if (n_in % 8) {
            e = ssd::linear_pad(x, ws + r.x, rows, n_in, s);
            if (e == cudaSuccess) e = ssd::linear_pad(weight, ws + r.w, n_out, n_in, s);
            x = ws + r.x;
            weight = ws + r.w;
        }
        if (e == cudaSuccess)
            e = ssd::linear_tc(x, ssd::up8(n_in), false, weight, ssd::up8(n_in), false, ep, out_dtype == SSD_F32, rows,
                               n_out, n_in, ws + r.part, static_cast<unsigned *>(workspace), true, s);
    }
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

SSD_API ssd_status ssd_linear_bwd(const void *x, const void *weight, const void *dy, const void *preact, void *dx,
                                  void *dweight, float *dbias, int64_t rows, int64_t n_out, int64_t n_in, int activation,
                                  int in_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const int asked = activation;
    if (activation > 0) activation &= ~SSD_DZ_WIDE;
    const bool acts = activation != SSD_ACT_NONE;
    const int back = activation != asked ? 2 : 1;
    const bool wide = back == 2 && acts && in_dtype == SSD_BF16;   // (else dz is whole as it is)
    const ssd_status st = ssd::check_sizes(rows, n_out, n_in, in_dtype, back == 2);
    if (st != SSD_OK) return st;
    if (!ssd::act_ok(activation)) return SSD_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || (acts && !preact) || (dx && !weight) || (dweight && !x))) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, weight, dy, preact, (const void *)dx, (const void *)dweight, (const void *)dbias})
        if (!ssd::a16(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::ws_bytes(rows, n_out, n_in, in_dtype, back)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    // the first product clears the status word itself
    if (rows == 0 || !(dx || dweight)) e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
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
    const ssd::Regions r = ssd::regions_of(rows, n_out, n_in, in_dtype, back);
    void *dz = ws + r.dz;
    float *sums = reinterpret_cast<float *>(ws + r.sums);
    const int64_t ld = bf ? ssd::up8(n_out) : n_out;
    const bool store = (acts || ld != n_out) && (dx || dweight);
    if (store || dbias) {
        e = (!bf ? ssd::dz_launch<float> : wide && store ? ssd::dz_launch<__nv_bfloat16, true> : ssd::dz_launch<__nv_bfloat16>)(
            dy, preact, store ? dz : nullptr, dbias ? sums : nullptr, rows, n_out, ld, activation, ssd::dz_plane(rows) * ld, s);
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
    if (r.parts && (dx || dweight)) {
        if (e == cudaSuccess)
            e = ssd::linear_parts((const float *)(dweight ? x : nullptr), rows, n_in, ws + r.x, (const float *)(dx ? weight : nullptr), n_out,
                                  n_in, ws + r.w, s);
        if (e == cudaSuccess) e = ssd::linear_parts((const float *)d, rows, n_out, ws + r.dz_parts, nullptr, 0, 0, nullptr, s);
        if (e == cudaSuccess && dx)
            e = ssd::linear_tc_parts(ws + r.dz_parts, false, ws + r.w, true, ex, rows, n_in, n_out, ws + r.part, status, true, s);
        if (e == cudaSuccess && dweight)
            e = ssd::linear_tc_parts(ws + r.dz_parts, true, ws + r.x, true, ew, n_out, n_in, rows, ws + r.part, status, !dx, s);
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    if (e == cudaSuccess && dx)
        e = bf ? ssd::linear_tc(d, ld, false, weight, ssd::up8(n_in), true, ex, 0, rows, n_in, n_out, ws + r.part, status, true, s, wide ? 2 : 1,
                             wide ? ssd::dz_plane(rows) : 0)
               : ssd::linear_f32((const float *)d, n_out, false, (const float *)weight, n_in, true, ex, rows, n_in, n_out,
                               status, s);
    if (e == cudaSuccess && dweight)
        e = bf ? ssd::linear_tc(d, ld, true, x, ssd::up8(n_in), true, ew, 0, n_out, n_in, rows, ws + r.part, status, !dx, s, wide ? 2 : 1,
                             wide ? ssd::dz_plane(rows) : 0)
               : ssd::linear_f32((const float *)d, n_out, true, (const float *)x, n_in, true, ew, n_out, n_in, rows,
                               dx ? nullptr : status, s);
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

}  // extern "C"
