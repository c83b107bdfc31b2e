// RMS norm of B and C over each group's state_dim values, and the rotation of
// their pairs by the token's position, in one pass; and its backward.
//   n = v rs w,  rs = 1 / sqrt(mean(v^2) + eps)
//   (p, q) -> (p cos A - q sin A, q cos A + p sin A),  A = position * inv_freq
// Backward: dn = the gradient rotated by -A,
//   dw += dn v rs,   dv = rs (dn w - v rs mean(dn w v rs)).
//
// The angle.  A position can be any 32-bit integer, where position * inv_freq
// in float32 has lost the angle, so the turn inv_freq / 2 pi is held as a
// 64-bit fixed-point fraction and multiplied by the position in integers:
// the product modulo 2^64 is the angle modulo one turn, exactly.
#include <math.h>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kNrWarps = 8;
constexpr int64_t kNrMaxWarps = 148 * 32;   // warps of a backward launch: rows of weight partials

// inv_freq (radians per position) as turns per position, modulo 1, in 2^-64
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
    double f = (double)inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
    f -= floor(f);
    return (uint64_t)(int64_t)llrint((f >= 0.5 ? f - 1.0 : f) * 18446744073709551616.0);
}

// cos and sin of position * turns
__device__ __forceinline__ void turn(int position, uint64_t turns, float &c, float &s) {
    const uint64_t t = (uint64_t)(int64_t)position * turns;
    // the top 32 bits as a signed count of 2^-31 half turns
    sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &s, &c);
}

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The elements of pair j: the rotated ones first, then the rest two by two
// (an odd last element has no partner: second = N).
__device__ __forceinline__ void pair_of(int j, int N, int R, int interleaved, int &e0, int &e1) {
    const int H = R >> 1;
    if (j < H) {
        e0 = interleaved ? 2 * j : j;
        e1 = interleaved ? 2 * j + 1 : j + H;
    } else {
        e0 = R + 2 * (j - H);
        e1 = e0 + 1;
    }
}

// One warp per (token, group), lanes across pairs, B then C.
template <typename T>
__global__ void __launch_bounds__(32 * kNrWarps)
norm_rotate_kernel(const T *__restrict__ B, const T *__restrict__ C, const float *__restrict__ wB,
                   const float *__restrict__ wC, const float *__restrict__ inv_freq,
                   const int32_t *__restrict__ positions, T *__restrict__ Bo, T *__restrict__ Co, int64_t rows, int64_t L,
                   int G, int N, int R, float eps, int interleaved) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kNrWarps + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t tok = row / G;
    const int pos = positions ? positions[tok] : (int)(tok % L);
    const int np = (N + 1) / 2;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const T *v = (which ? C : B) + row * N;
        T *o = (which ? Co : Bo) + row * N;
        const float *w = which ? wC : wB;
        float ss = 0.0f;
        for (int e = lane; e < N; e += 32) ss = fmaf(to_f(v[e]), to_f(v[e]), ss);
        const float rs = 1.0f / sqrtf(warp_sum(ss) / (float)N + eps);
        for (int j = lane; j < np; j += 32) {
            int e0, e1;
            pair_of(j, N, R, interleaved, e0, e1);
            float p = to_f(v[e0]) * rs * w[e0], q = e1 < N ? to_f(v[e1]) * rs * w[e1] : 0.0f;
            if (j < R / 2) {
                float c, s;
                turn(pos, turns_of(inv_freq[j]), c, s);
                const float p1 = p * c - q * s;
                q = q * c + p * s;
                p = p1;
            }
            o[e0] = from_f<T>(p);
            if (e1 < N) o[e1] = from_f<T>(q);
        }
    }
}

// Backward: warp i takes rows i, i + warps, ...; its weight partials are row
// i of part [warps, 2, N], which only its own lanes touch.
template <typename T>
__global__ void __launch_bounds__(32 * kNrWarps)
norm_rotate_bwd_kernel(const T *__restrict__ B, const T *__restrict__ C, const float *__restrict__ wB,
                       const float *__restrict__ wC, const float *__restrict__ inv_freq,
                       const int32_t *__restrict__ positions, const T *__restrict__ dBo, const T *__restrict__ dCo,
                       T *__restrict__ dB, T *__restrict__ dC, float *__restrict__ part, int64_t rows, int64_t warps,
                       int64_t L, int G, int N, int R, float eps, int interleaved) {
    const int lane = threadIdx.x & 31;
    const int64_t me = (int64_t)blockIdx.x * kNrWarps + (threadIdx.x >> 5);
    if (me >= warps) return;
    const int np = (N + 1) / 2;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const float *w = which ? wC : wB;
        float *acc = part + (me * 2 + which) * N;
        for (int64_t row = me; row < rows; row += warps) {
            const T *v = (which ? C : B) + row * N, *g = (which ? dCo : dBo) + row * N;
            T *o = (which ? dC : dB) + row * N;
            const int64_t tok = row / G;
            const int pos = positions ? positions[tok] : (int)(tok % L);
            float ss = 0.0f;
            for (int e = lane; e < N; e += 32) ss = fmaf(to_f(v[e]), to_f(v[e]), ss);
            const float rs = 1.0f / sqrtf(warp_sum(ss) / (float)N + eps);
            float m = 0.0f;
            for (int pass = 0; pass < 2; ++pass) {
                for (int j = lane; j < np; j += 32) {
                    int e0, e1;
                    pair_of(j, N, R, interleaved, e0, e1);
                    float p = to_f(g[e0]), q = e1 < N ? to_f(g[e1]) : 0.0f;
                    if (j < R / 2) {
                        float c, s;
                        turn(pos, turns_of(inv_freq[j]), c, s);
                        const float p1 = p * c + q * s;
                        q = q * c - p * s;
                        p = p1;
                    }
                    const float n0 = to_f(v[e0]) * rs, n1 = e1 < N ? to_f(v[e1]) * rs : 0.0f;
                    const float d0 = p * w[e0], d1 = e1 < N ? q * w[e1] : 0.0f;
                    if (pass == 0) {
                        m = fmaf(d0, n0, fmaf(d1, n1, m));
                        acc[e0] = (row == me ? 0.0f : acc[e0]) + p * n0;
                        if (e1 < N) acc[e1] = (row == me ? 0.0f : acc[e1]) + q * n1;
                    } else {
                        o[e0] = from_f<T>(rs * (d0 - n0 * m));
                        if (e1 < N) o[e1] = from_f<T>(rs * (d1 - n1 * m));
                    }
                }
                if (pass == 0) m = warp_sum(m) / (float)N;
            }
        }
    }
}

bool a16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ssd_status check_sizes(int64_t b, int64_t L, int64_t G, int64_t N) {
    if (b < 0 || L < 0 || G <= 0 || N <= 0) return SSD_ERR_INVALID_ARG;
    if (N > 8192 || G > 65535 || L >= (1ll << 31) || b >= (1ll << 31) || b * L >= (1ll << 33) ||
        b * L * G >= (1ll << 33))
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t bwd_warps(int64_t rows) { return rows < kNrMaxWarps ? rows : kNrMaxWarps; }

size_t bwd_bytes(int64_t rows, int64_t N) {
    return align256((size_t)bwd_warps(rows) * 2 * N * sizeof(float)) + align256(2 * N * sizeof(float));
}

ssd_status check_args(const float *wB, const float *wC, const float *inv_freq, const int32_t *positions, int64_t N,
                      int64_t R, float eps, int interleaved, int in_dtype) {
    if (R < 0 || R > N || R % 2 != 0 || !(eps >= 0.0f) || (interleaved != 0 && interleaved != 1))
        return SSD_ERR_INVALID_ARG;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (!wB || !wC || (R > 0 && !inv_freq)) return SSD_ERR_INVALID_ARG;
    if (!a16(wB) || !a16(wC) || ((reinterpret_cast<uintptr_t>(inv_freq) | reinterpret_cast<uintptr_t>(positions)) & 3u))
        return SSD_ERR_ALIGNMENT;
    return SSD_OK;
}

template <typename T>
void fwd_launch(const void *B, const void *C, const float *wB, const float *wC, const float *f, const int32_t *pos,
                void *Bo, void *Co, int64_t rows, int64_t L, int G, int N, int R, float eps, int il, cudaStream_t s) {
    TraceScope tr(s, kTrNormRotate);
    norm_rotate_kernel<T><<<(unsigned)((rows + kNrWarps - 1) / kNrWarps), 32 * kNrWarps, 0, s>>>(
        (const T *)B, (const T *)C, wB, wC, f, pos, (T *)Bo, (T *)Co, rows, L, G, N, R, eps, il);
}

template <typename T>
void bwd_launch(const void *B, const void *C, const float *wB, const float *wC, const float *f, const int32_t *pos,
                const void *dBo, const void *dCo, void *dB, void *dC, float *part, int64_t rows, int64_t L, int G, int N,
                int R, float eps, int il, cudaStream_t s) {
    TraceScope tr(s, kTrNormRotateBwd);
    const int64_t warps = bwd_warps(rows);
    norm_rotate_bwd_kernel<T><<<(unsigned)((warps + kNrWarps - 1) / kNrWarps), 32 * kNrWarps, 0, s>>>(
        (const T *)B, (const T *)C, wB, wC, f, pos, (const T *)dBo, (const T *)dCo, (T *)dB, (T *)dC, part, rows, warps,
        L, G, N, R, eps, il);
}

}  // namespace
}  // namespace ssd

extern "C" {

SSD_API ssd_status ssd_bc_norm_rotate_fwd(const void *B, const void *C, const float *weight_B, const float *weight_C,
                                          const float *inv_freq, const int32_t *positions, void *B_out, void *C_out,
                                          int64_t batch, int64_t seqlen, int64_t ngroups, int64_t state_dim,
                                          int64_t rot_dim, float eps, int interleaved, int in_dtype, void *stream) {
    ssd_status st = ssd::check_sizes(batch, seqlen, ngroups, state_dim);
    if (st == SSD_OK)
        st = ssd::check_args(weight_B, weight_C, inv_freq, positions, state_dim, rot_dim, eps, interleaved, in_dtype);
    if (st != SSD_OK) return st;
    const int64_t rows = batch * seqlen * ngroups;
    if (rows == 0) return SSD_OK;
    if (!B || !C || !B_out || !C_out) return SSD_ERR_INVALID_ARG;
    if (!ssd::a16(B) || !ssd::a16(C) || !ssd::a16(B_out) || !ssd::a16(C_out)) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    (in_dtype == SSD_BF16 ? ssd::fwd_launch<__nv_bfloat16> : ssd::fwd_launch<float>)(
        B, C, weight_B, weight_C, inv_freq, positions, B_out, C_out, rows, seqlen, (int)ngroups, (int)state_dim,
        (int)rot_dim, eps, interleaved, s);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

SSD_API ssd_status ssd_bc_norm_rotate_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t ngroups,
                                                         int64_t state_dim, size_t *bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status st = ssd::check_sizes(batch, seqlen, ngroups, state_dim);
    if (st == SSD_OK) *bytes = ssd::bwd_bytes(batch * seqlen * ngroups, state_dim);
    return st;
}

SSD_API ssd_status ssd_bc_norm_rotate_bwd(const void *B, const void *C, const float *weight_B, const float *weight_C,
                                          const float *inv_freq, const int32_t *positions, const void *dB_out,
                                          const void *dC_out, void *dB, void *dC, float *dweight_B, float *dweight_C,
                                          int64_t batch, int64_t seqlen, int64_t ngroups, int64_t state_dim,
                                          int64_t rot_dim, float eps, int interleaved, int in_dtype, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    ssd_status st = ssd::check_sizes(batch, seqlen, ngroups, state_dim);
    if (st == SSD_OK)
        st = ssd::check_args(weight_B, weight_C, inv_freq, positions, state_dim, rot_dim, eps, interleaved, in_dtype);
    if (st != SSD_OK) return st;
    if (!dweight_B || !dweight_C) return SSD_ERR_INVALID_ARG;
    const int64_t rows = batch * seqlen * ngroups;
    if (rows > 0 && (!B || !C || !dB_out || !dC_out || !dB || !dC)) return SSD_ERR_INVALID_ARG;
    for (const void *p : {B, C, dB_out, dC_out, (const void *)dB, (const void *)dC, (const void *)dweight_B,
                          (const void *)dweight_C})
        if (!ssd::a16(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::bwd_bytes(rows, state_dim)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t wn = (size_t)state_dim * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (rows == 0) {
        e = cudaMemsetAsync(dweight_B, 0, wn, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dweight_C, 0, wn, s);
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    float *part = static_cast<float *>(workspace);
    const int64_t warps = ssd::bwd_warps(rows);
    (in_dtype == SSD_BF16 ? ssd::bwd_launch<__nv_bfloat16> : ssd::bwd_launch<float>)(
        B, C, weight_B, weight_C, inv_freq, positions, dB_out, dC_out, dB, dC, part, rows, seqlen, (int)ngroups,
        (int)state_dim, (int)rot_dim, eps, interleaved, s);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = ssd::column_sum(part, dweight_B, nullptr, warps, state_dim, 2 * state_dim, s);
    if (e == cudaSuccess) e = ssd::column_sum(part + state_dim, dweight_C, nullptr, warps, state_dim, 2 * state_dim, s);
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

}  // extern "C"
