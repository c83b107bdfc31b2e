// The gated linear recurrence, one decay per channel: scan, backward, step.
//   r = sigmoid(r_raw), g = sigmoid(g_raw), u = c softplus(lam) r, a = e^-u,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) g_t x_t
// Written with om = 1 - a (which keeps its relative accuracy where a is near
// 1, the long memories):  h_t = h_{t-1} + (beta g x - om h_{t-1}),
// beta = sqrt(om (2 - om)).
#include <math.h>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kGatedChunk = 64;   // tokens between chunk states
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// a = e^-u and om = 1 - a for u >= 0, each to its own relative accuracy: om
// by the Taylor series below 0.35 (its seventh-order remainder is under 2e-8
// of the value there), a by the exponential above, the other from it.
__device__ __forceinline__ void decay_of(float u, float &a, float &om) {
    float p = fmaf(u, -1.0f / 5040.0f, 1.0f / 720.0f) * -1.0f;
    p = fmaf(u, p, 1.0f / 120.0f);
    p = fmaf(u, p, -1.0f / 24.0f);
    p = fmaf(u, p, 1.0f / 6.0f);
    p = fmaf(u, p, -0.5f);
    p = fmaf(u, p, 1.0f);
    const bool near = u < 0.35f;
    const float e = exp2f(-u * kLog2e);
    om = near ? u * p : 1.0f - e;
    a = near ? 1.0f - om : e;
}

struct Gate {
    float r, g, u, a, om, q;   // om = 1 - a, q = 1 - a^2
};

__device__ __forceinline__ Gate gate_of(float r_raw, float g_raw, float k) {
    Gate t;
    t.r = sigmoid_f(r_raw);
    t.g = sigmoid_f(g_raw);
    t.u = k * t.r;
    decay_of(t.u, t.a, t.om);
    t.q = t.om * (1.0f + t.a);
    return t;
}

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---- scan: one thread per (row, channel), tokens in order
template <typename T>
__global__ void __launch_bounds__(128)
gated_scan_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                  const float *__restrict__ lam, const float *__restrict__ init, const int32_t *__restrict__ seq_idx,
                  T *__restrict__ y, float *__restrict__ fin, float *__restrict__ states, int64_t L, int64_t D,
                  int64_t ldx, int64_t ldg, float c) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (d >= D) return;
    const float k = c * softplus_f(lam[d]);
    float h = init ? init[b * D + d] : 0.0f;
    const int64_t nc = (L + kGatedChunk - 1) / kGatedChunk;
    for (int64_t t = 0; t < L; ++t) {
        const int64_t row = b * L + t;
        const Gate e = gate_of(to_f(rr[row * ldg + d]), to_f(gr[row * ldg + d]), k);
        if (seq_idx && t > 0 && seq_idx[row] != seq_idx[row - 1]) h = 0.0f;
        h += fmaf(sqrtf(e.q) * e.g, to_f(x[row * ldx + d]), -e.om * h);
        y[row * D + d] = from_f<T>(h);
        if (states && (t % kGatedChunk == kGatedChunk - 1 || t == L - 1))
            states[(b * nc + t / kGatedChunk) * D + d] = h;
    }
    if (fin) fin[b * D + d] = h;
}

// ---- backward: one thread per (row, channel), chunks from the last to the
// first; each chunk's states are recomputed from the state entering it.
//   dh_t = dy_t + a_{t+1} dh_{t+1}       (nothing across a document start)
//   dx = dh beta g,  dg_raw = dh beta x g (1 - g)
//   p = dh (u a h_{t-1} - u a^2/beta g x)      (u times d/d log a)
//   dr_raw = -(1 - r) p,  dlam = -sigmoid(lam)/softplus(lam) sum p
template <typename T>
__global__ void __launch_bounds__(128)
gated_bwd_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                 const float *__restrict__ lam, const float *__restrict__ init, const int32_t *__restrict__ seq_idx,
                 const float *__restrict__ states, const T *__restrict__ dy, const float *__restrict__ dfin,
                 T *__restrict__ dx, T *__restrict__ dr, T *__restrict__ dg, float *__restrict__ part,
                 float *__restrict__ dinit, int64_t L, int64_t D, int64_t ldx, int64_t ldg, int64_t lddg, float c) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (d >= D) return;
    const float k = c * softplus_f(lam[d]);
    const int64_t nc = (L + kGatedChunk - 1) / kGatedChunk;
    float carry = dfin ? dfin[b * D + d] : 0.0f;   // a_{t+1} dh_{t+1}
    float before[kGatedChunk];
    for (int64_t ch = nc - 1; ch >= 0; --ch) {
        const int64_t t0 = ch * kGatedChunk, t1 = t0 + kGatedChunk < L ? t0 + kGatedChunk : L;
        float h = ch > 0 ? states[(b * nc + ch - 1) * D + d] : init ? init[b * D + d] : 0.0f;
        for (int64_t t = t0; t < t1; ++t) {
            const int64_t row = b * L + t;
            const Gate e = gate_of(to_f(rr[row * ldg + d]), to_f(gr[row * ldg + d]), k);
            if (seq_idx && t > 0 && seq_idx[row] != seq_idx[row - 1]) h = 0.0f;
            before[t - t0] = h;
            h += fmaf(sqrtf(e.q) * e.g, to_f(x[row * ldx + d]), -e.om * h);
        }
        float sum = 0.0f;
        for (int64_t t = t1 - 1; t >= t0; --t) {
            const int64_t row = b * L + t;
            const Gate e = gate_of(to_f(rr[row * ldg + d]), to_f(gr[row * ldg + d]), k);
            const float xv = to_f(x[row * ldx + d]), dh = to_f(dy[row * D + d]) + carry;
            const float a = e.a, beta = sqrtf(e.q);
            const float w = e.q > 0.0f ? e.u * a * a / beta : 0.0f;
            const float p = dh * (e.u * a * before[t - t0] - w * e.g * xv);
            dx[row * D + d] = from_f<T>(dh * beta * e.g);
            dg[row * lddg + d] = from_f<T>(dh * beta * xv * e.g * (1.0f - e.g));
            dr[row * lddg + d] = from_f<T>(-(1.0f - e.r) * p);
            sum += p;
            const bool start = seq_idx && t > 0 && seq_idx[row] != seq_idx[row - 1];
            carry = start ? 0.0f : a * dh;
        }
        part[(b * nc + ch) * D + d] = sum;
    }
    if (dinit) dinit[b * D + d] = carry;
}

// ---- one token
template <typename T>
__global__ void __launch_bounds__(128)
gated_step_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                  const float *__restrict__ lam, float *__restrict__ state, T *__restrict__ y, int64_t D, int64_t ldx,
                  int64_t ldg, float c) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (d >= D) return;
    const Gate e = gate_of(to_f(rr[b * ldg + d]), to_f(gr[b * ldg + d]), c * softplus_f(lam[d]));
    float h = state[b * D + d];
    h += fmaf(sqrtf(e.q) * e.g, to_f(x[b * ldx + d]), -e.om * h);
    state[b * D + d] = h;
    y[b * D + d] = from_f<T>(h);
}

bool element_aligned(const void *p, int in_dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (in_dtype == SSD_BF16 ? 1u : 3u)) == 0;
}
bool float_aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

ssd_status check_sizes(int64_t b, int64_t L, int64_t D, int in_dtype) {
    if (b < 0 || L < 0 || D <= 0) return SSD_ERR_INVALID_ARG;
    if (in_dtype != SSD_F32 && in_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
    if (D >= (1ll << 31) || b > 65535 || L >= (1ll << 31) || b * L >= (1ll << 40)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t chunks(int64_t L) { return (L + kGatedChunk - 1) / kGatedChunk; }

size_t workspace_bytes_of(int64_t b, int64_t L, int64_t D, int backward) {
    return kStatusBytes + (backward ? align256((size_t)(b * chunks(L) * D) * sizeof(float)) : 0);
}

}  // namespace
}  // namespace ssd

extern "C" {

SSD_API ssd_status ssd_gated_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int in_dtype, int backward,
                                                 size_t *bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return SSD_ERR_INVALID_ARG;
    const ssd_status st = ssd::check_sizes(batch, seqlen, dim, in_dtype);
    if (st == SSD_OK) *bytes = ssd::workspace_bytes_of(batch, seqlen, dim, backward);
    return st;
}

SSD_API ssd_status ssd_gated_scan_fwd(const void *x, const void *r_raw, const void *g_raw, const float *lam,
                                      const float *init_state, const int32_t *seq_idx, void *y, float *final_state,
                                      float *chunk_states, int64_t batch, int64_t seqlen, int64_t dim, int64_t ld_x,
                                      int64_t ld_gate, float decay_scale, int in_dtype, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    ssd_status st = ssd::check_sizes(batch, seqlen, dim, in_dtype);
    if (st != SSD_OK) return st;
    if (ld_x < dim || ld_gate < dim || !(decay_scale > 0.0f) || isinf(decay_scale) || !lam) return SSD_ERR_INVALID_ARG;
    if (batch > 0 && seqlen > 0 && (!x || !r_raw || !g_raw || !y)) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, r_raw, g_raw, (const void *)y})
        if (!ssd::element_aligned(p, in_dtype)) return SSD_ERR_ALIGNMENT;
    for (const void *p : {(const void *)lam, (const void *)init_state, (const void *)seq_idx,
                          (const void *)final_state, (const void *)chunk_states})
        if (!ssd::float_aligned(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::workspace_bytes_of(batch, seqlen, dim, 0)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
    if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
    if (batch == 0) return SSD_OK;
    if (seqlen == 0) {
        // no tokens: the state leaves as it came in
        if (final_state) {
            const size_t n = (size_t)(batch * dim) * sizeof(float);
            e = init_state ? cudaMemcpyAsync(final_state, init_state, n, cudaMemcpyDeviceToDevice, s)
                           : cudaMemsetAsync(final_state, 0, n, s);
            if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
        }
        return SSD_OK;
    }
    {
        ssd::TraceScope tr(s, ssd::kTrGatedScan);
        const dim3 grid((unsigned)((dim + 127) / 128), (unsigned)batch);
        if (in_dtype == SSD_BF16)
            ssd::gated_scan_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(
                (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)r_raw, (const __nv_bfloat16 *)g_raw, lam, init_state,
                seq_idx, (__nv_bfloat16 *)y, final_state, chunk_states, seqlen, dim, ld_x, ld_gate, decay_scale);
        else
            ssd::gated_scan_kernel<float><<<grid, 128, 0, s>>>(
                (const float *)x, (const float *)r_raw, (const float *)g_raw, lam, init_state, seq_idx, (float *)y,
                final_state, chunk_states, seqlen, dim, ld_x, ld_gate, decay_scale);
    }
    e = cudaGetLastError();
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

SSD_API ssd_status ssd_gated_scan_bwd(const void *x, const void *r_raw, const void *g_raw, const float *lam,
                                      const float *init_state, const int32_t *seq_idx, const float *chunk_states,
                                      const void *dy, const float *dfinal_state, void *dx, void *dr_raw, void *dg_raw,
                                      float *dlam, float *dinit_state, int64_t batch, int64_t seqlen, int64_t dim,
                                      int64_t ld_x, int64_t ld_gate, int64_t ld_dgate, float decay_scale, int in_dtype,
                                      void *workspace, size_t workspace_bytes, void *stream) {
    ssd_status st = ssd::check_sizes(batch, seqlen, dim, in_dtype);
    if (st != SSD_OK) return st;
    if (ld_x < dim || ld_gate < dim || ld_dgate < dim || !(decay_scale > 0.0f) || isinf(decay_scale) || !lam || !dlam)
        return SSD_ERR_INVALID_ARG;
    const bool has_tokens = batch > 0 && seqlen > 0;
    if (has_tokens && (!x || !r_raw || !g_raw || !dy || !dx || !dr_raw || !dg_raw)) return SSD_ERR_INVALID_ARG;
    if (has_tokens && seqlen > ssd::kGatedChunk && !chunk_states) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, r_raw, g_raw, dy, (const void *)dx, (const void *)dr_raw, (const void *)dg_raw})
        if (!ssd::element_aligned(p, in_dtype)) return SSD_ERR_ALIGNMENT;
    for (const void *p : {(const void *)lam, (const void *)init_state, (const void *)seq_idx,
                          (const void *)chunk_states, (const void *)dfinal_state, (const void *)dlam,
                          (const void *)dinit_state})
        if (!ssd::float_aligned(p)) return SSD_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < ssd::workspace_bytes_of(batch, seqlen, dim, 1)) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
    if (e != cudaSuccess) return (ssd_status)ssd::record_cuda_error(e);
    if (!has_tokens) {
        // no tokens: no gradient of lam, and the seed passes to the initial state as it is
        e = cudaMemsetAsync(dlam, 0, (size_t)dim * sizeof(float), s);
        if (e == cudaSuccess && dinit_state && batch > 0) {
            const size_t n = (size_t)(batch * dim) * sizeof(float);
            e = dfinal_state ? cudaMemcpyAsync(dinit_state, dfinal_state, n, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(dinit_state, 0, n, s);
        }
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + ssd::kStatusBytes);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedBwd);
        const dim3 grid((unsigned)((dim + 127) / 128), (unsigned)batch);
        if (in_dtype == SSD_BF16)
            ssd::gated_bwd_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(
                (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)r_raw, (const __nv_bfloat16 *)g_raw, lam, init_state,
                seq_idx, chunk_states, (const __nv_bfloat16 *)dy, dfinal_state, (__nv_bfloat16 *)dx,
                (__nv_bfloat16 *)dr_raw, (__nv_bfloat16 *)dg_raw, part, dinit_state, seqlen, dim, ld_x, ld_gate,
                ld_dgate, decay_scale);
        else
            ssd::gated_bwd_kernel<float><<<grid, 128, 0, s>>>(
                (const float *)x, (const float *)r_raw, (const float *)g_raw, lam, init_state, seq_idx, chunk_states,
                (const float *)dy, dfinal_state, (float *)dx, (float *)dr_raw, (float *)dg_raw, part, dinit_state,
                seqlen, dim, ld_x, ld_gate, ld_dgate, decay_scale);
    }
    e = cudaGetLastError();
    if (e == cudaSuccess) e = ssd::column_sum(part, dlam, lam, batch * ssd::chunks(seqlen), dim, dim, s);
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

SSD_API ssd_status ssd_gated_step(const void *x, const void *r_raw, const void *g_raw, const float *lam, float *state,
                                  void *y, int64_t batch, int64_t dim, int64_t ld_x, int64_t ld_gate,
                                  float decay_scale, int in_dtype, void *stream) {
    const ssd_status st = ssd::check_sizes(batch, 1, dim, in_dtype);
    if (st != SSD_OK) return st;
    if (ld_x < dim || ld_gate < dim || !(decay_scale > 0.0f) || isinf(decay_scale)) return SSD_ERR_INVALID_ARG;
    if (batch == 0) return SSD_OK;
    if (!x || !r_raw || !g_raw || !lam || !state || !y) return SSD_ERR_INVALID_ARG;
    for (const void *p : {x, r_raw, g_raw, (const void *)y})
        if (!ssd::element_aligned(p, in_dtype)) return SSD_ERR_ALIGNMENT;
    if (!ssd::float_aligned(lam) || !ssd::float_aligned(state)) return SSD_ERR_ALIGNMENT;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedStep);
        const dim3 grid((unsigned)((dim + 127) / 128), (unsigned)batch);
        if (in_dtype == SSD_BF16)
            ssd::gated_step_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(
                (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)r_raw, (const __nv_bfloat16 *)g_raw, lam, state,
                (__nv_bfloat16 *)y, dim, ld_x, ld_gate, decay_scale);
        else
            ssd::gated_step_kernel<float><<<grid, 128, 0, s>>>((const float *)x, (const float *)r_raw,
                                                               (const float *)g_raw, lam, state, (float *)y, dim, ld_x,
                                                               ld_gate, decay_scale);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

}  // extern "C"
