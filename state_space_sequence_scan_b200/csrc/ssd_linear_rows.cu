// The projection of few rows (decode): out = act(x W^T + bias) + residual for
// up to kLrMost bf16 rows.  Every weight is read once and used for all rows, so
// the weights' way from HBM is the bound (2 bytes a weight), then latency.
//
// A CTA takes 16 outputs; its warps share out k in chunks of 32.  The product
// is D[n, m] = sum_k W(n, k) x(m, k) by m16n8k16 matrix instructions, the
// weights as the 16-row operand: lane (g, t) of a warp loads 8 consecutive k
// of rows g and g + 8 straight to registers, 16 bytes each.  A matrix
// instruction wants other k of that lane, but the order of k is free as long
// as both operands agree, and x is loaded the same way.  No shared memory, no
// barrier until the warps' sums are joined, in warp order.  (tcgen05 would need
// its operands staged and a tile of 128 rows for the same bytes; the time here
// is the loads'.)
#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kLrOut = 16;
constexpr int kLrAhead = 4;    // chunks a warp loads before it multiplies them (fewer at once: 40 to 48 registers do not hold four)

__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 elements from p, of which `left` exist (zeros behind); kVec: elements of a
// load, by the rows' alignment.
template <int kVec> __device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p, int64_t left) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (kVec == 8) {
        if (left > 0) v = __ldg(reinterpret_cast<const uint4 *>(p));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kVec == 2) {
                w[i] = 2 * i < left ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0u;
            } else {
                const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
                const uint32_t lo = 2 * i < left ? __ldg(q + 2 * i) : 0, hi = 2 * i + 1 < left ? __ldg(q + 2 * i + 1) : 0;
                w[i] = lo | hi << 16;
            }
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// kTiles: rows of x in eights; kLrWarps: warps of the CTA
template <int kTiles, int kVec, int kLrWarps, typename TO>
__global__ void __launch_bounds__(32 * kLrWarps, kVec < 8 || kTiles > 2 ? 1 : kLrWarps == 16 ? 3 : 5)
linear_rows_kernel(const __nv_bfloat16 *__restrict__ x, const __nv_bfloat16 *__restrict__ W, LinearEpilogue ep, int M, int64_t N,
                   int K, unsigned *status) {
    __shared__ float s_sum[kLrWarps][kTiles * 8][kLrOut + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int64_t n0 = (int64_t)blockIdx.x * kLrOut;
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const __nv_bfloat16 *w0 = W + min(n0 + g, N - 1) * K + 8 * t, *w1 = W + min(n0 + g + 8, N - 1) * K + 8 * t;
    const __nv_bfloat16 *xr[kTiles];
    float acc[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        xr[i] = x + (int64_t)min(8 * i + g, M - 1) * K + 8 * t;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    }
    const int chunks = (int)(((int64_t)K + 31) / 32);
    // The matrix instructions cut a sum's low bits at every step, and a chain over
    // 32768 k would be 1e-5 off: a warp's sums are added up every 32 steps, in its
    // place in shared memory (registers for them would leave an SM fewer CTAs).
    // lane (g, t) holds outputs g (0, 1) and g + 8 (2, 3) of rows 2 t, 2 t + 1
    auto place = [&](int i, int j) -> float & { return s_sum[warp][8 * i + 2 * t + (j & 1)][g + (j >> 1) * 8]; };
    constexpr int kRounds = 4;
    int c0 = warp;
    for (bool first = true; first || c0 < chunks; first = false) {
#pragma unroll 1
        for (int n = 0; n < kRounds && c0 < chunks; ++n, c0 += kLrWarps * kLrAhead) {
            uint4 a[kLrAhead], b[kLrAhead], v[kLrAhead][kTiles];
#pragma unroll
            for (int q = 0; q < kLrAhead; ++q) {
                const int64_t k = (int64_t)(c0 + q * kLrWarps) * 32, left = K - k - 8 * t;
                a[q] = load8<kVec>(w0 + k, left);
                b[q] = load8<kVec>(w1 + k, left);
            }
#pragma unroll
            for (int q = 0; q < kLrAhead; ++q) {
                const int64_t k = (int64_t)(c0 + q * kLrWarps) * 32, left = K - k - 8 * t;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) v[q][i] = load8<kVec>(xr[i] + k, left);
            }
#pragma unroll
            for (int q = 0; q < kLrAhead; ++q)
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    mma_16x8(acc[i], a[q].x, b[q].x, a[q].y, b[q].y, v[q][i].x, v[q][i].y);
                    mma_16x8(acc[i], a[q].z, b[q].z, a[q].w, b[q].w, v[q][i].z, v[q][i].w);
                }
        }
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                place(i, j) = first ? acc[i][j] : place(i, j) + acc[i][j];
                acc[i][j] = 0.0f;
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kTiles * 8 * kLrOut; e += 32 * kLrWarps) {
        const int m = e / kLrOut;
        const int64_t n = n0 + e % kLrOut;
        if (m >= M || n >= N) continue;
        float z = s_sum[0][m][e % kLrOut];
#pragma unroll
        for (int k = 1; k < kLrWarps; ++k) z += s_sum[k][m][e % kLrOut];
        const int64_t at = m * N + n;
        if (ep.bias) z += ep.bias[n];
        if (ep.preact) static_cast<__nv_bfloat16 *>(ep.preact)[at] = __float2bfloat16_rn(z);
        z = linear_act<TO>(z, ep.act);
        if (ep.residual) z += to_f(static_cast<const TO *>(ep.residual)[at]);
        static_cast<TO *>(ep.out)[at] = linear_from_f<TO>(z);
    }
}

template <int kTiles, int kVec, int kWarps, typename TO>
void launch_as(const void *x, const void *W, const LinearEpilogue &ep, int M, int64_t N, int K, unsigned *status, cudaStream_t s) {
    linear_rows_kernel<kTiles, kVec, kWarps, TO><<<(unsigned)((N + kLrOut - 1) / kLrOut), 32 * kWarps, 0, s>>>(
        (const __nv_bfloat16 *)x, (const __nv_bfloat16 *)W, ep, M, N, K, status);
}

// 8 warps; 16 for up to 8 rows on 16 bytes where k is long enough to keep them
// loading and the outputs alone are too few CTAs, or k so long that it does not
// matter.  From a cold L2, 8 and 16 warps, 1 to 8 rows (all alike):
//   2560 x 1024  10.2, 8.3 us   2560 x 2560  14.4, 12.3   2560 x 5120  22.5, 16.4   6400 x 2560  16.4, 14.4
//   7168 x 2560  18.3, 18.5     10576 x 2560  20.5, 22.6  10576 x 5120  35, 37      10576 x 8192  53, 49
//   16384 x 5120  51, 47        5120 x 512  8.3, 8.2 to 10.2
// Rows that start elsewhere gain nothing (2560 x 5118: 18.6, 19.3; 5120 x 1026: 10.3, 12.4).
template <int kTiles, typename TO>
void launch(const void *x, const void *W, const LinearEpilogue &ep, int M, int64_t N, int K, unsigned *status, cudaStream_t s) {
    if constexpr (kTiles == 1) {
        if (K % 8 == 0 && (K >= 4096 || (K >= 1024 && N <= 6400))) return launch_as<1, 8, 16, TO>(x, W, ep, M, N, K, status, s);
    }
    if (K % 8 == 0) launch_as<kTiles, 8, 8, TO>(x, W, ep, M, N, K, status, s);
    else if (K % 2 == 0) launch_as<kTiles, 2, 8, TO>(x, W, ep, M, N, K, status, s);
    else launch_as<kTiles, 1, 8, TO>(x, W, ep, M, N, K, status, s);
}

}  // namespace

cudaError_t linear_rows(const void *x, const void *W, const LinearEpilogue &ep, int out_f32, int64_t M, int64_t N, int64_t K,
                        unsigned *status, cudaStream_t s) {
    TraceScope tr(s, kTrLinear);
    if (M <= 8) (out_f32 ? launch<1, float> : launch<1, __nv_bfloat16>)(x, W, ep, (int)M, N, (int)K, status, s);
    else if (M <= 16) (out_f32 ? launch<2, float> : launch<2, __nv_bfloat16>)(x, W, ep, (int)M, N, (int)K, status, s);
    else (out_f32 ? launch<4, float> : launch<4, __nv_bfloat16>)(x, W, ep, (int)M, N, (int)K, status, s);
    return cudaGetLastError();
}

}  // namespace ssd
