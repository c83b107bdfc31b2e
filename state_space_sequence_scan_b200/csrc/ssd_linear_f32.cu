// The projections' fp32 products:  D[m, n] = sum_k A(m, k) B(n, k), then the
// epilogue of ssd_linear.h.  On the CUDA cores (the tensor cores round fp32
// operands to 10 bits), two products an instruction (packed fma).
//
// A CTA of 128 or 256 threads owns a tile of 64 x 64 or 128 x 128, a thread
// 8 x 4 or 8 x 8 of it.  16 k at a time are staged in shared memory, k-major so
// that a thread reads its row and column values as vectors; the next 16 are
// loaded to registers meanwhile.  Bound by the fma pipe: 8 x 8 values need 32
// packed fma and 4 shared loads a k.  With few tiles, k is cut in parts that
// are joined in order.
#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kLfK = 16;

using f2 = unsigned long long;
__device__ __forceinline__ f2 twice(float a) {
    f2 r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ void unpack(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct LfShape {
    int64_t M, N, K, lda, ldb;
    int per;           // k of a part
    float *part;       // [parts, M, N], or null: one part
};

// kTile rows and columns, kTN columns of a thread (8 rows)
template <int kTile, int kTN, bool kAMN, bool kBMN>
__global__ void __launch_bounds__((kTile / 8) * (kTile / kTN))
linear_f32_kernel(const float *__restrict__ A, const float *__restrict__ B, LinearEpilogue ep, LfShape s) {
    constexpr int kThreads = (kTile / 8) * (kTile / kTN), kLoads = kTile * kLfK / kThreads;
    __shared__ __align__(16) float sA[2][kLfK][kTile + 4], sB[2][kLfK][kTile + 4];
    const int tid = threadIdx.x;
    const int64_t m0 = (int64_t)blockIdx.y * kTile, n0 = (int64_t)blockIdx.x * kTile;
    const int64_t k0 = (int64_t)blockIdx.z * s.per, k1 = min(s.K, k0 + s.per);
    // a warp covers 4 x 8 threads: few distinct addresses a shared load
    const int lane = tid & 31, warp = tid >> 5;
    constexpr int kWarpsN = kTile / kTN / 8;
    const int tm = ((warp / kWarpsN) * 4 + lane / 8) * 8, tn = ((warp % kWarpsN) * 8 + lane % 8) * 4;
    f2 acc[8][kTN / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < kTN / 2; ++j) acc[i][j] = 0;
    float ra[kLoads], rb[kLoads];
    auto fetch = [&](int64_t k) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int e = tid + i * kThreads;
            const int ka = kAMN ? e / kTile : e % kLfK, ia = kAMN ? e % kTile : e / kLfK;
            const int kb = kBMN ? e / kTile : e % kLfK, ib = kBMN ? e % kTile : e / kLfK;
            ra[i] = k + ka < k1 && m0 + ia < s.M ? A[kAMN ? (k + ka) * s.lda + m0 + ia : (m0 + ia) * s.lda + k + ka] : 0.0f;
            rb[i] = k + kb < k1 && n0 + ib < s.N ? B[kBMN ? (k + kb) * s.ldb + n0 + ib : (n0 + ib) * s.ldb + k + kb] : 0.0f;
        }
    };
    auto put = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int e = tid + i * kThreads;
            sA[buf][kAMN ? e / kTile : e % kLfK][kAMN ? e % kTile : e / kLfK] = ra[i];
            sB[buf][kBMN ? e / kTile : e % kLfK][kBMN ? e % kTile : e / kLfK] = rb[i];
        }
    };
    if (k0 < k1) {
        fetch(k0);
        put(0);
        __syncthreads();
    }
    int buf = 0;
    for (int64_t k = k0; k < k1; k += kLfK, buf ^= 1) {
        const bool more = k + kLfK < k1;
        if (more) fetch(k + kLfK);
#pragma unroll
        for (int q = 0; q < kLfK; ++q) {
            const float4 a0 = *reinterpret_cast<const float4 *>(&sA[buf][q][tm]), a1 = *reinterpret_cast<const float4 *>(&sA[buf][q][tm + 4]);
            f2 b[kTN / 2];
#pragma unroll
            for (int h = 0; h < kTN / 4; ++h) {   // columns tn .. tn + 3, and those half a tile on
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&sB[buf][q][tn + h * (kTile / 2)]);
                b[2 * h] = v.x;
                b[2 * h + 1] = v.y;
            }
            const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const f2 aa = twice(a[i]);
#pragma unroll
                for (int j = 0; j < kTN / 2; ++j) acc[i][j] = fma2(aa, b[j], acc[i][j]);
            }
        }
        if (more) {
            put(buf ^ 1);
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t m = m0 + tm + i;
        if (m >= s.M) break;
#pragma unroll
        for (int j = 0; j < kTN; ++j) {
            const int64_t n = n0 + tn + (j / 4) * (kTile / 2) + j % 4, at = m * s.N + n;
            if (n >= s.N) continue;
            float lo, hi;
            unpack(acc[i][j / 2], lo, hi);
            float z = j & 1 ? hi : lo;
            if (s.part) {
                s.part[blockIdx.z * s.M * s.N + at] = z;
                continue;
            }
            if (ep.bias) z += ep.bias[n];
            if (ep.preact) static_cast<float *>(ep.preact)[at] = z;
            z = linear_act(z, ep.act);
            if (ep.residual) z += static_cast<const float *>(ep.residual)[at];
            static_cast<float *>(ep.out)[at] = z;
        }
    }
}

struct Plan {
    int tile, parts, per;
};
// By an estimate of the cycles: an SM takes a 128 x 128 tile through a k in
// 128 (16384 products at 128 a cycle) with one CTA of 8 warps, and two CTAs of 64 x 64 in
// 70 (4 warps each hide less); joining parts costs a launch and 8 bytes a value.
Plan plan_of(int64_t M, int64_t N, int64_t K) {
    Plan best = {64, 1, (int)K};
    double least = 1e300;
    for (int tile : {128, 64}) {
        const int64_t tiles = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
        for (int want = 1; want <= 16; ++want) {
            const int64_t per = ((K + want - 1) / want + kLfK - 1) / kLfK * kLfK, parts = (K + per - 1) / per;
            if (want > 1 && (parts != want || per < 64)) continue;
            const double slots = tile == 128 ? 148 : 296, cost = tile == 128 ? 150 : 75;
            const double waves = (double)((int64_t)((tiles * parts + slots - 1) / slots));
            double t = waves * ((double)per * cost + 2000);
            if (parts > 1) t += 5000 + (double)M * N * parts * 8 / 3500;
            if (t < least) {
                least = t;
                best = {tile, (int)parts, (int)per};
            }
        }
    }
    return best;
}

template <int kTile, int kTN>
void launch(const float *A, const float *B, const LinearEpilogue &ep, const LfShape &s, bool a_mn, bool b_mn, int parts, cudaStream_t st) {
    const dim3 grid((unsigned)((s.N + kTile - 1) / kTile), (unsigned)((s.M + kTile - 1) / kTile), (unsigned)parts);
    auto kern = a_mn ? linear_f32_kernel<kTile, kTN, true, true>
                : b_mn ? linear_f32_kernel<kTile, kTN, false, true> : linear_f32_kernel<kTile, kTN, false, false>;
    kern<<<grid, (kTile / 8) * (kTile / kTN), 0, st>>>(A, B, ep, s);
}

}  // namespace

size_t linear_f32_part_bytes(int64_t M, int64_t N, int64_t K) {
    const Plan p = plan_of(M, N, K);
    return p.parts > 1 ? align256((size_t)(M * N) * p.parts * sizeof(float)) : 0;
}

cudaError_t linear_f32(const float *A, int64_t lda, bool a_mn, const float *B, int64_t ldb, bool b_mn,
                       const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K, void *part, cudaStream_t st) {
    TraceScope tr(st, kTrLinear);
    const Plan p = plan_of(M, N, K);
    const LfShape s = {M, N, K, lda, ldb, p.per, p.parts > 1 ? static_cast<float *>(part) : nullptr};
    if (p.tile == 128) launch<128, 8>(A, B, ep, s, a_mn, b_mn, p.parts, st);
    else launch<64, 4>(A, B, ep, s, a_mn, b_mn, p.parts, st);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.parts > 1) e = linear_join<float, float>(s.part, ep, M, N, p.parts, st);
    return e;
}

}  // namespace ssd
