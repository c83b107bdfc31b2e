// The projections' smaller fp32 products:  D[m, n] = sum_k A(m, k) B(n, k), then
// the epilogue of ssd_linear.h.  On the CUDA cores, two products an instruction
// (packed fma); larger ones take ssd_linear_tc.cu's way in bf16 parts.
//
// A CTA of 128 threads owns a tile of 128 x 64, a thread 8 x 8 of it (fewer rows
// where M is small: 1, 2 or 4).  16 k at a time are staged in shared memory,
// k-major so that a thread reads its row and column values as vectors, by
// 4-byte asynchronous copies that turn the tile on the way and fill with zeros
// where it ends (rows of odd lengths start anywhere, so wider ones would not
// fit them); three stages are on their way, and no register holds them.  Bound
// by the fma pipe, next by shared memory: a k of 8 x 8 values is 32 packed fma
// (64 cycles a warp) and 4 loads of 2 to 4 cycles each; with 8 x 4 a thread the
// loads took 59% of the cycles and the fma 41%.
// With few tiles, k is cut in parts, one CTA of a cluster each; they add their
// sums up in order through one another's shared memory and share the
// epilogue, so it stays one launch.
#include "ssd_f2.cuh"
#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kLfK = 16, kLfCols = 64, kLfThreads = 128, kLfStages = 3;
constexpr int kLfPitchB = kLfCols + 4;       // floats of a staged k of B, and of a row of sums

__device__ __forceinline__ void copy4(uint32_t to, const float *from, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
struct LfShape {
    int64_t M, N, K, lda, ldb;
    int per, parts;    // k of a part; parts: CTAs of a cluster
    unsigned nt;       // tiles of columns
};

__device__ __forceinline__ void finish_one(float z, int64_t m, int64_t n, const LinearEpilogue &ep, const LfShape &s) {
    const int64_t at = m * s.N + n;
    if (ep.bias) z += ep.bias[n];
    if (ep.preact) static_cast<float *>(ep.preact)[at] = z;
    z = linear_act<float>(z, ep.act);
    if (ep.residual) z += static_cast<const float *>(ep.residual)[at];
    static_cast<float *>(ep.out)[at] = z;
}

// kRows: rows of a thread
template <int kRows, bool kAMN, bool kBMN>
__global__ void __launch_bounds__(kLfThreads, 4)
linear_f32_kernel(const float *__restrict__ A, const float *__restrict__ B, LinearEpilogue ep, LfShape s, unsigned *status) {
    constexpr int kTile = 16 * kRows, kPitchA = kTile + 4;
    constexpr int kBufA = kLfK * kPitchA, kBufB = kLfK * kLfPitchB;
    constexpr int kFloats = kLfStages * (kBufA + kBufB), kSums = kTile * kLfPitchB;
    __shared__ __align__(16) float smem[kFloats > kSums ? kFloats : kSums];   // stages of A, then of B; at the end a part's sums
    const int tid = threadIdx.x;
    if (status && blockIdx.x == 0 && blockIdx.z == 0 && tid == 0) *status = 0;
    const unsigned mi = blockIdx.x / s.nt;   // (rows may be more than a grid's second axis takes)
    const int64_t m0 = (int64_t)mi * kTile, n0 = (int64_t)(blockIdx.x - mi * s.nt) * kLfCols;
    const int64_t k0 = (int64_t)blockIdx.z * s.per, k1 = min(s.K, k0 + s.per);
    // a warp covers 4 x 8 threads: rows tm .. tm + kRows - 1, columns tn .. tn + 3 and those 32 on
    const int lane = tid & 31, warp = tid >> 5;
    const int tm = (warp * 4 + lane / 8) * kRows, tn = lane % 8 * 4;
    f2 acc[kRows][4];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0;
    // thread's element i of a staged tile: e = tid + 128 i, row e % rows and k e / rows
    // where m (n) is contiguous, else row e / 16 and k e % 16
    const int ra = kAMN ? tid % kTile : tid / kLfK, ka = kAMN ? tid / kTile : tid % kLfK;
    const int rb = kBMN ? tid % kLfCols : tid / kLfK, kb = kBMN ? tid / kLfCols : tid % kLfK;
    constexpr int kStepA = kLfThreads / (kAMN ? kTile : kLfK), kStepB = kLfThreads / (kBMN ? kLfCols : kLfK);
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const uint32_t toA = base + (ka * kPitchA + ra) * 4, toB = base + (kLfStages * kBufA + kb * kLfPitchB + rb) * 4;
    constexpr uint32_t kNextA = (kAMN ? kStepA * kPitchA : kStepA) * 4, kNextB = (kBMN ? kStepB * kLfPitchB : kStepB) * 4;
    constexpr int kLoadsA = kTile * kLfK / kLfThreads, kLoadsB = kLfCols * kLfK / kLfThreads;
    // the common step needs no test: the tile's rows and columns are all there, and 16 k are left
    const bool inner = m0 + kTile <= s.M && n0 + kLfCols <= s.N;
    auto fetch = [&](int64_t k, int st) {
        if (k < k1) {
            const float *pa = A + (kAMN ? (k + ka) * s.lda + m0 + ra : (m0 + ra) * s.lda + k + ka);
            const float *pb = B + (kBMN ? (k + kb) * s.ldb + n0 + rb : (n0 + rb) * s.ldb + k + kb);
            const uint32_t da = toA + st * (kBufA * 4), db = toB + st * (kBufB * 4);
            if (inner && k + kLfK <= k1) {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i) copy4(da + i * kNextA, pa + (int64_t)(i * kStepA) * s.lda, true);
#pragma unroll
                for (int i = 0; i < kLoadsB; ++i) copy4(db + i * kNextB, pb + (int64_t)(i * kStepB) * s.ldb, true);
            } else {
#pragma unroll
                for (int i = 0; i < kLoadsA; ++i) {
                    const bool a = k + ka + (kAMN ? i * kStepA : 0) < k1 && m0 + ra + (kAMN ? 0 : i * kStepA) < s.M;
                    copy4(da + i * kNextA, a ? pa + (int64_t)(i * kStepA) * s.lda : A, a);
                }
#pragma unroll
                for (int i = 0; i < kLoadsB; ++i) {
                    const bool b = k + kb + (kBMN ? i * kStepB : 0) < k1 && n0 + rb + (kBMN ? 0 : i * kStepB) < s.N;
                    copy4(db + i * kNextB, b ? pb + (int64_t)(i * kStepB) * s.ldb : B, b);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kLfStages - 1; ++i) fetch(k0 + i * kLfK, i);
    int st = 0;
    for (int64_t k = k0; k < k1; k += kLfK) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLfStages - 2) : "memory");
        __syncthreads();   // this stage has landed for all, and the one before has been read by all
        fetch(k + (kLfStages - 1) * kLfK, st == 0 ? kLfStages - 1 : st - 1);
        const float *pa = smem + st * kBufA + tm, *pb = smem + kLfStages * kBufA + st * kBufB + tn;
#pragma unroll
        for (int q = 0; q < kLfK; ++q) {
            float a[kRows];
            if constexpr (kRows >= 4) {
#pragma unroll
                for (int i = 0; i < kRows; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(pa + q * kPitchA + i);
                    a[i] = v.x; a[i + 1] = v.y; a[i + 2] = v.z; a[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kRows; ++i) a[i] = pa[q * kPitchA + i];
            }
            const ulonglong2 b0 = *reinterpret_cast<const ulonglong2 *>(pb + q * kLfPitchB);
            const ulonglong2 b1 = *reinterpret_cast<const ulonglong2 *>(pb + q * kLfPitchB + 32);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const f2 aa = two(a[i]);
                acc[i][0] = fma(aa, b0.x, acc[i][0]);
                acc[i][1] = fma(aa, b0.y, acc[i][1]);
                acc[i][2] = fma(aa, b1.x, acc[i][2]);
                acc[i][3] = fma(aa, b1.y, acc[i][3]);
            }
        }
        st = st == kLfStages - 1 ? 0 : st + 1;
    }
    if (s.parts == 1) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t m = m0 + tm + i;
            if (m >= s.M) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t n = n0 + tn + (j / 4) * 32 + j % 4;
                if (n < s.N) finish_one(j & 1 ? hi(acc[i][j / 2]) : lo(acc[i][j / 2]), m, n, ep, s);
            }
        }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        *reinterpret_cast<ulonglong2 *>(smem + (tm + i) * kLfPitchB + tn) = make_ulonglong2(acc[i][0], acc[i][1]);
        *reinterpret_cast<ulonglong2 *>(smem + (tm + i) * kLfPitchB + tn + 32) = make_ulonglong2(acc[i][2], acc[i][3]);
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    // each CTA finishes its share of the rows
    const int rows = (kTile + s.parts - 1) / s.parts, r0 = blockIdx.z * rows, r1 = min(r0 + rows, kTile);
    for (int e = r0 * kLfCols + tid; e < r1 * kLfCols; e += kLfThreads) {
        const int r = e / kLfCols, c = e % kLfCols;
        if (m0 + r >= s.M || n0 + c >= s.N) continue;
        float z = 0.0f;
#pragma unroll 4
        for (int p = 0; p < s.parts; ++p) {
            uint32_t at;
            float v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + (r * kLfPitchB + c) * 4), "r"(p));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            z += v;
        }
        finish_one(z, m0 + r, n0 + c, ep, s);
    }
    // nobody leaves while its sums are read
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

struct Plan {
    int rows, parts, per;
};
// Rows of a thread and parts of k by an estimate of the cycles: a k of a tile
// takes an SM `busy` cycles, and `alone` where a CTA has the SM to itself (as measured);
// four CTAs share an SM.  Parts are powers of two: clusters of other sizes
// leave SMs empty (333 x 1001 x 771 in 4, 6 and 8 parts: 28, 33 and 31 us).
Plan plan_of(int64_t M, int64_t N, int64_t K, double *cycles = nullptr) {
    const int64_t sms = 148, most = 4;
    Plan best = {8, 1, (int)K};
    double least = 1e300;
    for (int rows : {8, 4, 2, 1}) {
        if (rows < 4 && M > 16 * rows) continue;
        const int64_t tiles = ((M + 16 * rows - 1) / (16 * rows)) * ((N + kLfCols - 1) / kLfCols);
        const double busy = rows == 8 ? 117 : rows == 4 ? 70 : rows == 2 ? 58 : 52;
        const double alone = rows == 8 ? 127 : rows == 4 ? 95 : rows == 2 ? 75 : 65;
        for (int want : {1, 2, 4, 8}) {
            const int64_t per = ((K + want - 1) / want + kLfK - 1) / kLfK * kLfK, parts = (K + per - 1) / per;
            if (want > 1 && (parts != want || per < 2 * kLfK)) continue;
            const int64_t ctas = tiles * parts, full = ctas / (sms * most), rest = ctas - full * sms * most;
            const double last = (double)((rest + sms - 1) / sms) * busy;   // cycles a k of the last wave
            double t = (double)full * ((double)per * most * busy + 3000);
            if (rest) t += (double)per * (last > alone ? last : alone) + 3000;
            if (parts > 1) t += 2500;
            if (t < least) {
                least = t;
                best = {rows, (int)parts, (int)(per < K ? per : K)};
            }
        }
    }
    if (cycles) *cycles = least;
    return best;
}

template <int kRows>
cudaError_t launch(const float *A, const float *B, const LinearEpilogue &ep, const LfShape &s, bool a_mn, bool b_mn, unsigned *status,
                   cudaStream_t st) {
    auto kern = a_mn ? linear_f32_kernel<kRows, true, true>
                : b_mn ? linear_f32_kernel<kRows, false, true> : linear_f32_kernel<kRows, false, false>;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(s.nt * (unsigned)((s.M + 16 * kRows - 1) / (16 * kRows)), 1, (unsigned)s.parts);
    c.blockDim = dim3(kLfThreads);
    c.stream = st;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = (unsigned)s.parts;
    c.attrs = &cluster;
    c.numAttrs = s.parts > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&c, kern, A, B, ep, s, status);
}

}  // namespace

double linear_f32_cycles(int64_t M, int64_t N, int64_t K) {
    double cycles = 0;
    plan_of(M, N, K, &cycles);
    return cycles;
}

cudaError_t linear_f32(const float *A, int64_t lda, bool a_mn, const float *B, int64_t ldb, bool b_mn,
                       const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K, unsigned *status, cudaStream_t st) {
    TraceScope tr(st, kTrLinear);
    const Plan p = plan_of(M, N, K);
    const LfShape s = {M, N, K, lda, ldb, p.per, p.parts, (unsigned)((N + kLfCols - 1) / kLfCols)};
    return (p.rows == 8 ? launch<8> : p.rows == 4 ? launch<4> : p.rows == 2 ? launch<2> : launch<1>)(A, B, ep, s, a_mn, b_mn, status, st);
}

}  // namespace ssd
