// Column sums of float partials in a fixed order: the last step of every
// parameter gradient of the operators around the scan (the gated
// recurrence's lam, the norm's weights, a projection's bias).
#include "ssd_internal.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kCsCols = 32, kCsRows = 32;

// out[c] = scale(c) * sum over rows r of part[r, c].  A block takes 32
// columns; thread (tx, ty) adds rows ty, ty + 32, ... and the 32 partial sums
// are added in ty order.  The running sums are doubles: up to millions of
// rows stand behind one gradient, and this pass reads a partial per 64 or
// more tokens only.
__global__ void __launch_bounds__(kCsCols *kCsRows)
column_sum_kernel(const float *__restrict__ part, float *__restrict__ out, const float *__restrict__ lam, int64_t rows,
                  int64_t cols, int64_t ld, float *__restrict__ out2, int64_t split) {
    __shared__ double s_sum[kCsRows][kCsCols];
    const int tx = threadIdx.x % kCsCols, ty = threadIdx.x / kCsCols;
    const int64_t c = (int64_t)blockIdx.x * kCsCols + tx;
    double acc = 0.0;
    if (c < cols) {
#pragma unroll 8
        for (int64_t r = ty; r < rows; r += kCsRows) acc += (double)part[r * ld + c];
    }
    s_sum[ty][tx] = acc;
    __syncthreads();
    if (ty == 0 && c < cols) {
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < kCsRows; ++i) t += s_sum[i][tx];
        if (lam) {
            // d(k r)/d lam relative to k r: sigmoid(lam) / softplus(lam),
            // which tends to 1 as lam -> -inf (both vanish alike)
            const double l = (double)lam[c];
            const double sp = fmax(l, 0.0) + log1p(exp(-fabs(l)));
            const double sg = l >= 0.0 ? 1.0 / (1.0 + exp(-l)) : exp(l) / (1.0 + exp(l));
            t *= sp > 0.0 ? -sg / sp : -1.0;
        }
        if (c < split) out[c] = (float)t;
        else out2[c - split] = (float)t;
    }
}

}  // namespace

cudaError_t column_sum(const float *part, float *out, const float *lam, int64_t rows, int64_t cols, int64_t ld,
                       cudaStream_t s, float *out2, int64_t split) {
    TraceScope tr(s, kTrColumnSum);
    column_sum_kernel<<<(unsigned)((cols + kCsCols - 1) / kCsCols), kCsCols * kCsRows, 0, s>>>(part, out, lam, rows,
                                                                                              cols, ld, out2, out2 ? split : cols);
    return cudaGetLastError();
}

}  // namespace ssd
