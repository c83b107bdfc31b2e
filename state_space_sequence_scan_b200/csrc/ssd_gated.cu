// The gated linear recurrence, one decay per channel: scan, backward, step.
//   r = sigmoid(r_raw), g = sigmoid(g_raw), u = c softplus(lam) r, a = e^-u,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) g_t x_t
// Written with om = 1 - a (which keeps its relative accuracy where a is near
// 1, the long memories):  h_t = h_{t-1} + (beta g x - om h_{t-1}),
// beta = sqrt(om (1 + a)).
//
// One pass over the data.  A CTA takes a chunk of tokens by 64 channels; a
// warp 8 consecutive tokens, a lane two channels.  A warp keeps (1 - a, beta
// g x) of its tokens in registers and folds them into a segment (A, H): the
// state after it is A h + H.  Segments join in a fixed order, inside the CTA
// through shared memory and across chunks through the workspace (Segment and
// look_back below), and then the kept tokens are run once more from their true
// state.  So x and the gates are read once and y is written once, where a
// first pass over the chunks' totals would read the inputs twice; and the
// order of every sum is fixed by the sizes alone, whichever CTA runs first.
//
// What bounds it: HBM (8 bytes an element of bf16 forward, 14 backward), next
// to the special function units (two sigmoids, an exponential, a root).
#include <math.h>

#include <initializer_list>
#include <type_traits>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_internal.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kGatedChunk = 64;   // tokens between chunk states
constexpr int kSegTokens = 8;     // tokens of a warp
constexpr int kTileCh = 64;       // channels of a CTA: two a lane
constexpr int kFwdWarps = 16, kBwdWarps = 8;
constexpr int kFwdChunk = kFwdWarps * kSegTokens, kBwdChunk = kBwdWarps * kSegTokens;
constexpr int kGroup = 16;        // chunks a look-back joins before it needs the state of the group before
constexpr long long kBudget = 1ll << 32;   // clock cycles before a wait gives up (~2 s)
static_assert(kBwdChunk == kGatedChunk && kFwdChunk % kGatedChunk == 0, "chunk states at chunk ends");
constexpr float kLog2e = 1.4426950408889634f;

// The special functions as the hardware has them, numbers below float32's
// normal range taken as 0: the library forms rescale around that range, which
// more than doubled this file's instructions (123 an element of the scan,
// against 50) and moves nothing here.  Each is within 2 roundings of a float32.
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / sqrt(q); at q = 0, where the factor it multiplies is 0, a finite number
__device__ __forceinline__ float over_root(float q) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q + 1e-37f));
    return r;
}
__device__ __forceinline__ float root(float q) { return q * over_root(q); }

__device__ __forceinline__ float sigmoid_f(float v) { return rcp(1.0f + ex2(v * -kLog2e)); }

// 1 - a = 1 - e^-u for u >= 0 and a, each to its own relative accuracy: the
// Taylor series below kNear (its seventh-order remainder is under 2e-8 of the
// value there), the exponential above.  kAllNear: the caller knows that u is
// below, and saves the exponential and the choice.
constexpr float kNear = 0.35f;
template <bool kAllNear> __device__ __forceinline__ float loss_of(float u) {
    float p = fmaf(u, 1.0f / 5040.0f, -1.0f / 720.0f);
    p = fmaf(u, p, 1.0f / 120.0f);
    p = fmaf(u, p, -1.0f / 24.0f);
    p = fmaf(u, p, 1.0f / 6.0f);
    p = fmaf(u, p, -0.5f);
    p = fmaf(u, p, 1.0f);
    if (kAllNear) return u * p;
    return u < kNear ? u * p : 1.0f - ex2(u * -kLog2e);
}
template <bool kAllNear> __device__ __forceinline__ float decay_of(float om, float u) {
    if (kAllNear) return 1.0f - om;
    return u < kNear ? 1.0f - om : ex2(u * -kLog2e);
}
// 1 - a^2
__device__ __forceinline__ float input_square(float om) { return om * (2.0f - om); }

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }


// ---- segments of two channels: the state after one is a h + h0 (a < 0: a
// document starts inside, nothing of the state before it reaches the end)
struct Segment {
    float a[2], h[2];
};

// `first`, then `s`
__device__ __forceinline__ Segment joined(const Segment &first, const Segment &s) {
    Segment r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r.h[i] = s.a[i] < 0.0f ? s.h[i] : fmaf(s.a[i], first.h[i], s.h[i]);
        r.a[i] = s.a[i] < 0.0f || first.a[i] < 0.0f ? -1.0f : first.a[i] * s.a[i];
    }
    return r;
}
__device__ __forceinline__ void apply(const Segment &s, float (&h)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) h[i] = s.a[i] < 0.0f ? s.h[i] : fmaf(s.a[i], h[i], s.h[i]);
}
__device__ __forceinline__ Segment segment_of(float4 v) { return Segment{{v.x, v.z}, {v.y, v.w}}; }
__device__ __forceinline__ float4 packed(const Segment &s) { return make_float4(s.a[0], s.h[0], s.a[1], s.h[1]); }

__device__ __forceinline__ unsigned load_acquire(const unsigned *p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(unsigned *p, unsigned v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// What the chunks of a row and channel tile hand on, in the workspace.  The
// words up to the segments are zero when the kernel starts.
struct Handoff {
    unsigned *status, *ticket;
    unsigned *seg_ready;      // [b, chunks, tiles]
    unsigned *state_ready;    // [b, groups, tiles]
    float4 *seg;              // [b, chunks, tiles, 32]: a chunk's segment, two channels a lane
    float2 *state;            // [b, groups, tiles, 32]: the state after a group's last chunk
    int chunks, groups, tiles;
};

// Publishes the chunk's segment, waits for what stands before it and returns
// the state entering chunk c (0 is the first in scan order).  One warp.  The
// chunks of a group are joined one by one on the state that the last chunk of
// the group before has published: a chain of chunks / 16 hops, and the same
// sums in the same order on every run.  A CTA waits only for tickets below
// its own, so for CTAs that run already.
__device__ __forceinline__ void look_back(const Handoff &w, int64_t b, int c, int tile, int lane, const Segment &mine,
                                          float (&h)[2]) {
    const int64_t at = (b * w.chunks + c) * w.tiles + tile;
    const int group = c / kGroup, pos = c % kGroup;
    if (c + 1 < w.chunks && pos + 1 < kGroup) {
        __stcg(&w.seg[at * 32 + lane], packed(mine));
        __threadfence();
        __syncwarp();
        if (lane == 0) store_release(&w.seg_ready[at], 1u);
    }
    if (c > 0) {
        const unsigned *flag = nullptr;
        if (lane < pos) flag = &w.seg_ready[at - (int64_t)(pos - lane) * w.tiles];
        else if (lane == 31 && group > 0) flag = &w.state_ready[(b * w.groups + group - 1) * w.tiles + tile];
        const long long t0 = clock64();
        bool ready = flag == nullptr;
        while (!__all_sync(0xffffffffu, ready)) {
            if (!ready) ready = load_acquire(flag) != 0u;
            if (!ready && clock64() - t0 > kBudget) {
                atomicOr(w.status, kStatusTimeout);
                ready = true;
            }
        }
        __syncwarp();
        if (group > 0) {
            const float2 v = __ldcg(&w.state[((b * w.groups + group - 1) * w.tiles + tile) * 32 + lane]);
            h[0] = v.x;
            h[1] = v.y;
        }
        const float4 *from = &w.seg[(at - (int64_t)pos * w.tiles) * 32 + lane];
#pragma unroll 4
        for (int j = 0; j < pos; ++j) apply(segment_of(__ldcg(from + (int64_t)j * w.tiles * 32)), h);
    }
    if (c + 1 < w.chunks && pos + 1 == kGroup) {
        float e[2] = {h[0], h[1]};
        apply(mine, e);
        const int64_t g = (b * w.groups + group) * w.tiles + tile;
        __stcg(&w.state[g * 32 + lane], make_float2(e[0], e[1]));
        __threadfence();
        __syncwarp();
        if (lane == 0) store_release(&w.state_ready[g], 1u);
    }
}

// ---- two channels of a token: adjacent ones where rows start on pairs of
// elements (kPair: one load), else 32 apart
template <typename T, bool kPair> struct Two;
template <> struct Two<__nv_bfloat16, true> {
    uint32_t v = 0;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool, bool in1) {
        if (in1) v = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(i ? v & 0xFFFF0000u : v << 16); }
};
template <> struct Two<float, true> {
    float2 v = {0.0f, 0.0f};
    __device__ __forceinline__ void load(const float *p, bool, bool in1) {
        if (in1) v = __ldg(reinterpret_cast<const float2 *>(p));
    }
    __device__ __forceinline__ float at(int i) const { return i ? v.y : v.x; }
};
template <typename T> struct Two<T, false> {
    T v[2] = {T(0.0f), T(0.0f)};
    __device__ __forceinline__ void load(const T *p, bool in0, bool in1) {
        if (in0) v[0] = p[0];
        if (in1) v[1] = p[32];
    }
    __device__ __forceinline__ float at(int i) const { return to_f(v[i]); }
};
template <typename T, bool kPair>
__device__ __forceinline__ void store_two(T *p, float a, float b, bool in0, bool in1) {
    if constexpr (kPair) {
        if (!in1) return;
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
            *reinterpret_cast<__nv_bfloat162 *>(p) = v;
        } else {
            *reinterpret_cast<float2 *>(p) = make_float2(a, b);
        }
    } else {
        if (in0) p[0] = from_f<T>(a);
        if (in1) p[32] = from_f<T>(b);
    }
}

struct ScanShape {
    int64_t L, D, ldx, ldg, lddg;
    float c;
    int rows, tiles;      // batch, channel tiles
};

// Which (chunk in scan order, row, tile) a CTA takes.  All rows and tiles of
// a chunk come before the next chunk's, by ticket: a CTA that waits waits for
// CTAs that started before it.
__device__ __forceinline__ void place_of(const Handoff &w, const ScanShape &s, int &c, int64_t &b, int &tile, unsigned *slot) {
    unsigned n = blockIdx.x;
    if (w.chunks > 1) {
        if (threadIdx.x == 0) *slot = atomicAdd(w.ticket, 1u);
        __syncthreads();
        n = *slot;
    }
    const unsigned plane = (unsigned)s.rows * (unsigned)s.tiles;
    c = (int)(n / plane);
    const unsigned r = n - (unsigned)c * plane;
    b = r / (unsigned)s.tiles;
    tile = (int)(r - (unsigned)b * (unsigned)s.tiles);
}

// The starts of documents among tokens t0 .. t0 + 7, as bits (token 0 of a row starts none).
__device__ __forceinline__ unsigned starts_of(const int32_t *ids, int64_t row0, int64_t t0, int64_t L, int lane) {
    bool start = false;
    if (ids && lane < kSegTokens && t0 + lane > 0 && t0 + lane < L)
        start = ids[row0 + t0 + lane] != ids[row0 + t0 + lane - 1];
    return __ballot_sync(0xffffffffu, start);
}

template <typename T, bool kPair>
__global__ void __launch_bounds__(32 * kFwdWarps, sizeof(T) == 2 ? 2 : 1)
gated_scan_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                  const float *__restrict__ lam, const float *__restrict__ init, const int32_t *__restrict__ ids,
                  T *__restrict__ y, float *__restrict__ fin, float *__restrict__ states, ScanShape s, Handoff w) {
    __shared__ float4 s_seg[kFwdWarps][32];
    __shared__ float2 s_in[32];
    __shared__ unsigned s_slot;
    int c, tile;
    int64_t b;
    place_of(w, s, c, b, tile, &s_slot);
    if (w.chunks == 1 && blockIdx.x == 0 && threadIdx.x == 0) *w.status = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t d0 = (int64_t)tile * kTileCh + (kPair ? 2 * lane : lane), d1 = d0 + (kPair ? 1 : 32);
    const bool in0 = d0 < s.D, in1 = d1 < s.D;
    const int64_t t0 = (int64_t)c * kFwdChunk + warp * kSegTokens, row0 = b * s.L;
    const int n = (int)(s.L - t0 < kSegTokens ? (s.L - t0 > 0 ? s.L - t0 : 0) : kSegTokens);
    const bool whole = n == kSegTokens;

    Two<T, kPair> vx[kSegTokens], vr[kSegTokens], vg[kSegTokens];
    {
        const T *pr = rr + (row0 + t0) * s.ldg + d0, *pg = gr + (row0 + t0) * s.ldg + d0, *px = x + (row0 + t0) * s.ldx + d0;
#pragma unroll
        for (int t = 0; t < kSegTokens; ++t)
            if (whole || t < n) {
                vr[t].load(pr + t * s.ldg, in0, in1);
                vg[t].load(pg + t * s.ldg, in0, in1);
                vx[t].load(px + t * s.ldx, in0, in1);
            }
    }
    const float k[2] = {in0 ? s.c * softplus_f(lam[d0]) : 0.0f, in1 ? s.c * softplus_f(lam[d1]) : 0.0f};
    const unsigned starts = starts_of(ids, row0, t0, s.L, lane);

    // (1 - a, beta g x) of each token, and the segment they make
    float om[kSegTokens][2], in[kSegTokens][2], sum[2] = {0.0f, 0.0f}, most = 0.0f;
    Segment seg = {{1.0f, 1.0f}, {0.0f, 0.0f}};
#pragma unroll
    for (int t = 0; t < kSegTokens; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            om[t][i] = k[i] * sigmoid_f(vr[t].at(i));   // u
            in[t][i] = sigmoid_f(vg[t].at(i)) * vx[t].at(i);
            most = fmaxf(most, om[t][i]);
        }
    // the common warp: all of its tokens there, none starting a document, every u near
    const bool easy = whole && starts == 0 && __all_sync(0xffffffffu, most < kNear);
    auto fold = [&](auto is_easy) {
        constexpr bool kEasy = decltype(is_easy)::value;
#pragma unroll
        for (int t = 0; t < kSegTokens; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool there = kEasy || t < n;
                if (there) sum[i] += om[t][i];
                const float o = loss_of<kEasy>(om[t][i]);
                om[t][i] = there ? o : 0.0f;
                in[t][i] = there ? root(input_square(o)) * in[t][i] : 0.0f;
                if (!kEasy && (starts >> t & 1)) seg.h[i] = 0.0f;
                seg.h[i] += fmaf(-om[t][i], seg.h[i], in[t][i]);
            }
    };
    if (easy) fold(std::true_type{});
    else fold(std::false_type{});
#pragma unroll
    for (int i = 0; i < 2; ++i) seg.a[i] = starts ? -1.0f : ex2(-sum[i] * kLog2e);
    s_seg[warp][lane] = packed(seg);
    __syncthreads();

    // the segments before this warp's, in order; warp 0 hands the chunk on
    Segment before = {{1.0f, 1.0f}, {0.0f, 0.0f}};
    if (warp == 0) {
        Segment all = segment_of(s_seg[0][lane]);
#pragma unroll
        for (int j = 1; j < kFwdWarps; ++j) all = joined(all, segment_of(s_seg[j][lane]));
        float h[2] = {0.0f, 0.0f};
        if (init && c < kGroup) {
            if (in0) h[0] = init[b * s.D + d0];
            if (in1) h[1] = init[b * s.D + d1];
        }
        if (w.chunks > 1) look_back(w, b, c, tile, lane, all, h);
        s_in[lane] = make_float2(h[0], h[1]);
    } else {
        for (int j = 0; j < warp; ++j) before = joined(before, segment_of(s_seg[j][lane]));
    }
    __syncthreads();
    float h[2] = {s_in[lane].x, s_in[lane].y};
    if (warp > 0) apply(before, h);

    {
        T *py = y + (row0 + t0) * s.D + d0;
        if (whole && starts == 0) {
#pragma unroll
            for (int t = 0; t < kSegTokens; ++t) {
#pragma unroll
                for (int i = 0; i < 2; ++i) h[i] += fmaf(-om[t][i], h[i], in[t][i]);
                store_two<T, kPair>(py + t * s.D, h[0], h[1], in0, in1);
            }
        } else {
#pragma unroll
            for (int t = 0; t < kSegTokens; ++t)
                if (t < n) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (starts >> t & 1) h[i] = 0.0f;
                        h[i] += fmaf(-om[t][i], h[i], in[t][i]);
                    }
                    store_two<T, kPair>(py + t * s.D, h[0], h[1], in0, in1);
                }
        }
    }
    if (n > 0) {
        const int64_t end = t0 + n;   // one past this warp's last token
        if (states && (end % kGatedChunk == 0 || end == s.L)) {
            float *o = states + (b * ((s.L + kGatedChunk - 1) / kGatedChunk) + (end - 1) / kGatedChunk) * s.D;
            if (in0) o[d0] = h[0];
            if (in1) o[d1] = h[1];
        }
        if (fin && end == s.L) {
            if (in0) fin[b * s.D + d0] = h[0];
            if (in1) fin[b * s.D + d1] = h[1];
        }
    }
}

// ---- backward: chunks of 64 tokens from the last to the first.  The states
// inside a chunk come from the one entering it (the forward's chunk states);
// the gradient's recurrence runs the other way over the same decays:
//   dh_t = dy_t + c_{t+1},   c_t = a_t dh_t (nothing past a document start)
//   dx = dh beta g,  dg_raw = dh beta x g (1 - g)
//   p = dh (u a h_{t-1} - u a^2/beta g x)      (u times d/d log a)
//   dr_raw = -(1 - r) p,  dlam = -sigmoid(lam)/softplus(lam) sum p
// (u/beta stays finite where the gate shuts and beta goes to 0.)
template <typename T, bool kPair>
__global__ void __launch_bounds__(32 * kBwdWarps, sizeof(T) == 2 ? 2 : 1)
gated_bwd_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                 const float *__restrict__ lam, const float *__restrict__ init, const int32_t *__restrict__ ids,
                 const float *__restrict__ states, const T *__restrict__ dy, const float *__restrict__ dfin,
                 T *__restrict__ dx, T *__restrict__ dr, T *__restrict__ dg, float *__restrict__ part,
                 float *__restrict__ dinit, ScanShape s, Handoff w) {
    __shared__ float4 s_fwd[kBwdWarps][32], s_rev[kBwdWarps][32];
    __shared__ float2 s_in[32], s_sum[kBwdWarps][32];
    __shared__ unsigned s_slot;
    int back, tile;
    int64_t b;
    place_of(w, s, back, b, tile, &s_slot);
    if (w.chunks == 1 && blockIdx.x == 0 && threadIdx.x == 0) *w.status = 0;
    const int c = w.chunks - 1 - back;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t d0 = (int64_t)tile * kTileCh + (kPair ? 2 * lane : lane), d1 = d0 + (kPair ? 1 : 32);
    const bool in0 = d0 < s.D, in1 = d1 < s.D;
    const int64_t t0 = (int64_t)c * kBwdChunk + warp * kSegTokens, row0 = b * s.L;
    const int n = (int)(s.L - t0 < kSegTokens ? (s.L - t0 > 0 ? s.L - t0 : 0) : kSegTokens);

    const bool whole = n == kSegTokens;
    Two<T, kPair> vx[kSegTokens], vr[kSegTokens], vg[kSegTokens], vy[kSegTokens];
    {
        const T *pr = rr + (row0 + t0) * s.ldg + d0, *pg = gr + (row0 + t0) * s.ldg + d0;
        const T *px = x + (row0 + t0) * s.ldx + d0, *py = dy + (row0 + t0) * s.D + d0;
#pragma unroll
        for (int t = 0; t < kSegTokens; ++t)
            if (whole || t < n) {
                vr[t].load(pr + t * s.ldg, in0, in1);
                vg[t].load(pg + t * s.ldg, in0, in1);
                vx[t].load(px + t * s.ldx, in0, in1);
                vy[t].load(py + t * s.D, in0, in1);
            }
    }
    const float k[2] = {in0 ? s.c * softplus_f(lam[d0]) : 0.0f, in1 ? s.c * softplus_f(lam[d1]) : 0.0f};
    const unsigned starts = starts_of(ids, row0, t0, s.L, lane);
    float h[2] = {0.0f, 0.0f};
    {
        const float *from = c > 0 ? states + (b * w.chunks + c - 1) * s.D : init ? init + b * s.D : nullptr;
        if (from && in0) h[0] = from[d0];
        if (from && in1) h[1] = from[d1];
    }

    float om[kSegTokens][2], r[kSegTokens][2], g[kSegTokens][2], sum[2] = {0.0f, 0.0f}, most = 0.0f;
    Segment seg = {{1.0f, 1.0f}, {0.0f, 0.0f}};
    Segment rev = {{1.0f, 1.0f}, {0.0f, 0.0f}};   // the same products, from the last token to the first
#pragma unroll
    for (int t = 0; t < kSegTokens; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            r[t][i] = sigmoid_f(vr[t].at(i));
            g[t][i] = sigmoid_f(vg[t].at(i));
            most = fmaxf(most, k[i] * r[t][i]);
        }
    // the common warp: all of its tokens there, none starting a document, every u near
    const bool easy = whole && starts == 0 && __all_sync(0xffffffffu, most < kNear);
    auto fold = [&](auto is_easy) {
        constexpr bool kEasy = decltype(is_easy)::value;
#pragma unroll
        for (int t = 0; t < kSegTokens; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (kEasy || t < n) {
                    const float u = k[i] * r[t][i];
                    sum[i] += u;
                    om[t][i] = loss_of<kEasy>(u);
                    if (!kEasy && (starts >> t & 1)) seg.h[i] = 0.0f;
                    seg.h[i] += fmaf(root(input_square(om[t][i])), g[t][i] * vx[t].at(i), -om[t][i] * seg.h[i]);
                }
#pragma unroll
        for (int t = kSegTokens - 1; t >= 0; --t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (kEasy || t < n) {
                    const float dh = vy[t].at(i) + rev.h[i];
                    rev.h[i] = !kEasy && (starts >> t & 1) ? 0.0f : decay_of<kEasy>(om[t][i], k[i] * r[t][i]) * dh;
                }
    };
    if (easy) fold(std::true_type{});
    else fold(std::false_type{});
#pragma unroll
    for (int i = 0; i < 2; ++i) seg.a[i] = rev.a[i] = starts ? -1.0f : ex2(-sum[i] * kLog2e);
    s_fwd[warp][lane] = packed(seg);
    s_rev[warp][lane] = packed(rev);
    __syncthreads();

    Segment after = {{1.0f, 1.0f}, {0.0f, 0.0f}};
    for (int j = 0; j < warp; ++j) apply(segment_of(s_fwd[j][lane]), h);
    if (warp == 0) {
        Segment all = segment_of(s_rev[kBwdWarps - 1][lane]);
#pragma unroll
        for (int j = kBwdWarps - 2; j >= 0; --j) all = joined(all, segment_of(s_rev[j][lane]));
        float e[2] = {0.0f, 0.0f};
        if (dfin && back < kGroup) {
            if (in0) e[0] = dfin[b * s.D + d0];
            if (in1) e[1] = dfin[b * s.D + d1];
        }
        if (w.chunks > 1) look_back(w, b, back, tile, lane, all, e);
        s_in[lane] = make_float2(e[0], e[1]);
    }
    for (int j = kBwdWarps - 1; j > warp; --j) after = joined(after, segment_of(s_rev[j][lane]));
    __syncthreads();
    float carry[2] = {s_in[lane].x, s_in[lane].y};
    if (warp < kBwdWarps - 1) apply(after, carry);

    float prev[kSegTokens][2], total[2] = {0.0f, 0.0f};
    T *ox = dx + (row0 + t0) * s.D + d0, *orr = dr + (row0 + t0) * s.lddg + d0, *og = dg + (row0 + t0) * s.lddg + d0;
    auto finish = [&](auto is_easy) {
        constexpr bool kEasy = decltype(is_easy)::value;
#pragma unroll
        for (int t = 0; t < kSegTokens; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (kEasy || t < n) {
                    if (!kEasy && (starts >> t & 1)) h[i] = 0.0f;
                    prev[t][i] = h[i];
                    h[i] += fmaf(root(input_square(om[t][i])), g[t][i] * vx[t].at(i), -om[t][i] * h[i]);
                }
#pragma unroll
        for (int t = kSegTokens - 1; t >= 0; --t)
            if (kEasy || t < n) {
                float vox[2], vog[2], vor[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float u = k[i] * r[t][i], a = decay_of<kEasy>(om[t][i], u), ua = u * a;
                    const float q = input_square(om[t][i]), rs = over_root(q), dh = vy[t].at(i) + carry[i];
                    const float gx = g[t][i] * vx[t].at(i), db = dh * (q * rs);
                    const float p = dh * (ua * prev[t][i] - ua * a * rs * gx);
                    vox[i] = db * g[t][i];
                    vog[i] = db * gx * (1.0f - g[t][i]);
                    vor[i] = (r[t][i] - 1.0f) * p;
                    total[i] += p;
                    carry[i] = !kEasy && (starts >> t & 1) ? 0.0f : a * dh;
                }
                store_two<T, kPair>(ox + t * s.D, vox[0], vox[1], in0, in1);
                store_two<T, kPair>(orr + t * s.lddg, vor[0], vor[1], in0, in1);
                store_two<T, kPair>(og + t * s.lddg, vog[0], vog[1], in0, in1);
            }
    };
    if (easy) finish(std::true_type{});
    else finish(std::false_type{});
    s_sum[warp][lane] = make_float2(total[0], total[1]);
    if (dinit && c == 0 && warp == 0) {
        if (in0) dinit[b * s.D + d0] = carry[0];
        if (in1) dinit[b * s.D + d1] = carry[1];
    }
    __syncthreads();
    if (warp == 0) {
        float2 v = s_sum[0][lane];
#pragma unroll
        for (int j = 1; j < kBwdWarps; ++j) {
            v.x += s_sum[j][lane].x;
            v.y += s_sum[j][lane].y;
        }
        float *o = part + (b * w.chunks + c) * s.D;
        if (in0) o[d0] = v.x;
        if (in1) o[d1] = v.y;
    }
}

// ---- one token
template <typename T>
__global__ void __launch_bounds__(128)
gated_step_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                  const float *__restrict__ lam, float *__restrict__ state, T *__restrict__ y, int64_t D, int64_t ldx,
                  int64_t ldg, float c) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (d >= D) return;
    const float u = c * softplus_f(lam[d]) * sigmoid_f(to_f(rr[b * ldg + d])), om = loss_of<false>(u);
    float h = state[b * D + d];
    h += fmaf(root(input_square(om)), sigmoid_f(to_f(gr[b * ldg + d])) * to_f(x[b * ldx + d]), -om * h);
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
    // one CTA per 64 tokens and 64 channels, numbered in 31 bits
    if ((double)b * (double)((L + kGatedChunk - 1) / kGatedChunk) * (double)((D + kTileCh - 1) / kTileCh) >= 2147483648.0)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int64_t chunks_of(int64_t L, int backward) {
    const int q = backward ? kBwdChunk : kFwdChunk;
    return (L + q - 1) / q;
}

// The workspace: status and ticket, the flags (zeroed with them), the
// segments and states of the chunks, and the backward's sums of p per chunk.
struct Regions {
    Handoff w;
    float *part;
    size_t zeroed, total;
};

Regions regions_of(void *workspace, int64_t b, int64_t L, int64_t D, int backward) {
    Regions r = {};
    const int64_t chunks = chunks_of(L, backward), groups = (chunks + kGroup - 1) / kGroup;
    const int64_t tiles = (D + kTileCh - 1) / kTileCh;
    size_t at = kStatusBytes;
    auto take = [&](size_t bytes) {
        char *p = static_cast<char *>(workspace) + at;
        at += align256(bytes);
        return p;
    };
    r.w.status = static_cast<unsigned *>(workspace);
    r.w.ticket = r.w.status + 1;
    r.w.chunks = (int)chunks; r.w.groups = (int)groups; r.w.tiles = (int)tiles;
    if (chunks > 1) {
        r.w.seg_ready = reinterpret_cast<unsigned *>(take((size_t)(b * chunks * tiles) * 4));
        r.w.state_ready = reinterpret_cast<unsigned *>(take((size_t)(b * groups * tiles) * 4));
        r.zeroed = at;
        r.w.seg = reinterpret_cast<float4 *>(take((size_t)(b * chunks * tiles) * 32 * sizeof(float4)));
        r.w.state = reinterpret_cast<float2 *>(take((size_t)(b * groups * tiles) * 32 * sizeof(float2)));
    }
    if (backward) r.part = reinterpret_cast<float *>(take((size_t)(b * chunks * D) * sizeof(float)));
    r.total = at;
    return r;
}

size_t workspace_bytes_of(int64_t b, int64_t L, int64_t D, int backward) {
    return regions_of(nullptr, b, L, D, backward).total;
}

// Whether rows of these tensors start on pairs of elements.
bool pairs_of(int64_t D, int in_dtype, std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> lds) {
    if (D % 2) return false;
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & (in_dtype == SSD_BF16 ? 3u : 7u)) return false;
    for (int64_t ld : lds)
        if (ld % 2) return false;
    return true;
}

struct FwdArgs {
    const void *x, *r, *g;
    const float *lam, *init;
    const int32_t *ids;
    void *y;
    float *fin, *states;
};
struct BwdArgsOf {
    FwdArgs f;
    const void *dy;
    const float *dfin;
    void *dx, *dr, *dg;
    float *dinit;
};

template <typename T, bool kPair>
void scan_launch(const FwdArgs &a, const ScanShape &s, const Handoff &w, unsigned grid, cudaStream_t st) {
    gated_scan_kernel<T, kPair><<<grid, 32 * kFwdWarps, 0, st>>>((const T *)a.x, (const T *)a.r, (const T *)a.g, a.lam,
                                                                 a.init, a.ids, (T *)a.y, a.fin, a.states, s, w);
}
template <typename T, bool kPair>
void bwd_launch(const BwdArgsOf &a, const ScanShape &s, const Handoff &w, float *part, unsigned grid, cudaStream_t st) {
    gated_bwd_kernel<T, kPair><<<grid, 32 * kBwdWarps, 0, st>>>(
        (const T *)a.f.x, (const T *)a.f.r, (const T *)a.f.g, a.f.lam, a.f.init, a.f.ids, a.f.states, (const T *)a.dy,
        a.dfin, (T *)a.dx, (T *)a.dr, (T *)a.dg, part, a.dinit, s, w);
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
    cudaError_t e = cudaSuccess;
    if (batch == 0 || seqlen == 0) {
        // no tokens: the state leaves as it came in
        e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
        if (e == cudaSuccess && batch > 0 && final_state) {
            const size_t n = (size_t)(batch * dim) * sizeof(float);
            e = init_state ? cudaMemcpyAsync(final_state, init_state, n, cudaMemcpyDeviceToDevice, s)
                           : cudaMemsetAsync(final_state, 0, n, s);
        }
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    const ssd::Regions r = ssd::regions_of(workspace, batch, seqlen, dim, 0);
    // with one chunk nothing is handed on, and the kernel clears the status itself
    if (r.w.chunks > 1 && (e = cudaMemsetAsync(workspace, 0, r.zeroed, s)) != cudaSuccess)
        return (ssd_status)ssd::record_cuda_error(e);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedScan);
        const ssd::FwdArgs a = {x, r_raw, g_raw, lam, init_state, seq_idx, y, final_state, chunk_states};
        const ssd::ScanShape sh = {seqlen, dim, ld_x, ld_gate, 0, decay_scale, (int)batch, r.w.tiles};
        const unsigned grid = (unsigned)(batch * r.w.chunks * r.w.tiles);
        const bool pair = ssd::pairs_of(dim, in_dtype, {x, r_raw, g_raw, y}, {ld_x, ld_gate});
        if (in_dtype == SSD_BF16)
            (pair ? ssd::scan_launch<__nv_bfloat16, true> : ssd::scan_launch<__nv_bfloat16, false>)(a, sh, r.w, grid, s);
        else
            (pair ? ssd::scan_launch<float, true> : ssd::scan_launch<float, false>)(a, sh, r.w, grid, s);
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
    cudaError_t e = cudaSuccess;
    if (!has_tokens) {
        // no tokens: no gradient of lam, and the seed passes to the initial state as it is
        e = cudaMemsetAsync(workspace, 0, ssd::kStatusBytes, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(dlam, 0, (size_t)dim * sizeof(float), s);
        if (e == cudaSuccess && dinit_state && batch > 0) {
            const size_t n = (size_t)(batch * dim) * sizeof(float);
            e = dfinal_state ? cudaMemcpyAsync(dinit_state, dfinal_state, n, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(dinit_state, 0, n, s);
        }
        return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
    }
    const ssd::Regions r = ssd::regions_of(workspace, batch, seqlen, dim, 1);
    if (r.w.chunks > 1 && (e = cudaMemsetAsync(workspace, 0, r.zeroed, s)) != cudaSuccess)
        return (ssd_status)ssd::record_cuda_error(e);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedBwd);
        const ssd::BwdArgsOf a = {{x, r_raw, g_raw, lam, init_state, seq_idx, nullptr, nullptr,
                                   const_cast<float *>(chunk_states)},
                                  dy, dfinal_state, dx, dr_raw, dg_raw, dinit_state};
        const ssd::ScanShape sh = {seqlen, dim, ld_x, ld_gate, ld_dgate, decay_scale, (int)batch, r.w.tiles};
        const unsigned grid = (unsigned)(batch * r.w.chunks * r.w.tiles);
        const bool pair = ssd::pairs_of(dim, in_dtype, {x, r_raw, g_raw, dy, dx, dr_raw, dg_raw}, {ld_x, ld_gate, ld_dgate});
        if (in_dtype == SSD_BF16)
            (pair ? ssd::bwd_launch<__nv_bfloat16, true> : ssd::bwd_launch<__nv_bfloat16, false>)(a, sh, r.w, r.part, grid, s);
        else
            (pair ? ssd::bwd_launch<float, true> : ssd::bwd_launch<float, false>)(a, sh, r.w, r.part, grid, s);
    }
    e = cudaGetLastError();
    if (e == cudaSuccess) e = ssd::column_sum(r.part, dlam, lam, batch * r.w.chunks, dim, dim, s);
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
