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
// the product modulo 2^64 is the angle modulo one turn, to position * 2^-64 of a
// turn (2^-33 at most) for frequencies up to 2^40 radians per position.
#include <math.h>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_f2.cuh"
#include "ssd_internal.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kNrWarps = 8;
constexpr int64_t kNrMaxWarps = 148 * 32;   // warps of a backward launch: rows of weight partials
constexpr int kNrSumRows = 64;              // most rows behind one float32 running sum

// inv_freq (radians per position) as turns per position, modulo 1, in 2^-64.  The
// quotient by 2 pi is carried in two doubles (1 / (2 pi) to 107 bits), since whole
// turns take bits from its fraction and a far position multiplies what is lost: in
// one double a frequency of 1 was 1.3e-7 rad off at position 2^31, 1e4 1.6e-3.
__device__ __forceinline__ uint64_t turns_of(float inv_freq) {
    constexpr double kScale = 18446744073709551616.0;   // 2^64
    const double f = (double)inv_freq, hi = 0.15915494309189535, lo = -9.839338337591243e-18;
    const double p = f * hi, rest = __fma_rn(f, lo, __fma_rn(f, hi, -p)), v = p - rint(p);   // v in [-1/2, 1/2], exact
    return (uint64_t)__double2ll_rn((v >= 0.5 ? -v : v) * kScale) + (uint64_t)__double2ll_rn(rest * kScale);
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

// ---- widths of a multiple of 8, up to 512 (and rotated widths of a multiple of 8)
//
// A group of kW lanes takes a token.  A lane holds a unit of 8 elements, the
// same in every row: 8 consecutive ones, or with pairs across halves 4 of the
// first half and their 4 partners, so no pair crosses lanes; two 8-byte (bf16)
// or 16-byte loads.  Its cosines and sines are made once for the token and
// serve B and C of all groups, its weights stay in registers, and the rows'
// sums of squares cross the group by shuffles.  Bound by HBM (4 bytes an
// element of bf16 forward, 6 backward), next by issue slots (hence packed
// float32): the rows of the next two groups (backward: one) are loaded while
// these are worked on, at two blocks an SM (three spill, and the fp32 backward 10 to 17
// words at two).  Measured: 65536 x 8 groups x 128 bf16 99 to 102 us (0.83 to 0.81 of
// HBM), backward 183 us (0.67); fp32 184 us (0.89) and 280 us (0.88).
struct NormArgs {
    const void *B, *C, *dBo, *dCo;
    const float *wB, *wC, *freq;
    const int32_t *pos;
    void *Bo, *Co;                 // backward: dB, dC
    float *part;                   // backward: [blocks, 2, N]
    int64_t items, L;              // items: tokens x parts of the groups
    int G, N, R, per, parts, turns_each;   // per: groups of an item; turns_each: items of a lane group (backward)
    float eps;
};
constexpr int kNrThreads = 256;

// Four elements as two packed pairs: (0, 1), (2, 3)
template <typename T> struct Quad;
template <> struct Quad<float> {
    using type = ulonglong2;
    static __device__ __forceinline__ void get(ulonglong2 q, f2 &a, f2 &b) {
        a = q.x;
        b = q.y;
    }
    static __device__ __forceinline__ ulonglong2 of(f2 a, f2 b) { return make_ulonglong2(a, b); }
};
template <> struct Quad<__nv_bfloat16> {
    using type = uint2;
    static __device__ __forceinline__ void get(uint2 q, f2 &a, f2 &b) {
        a = two(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u));
        b = two(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint2 of(f2 a, f2 b) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(lo(a), hi(a)), y = __floats2bfloat162_rn(lo(b), hi(b));
        return make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
};

// The 8 elements of a unit: p and q hold the first and the second of its four
// pairs (without rotation the pairing means nothing).
struct Octet {
    f2 p[2], q[2];
};
template <typename T, bool kInter> __device__ __forceinline__ Octet octet_of(const typename Quad<T>::type (&v)[2]) {
    Octet o;
    if constexpr (kInter) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f2 a, b;
            Quad<T>::get(v[i], a, b);
            o.p[i] = two(lo(a), lo(b));
            o.q[i] = two(hi(a), hi(b));
        }
    } else {
        Quad<T>::get(v[0], o.p[0], o.p[1]);
        Quad<T>::get(v[1], o.q[0], o.q[1]);
    }
    return o;
}

template <int kW> __device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// What a lane knows of its units.
template <bool kInter, int kW, int kUnits> struct Unit {
    int e0[kUnits], e1[kUnits];    // where its two quads start
    bool on[kUnits], rot[kUnits];
    uint64_t turns[kUnits][4];
    f2 c[kUnits][2], s[kUnits][2];      // of its four pairs
    __device__ __forceinline__ explicit Unit(const NormArgs &a) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = threadIdx.x % kW + i * kW;
            on[i] = u < a.N / 8;
            rot[i] = u < a.R / 8;
            const bool apart = !kInter && rot[i];
            e0[i] = apart ? 4 * u : 8 * u;
            e1[i] = apart ? 4 * u + a.R / 2 : 8 * u + 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                turns[i][j] = rot[i] ? turns_of(a.freq[4 * u + j]) : 0;
            }
            c[i][0] = c[i][1] = two(1.0f);
            s[i][0] = s[i][1] = two(0.0f);
        }
    }
    __device__ __forceinline__ void turn_to(int pos) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            if (rot[i]) {
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) turn(pos, turns[i][j], x[j], y[j]);
                c[i][0] = two(x[0], x[1]);
                c[i][1] = two(x[2], x[3]);
                s[i][0] = two(y[0], y[1]);
                s[i][1] = two(y[2], y[3]);
            }
    }
    // rotated by the angle (kSign 1) or back (-1); units past the rotated part stay as
    // they are (a turn by 0 would bring 0 times an infinity to its neighbour)
    template <int kSign, bool kAll = false> __device__ __forceinline__ void rotate(int i, Octet &v) const {
        if (!kAll && !rot[i]) return;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const f2 ns = mul(s[i][j], two(-1.0f)), p = v.p[j], q = v.q[j];
            v.p[j] = fma(p, c[i][j], mul(q, kSign > 0 ? ns : s[i][j]));
            v.q[j] = fma(q, c[i][j], mul(p, kSign > 0 ? s[i][j] : ns));
        }
    }
    template <typename T> __device__ __forceinline__ void load(int i, const T *row, bool there, typename Quad<T>::type (&q)[2]) const {
        using Q = typename Quad<T>::type;
        q[0] = q[1] = Q{};
        if (there && on[i]) {
            q[0] = *reinterpret_cast<const Q *>(row + e0[i]);
            q[1] = *reinterpret_cast<const Q *>(row + e1[i]);
        }
    }
    template <typename T> __device__ __forceinline__ void store(int i, T *row, const Octet &v) const {
        using Q = typename Quad<T>::type;
        if (!on[i]) return;
        if constexpr (kInter) {
            *reinterpret_cast<Q *>(row + e0[i]) = Quad<T>::of(two(lo(v.p[0]), lo(v.q[0])), two(hi(v.p[0]), hi(v.q[0])));
            *reinterpret_cast<Q *>(row + e1[i]) = Quad<T>::of(two(lo(v.p[1]), lo(v.q[1])), two(hi(v.p[1]), hi(v.q[1])));
        } else {
            *reinterpret_cast<Q *>(row + e0[i]) = Quad<T>::of(v.p[0], v.p[1]);
            *reinterpret_cast<Q *>(row + e1[i]) = Quad<T>::of(v.q[0], v.q[1]);
        }
    }
    __device__ __forceinline__ void weights(const float *w, Octet (&v)[kUnits]) const {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            ulonglong2 q[2] = {};
            if (on[i]) {
                q[0] = make_ulonglong2(two(w[e0[i]], w[e0[i] + 1]), two(w[e0[i] + 2], w[e0[i] + 3]));
                q[1] = make_ulonglong2(two(w[e1[i]], w[e1[i] + 1]), two(w[e1[i] + 2], w[e1[i] + 3]));
            }
            v[i] = octet_of<float, kInter>(q);
        }
    }
};

__device__ __forceinline__ int position_of(const NormArgs &a, int64_t tok) {
    if (a.pos) return a.pos[tok];
    return (uint64_t)tok >> 32 ? (int)(tok % a.L) : (int)((uint32_t)tok % (uint32_t)a.L);
}

// kAll: all elements are rotated.  The test for it in the loop takes the forward of 65536 x 8 x
// 128 bf16 from 94 to 96 us (fp32 183 either way), and the backward of 8192 x 2 x 512 from 38.7
// to 40.4; the backward of narrower rows is faster with it (65536 x 8 x 128 bf16 174, 178 without; fp32 265, 267).
template <typename T, bool kInter, bool kAll, int kW, int kUnits>
__global__ void __launch_bounds__(kNrThreads, kUnits == 1 ? 2 : 1)
norm_rotate_units_kernel(const __grid_constant__ NormArgs a) {
    using Q = typename Quad<T>::type;
    Unit<kInter, kW, kUnits> unit(a);
    Octet w[2][kUnits];
    unit.weights(a.wB, w[0]);
    unit.weights(a.wC, w[1]);
    const float inv_n = 1.0f / (float)a.N;
    const int64_t step = (int64_t)gridDim.x * (kNrThreads / kW);
    const int64_t item0 = (int64_t)blockIdx.x * (kNrThreads / kW) + threadIdx.x / kW;
    // two groups of a token at a time; the next two are loaded while these are worked on
    struct Place {
        int64_t tok, at;
        int g, last;      // groups g and g + 1, up to `last`
    };
    auto place = [&](int64_t item, int g) -> Place {
        const bool valid = item < a.items;
        const int64_t it = valid ? item : 0, tok = a.parts == 1 ? it : it / a.parts;
        const int g0 = (int)(it - tok * a.parts) * a.per;
        return Place{tok, (tok * a.G + g0 + g) * a.N, g0 + g, valid ? min(a.G, g0 + a.per) : 0};
    };
    Q q[2][2][kUnits][2];
    auto load = [&](const Place &p) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    unit.template load<T>(i, static_cast<const T *>(which ? a.C : a.B) + p.at + k * a.N, p.g + k < p.last, q[k][which][i]);
    };
    Place next = place(item0, 0);
    load(next);
    // all lanes of a warp go round together: shuffles
    for (int64_t item = item0; __any_sync(0xffffffffu, item < a.items); item += step) {
        unit.turn_to(position_of(a, next.tok));
#pragma unroll 1
        for (int g = 0; g < a.per; g += 2) {
            const Place p = next;
            Q r[2][2][kUnits][2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int which = 0; which < 2; ++which)
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        r[k][which][i][0] = q[k][which][i][0];
                        r[k][which][i][1] = q[k][which][i][1];
                    }
            next = g + 2 < a.per ? place(item, g + 2) : place(item + step, 0);
            load(next);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (k && g + 1 >= a.per) break;
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    Octet v[kUnits];
                    f2 sq = two(0.0f);
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
                        v[i] = octet_of<T, kInter>(r[k][which][i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) sq = fma(v[i].p[j], v[i].p[j], fma(v[i].q[j], v[i].q[j], sq));
                    }
                    const f2 rs = two(1.0f / sqrtf(fmaf(group_sum<kW>(lo(sq) + hi(sq)), inv_n, a.eps)));
                    T *o = static_cast<T *>(which ? a.Co : a.Bo) + p.at + k * a.N;
#pragma unroll
                    for (int i = 0; i < kUnits; ++i) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            v[i].p[j] = mul(mul(v[i].p[j], rs), w[which][i].p[j]);
                            v[i].q[j] = mul(mul(v[i].q[j], rs), w[which][i].q[j]);
                        }
                        unit.template rotate<1, kAll>(i, v[i]);
                        if (p.g + k < p.last) unit.template store<T>(i, o, v[i]);
                    }
                }
            }
        }
    }
}

// Backward.  A lane group takes turns_each items, a lane keeps the weights'
// gradients of its elements; the block adds them up in lane group order.
template <typename T, bool kInter, bool kAll, int kW, int kUnits>
__global__ void __launch_bounds__(kNrThreads, kUnits == 1 ? 2 : 1)
norm_rotate_units_bwd_kernel(const __grid_constant__ NormArgs a) {
    using Q = typename Quad<T>::type;
    constexpr int kGroups = kNrThreads / kW;
    __shared__ __align__(16) float s_acc[kGroups][kUnits * kW * 8 + 4];
    Unit<kInter, kW, kUnits> unit(a);
    Octet w[2][kUnits], acc[2][kUnits];
    unit.weights(a.wB, w[0]);
    unit.weights(a.wC, w[1]);
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < kUnits; ++i) acc[which][i] = Octet{{0, 0}, {0, 0}};
    const float inv_n = 1.0f / (float)a.N;
    const int me = threadIdx.x / kW;
    // one (token, group) after the other; the next one's rows are loaded while
    // this one's are worked on
    struct Place {
        int64_t at;     // where its rows start
        int64_t tok;
        bool there;
    };
    auto place = [&](int n, int g) -> Place {
        const int64_t item = ((int64_t)blockIdx.x * a.turns_each + n) * kGroups + me;
        const bool valid = n < a.turns_each && item < a.items;
        const int64_t it = valid ? item : 0, tok = a.parts == 1 ? it : it / a.parts;
        const int g0 = (int)(it - tok * a.parts) * a.per;
        return Place{(tok * a.G + g0 + g) * a.N, tok, valid && g0 + g < a.G};
    };
    Q qv[2][kUnits][2], qd[2][kUnits][2];
    auto load = [&](const Place &p) {
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                unit.template load<T>(i, static_cast<const T *>(which ? a.C : a.B) + p.at, p.there, qv[which][i]);
                unit.template load<T>(i, static_cast<const T *>(which ? a.dCo : a.dBo) + p.at, p.there, qd[which][i]);
            }
    };
    Place next = place(0, 0);
    load(next);
#pragma unroll 1
    for (int n = 0; n < a.turns_each; ++n) {
        unit.turn_to(position_of(a, next.tok));
#pragma unroll 1
        for (int g = 0; g < a.per; ++g) {
            const bool there = next.there;
            const int64_t at = next.at;
            Q rv[2][kUnits][2], rd[2][kUnits][2];
#pragma unroll
            for (int which = 0; which < 2; ++which)
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        rv[which][i][k] = qv[which][i][k];
                        rd[which][i][k] = qd[which][i][k];
                    }
            next = g + 1 < a.per ? place(n, g + 1) : place(n + 1, 0);
            load(next);
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                Octet v[kUnits], d[kUnits];
                f2 sq = two(0.0f), sm = two(0.0f);
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    v[i] = octet_of<T, kInter>(rv[which][i]);
                    d[i] = octet_of<T, kInter>(rd[which][i]);
                    unit.template rotate<-1, kAll>(i, d[i]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        sq = fma(v[i].p[j], v[i].p[j], fma(v[i].q[j], v[i].q[j], sq));
                        sm = fma(mul(d[i].p[j], w[which][i].p[j]), v[i].p[j], sm);
                        sm = fma(mul(d[i].q[j], w[which][i].q[j]), v[i].q[j], sm);
                    }
                }
                // (0 where the lanes have no row: their zeros with eps 0 would make it infinite, and the weights' sums NaN)
                const float mean = fmaf(group_sum<kW>(lo(sq) + hi(sq)), inv_n, a.eps), r = there ? 1.0f / sqrtf(mean) : 0.0f;
                const float m = group_sum<kW>(lo(sm) + hi(sm)) * r * inv_n;   // mean of dn w n
                const f2 rs = two(r), nm = two(-m);
                T *o = static_cast<T *>(which ? a.Co : a.Bo) + at;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    Octet out;
                    auto one = [&](f2 x, f2 dn, f2 weight, f2 &sum) -> f2 {
                        const f2 nrm = mul(x, rs);
                        sum = fma(dn, nrm, sum);
                        return mul(rs, fma(dn, weight, mul(nrm, nm)));
                    };
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        out.p[j] = one(v[i].p[j], d[i].p[j], w[which][i].p[j], acc[which][i].p[j]);
                        out.q[j] = one(v[i].q[j], d[i].q[j], w[which][i].q[j], acc[which][i].q[j]);
                    }
                    if (there) unit.template store<T>(i, o, out);
                }
            }
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            unit.template store<float>(i, s_acc[me], acc[which][i]);
        __syncthreads();
        for (int e = threadIdx.x; e < a.N; e += kNrThreads) {
            float t = s_acc[0][e];
#pragma unroll
            for (int k = 1; k < kGroups; ++k) t += s_acc[k][e];
            a.part[((int64_t)blockIdx.x * 2 + which) * a.N + e] = t;
        }
    }
}

// ---- other widths: one warp per (token, group), lanes across pairs, B then C.
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

int64_t bwd_warps(int64_t rows) {
    const int64_t least = (rows + kNrSumRows - 1) / kNrSumRows;
    return rows < kNrMaxWarps ? rows : least < kNrMaxWarps ? kNrMaxWarps : least;
}

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

bool units_fit(int64_t N, int64_t R) { return N % 8 == 0 && R % 8 == 0 && N <= 512; }

// The groups of an item: all of a token's while that leaves every SM lane
// groups to hide the loads with, fewer when tokens are few.
void split_groups(NormArgs *a, int64_t tokens, int most) {
    const int64_t want = 148 * 64;
    int64_t parts = tokens >= want ? 1 : (want + tokens - 1) / tokens;
    if (parts > a->G) parts = a->G;
    int per = (int)((a->G + parts - 1) / parts);
    if (per > most) per = most;
    a->per = per;
    a->parts = (a->G + per - 1) / per;
    a->items = tokens * a->parts;
}

template <typename T, bool kInter, int kW, int kUnits> void units_launch(const NormArgs &a, unsigned blocks, bool back, cudaStream_t s) {
    auto kern = a.R == a.N ? norm_rotate_units_kernel<T, kInter, true, kW, kUnits> : norm_rotate_units_kernel<T, kInter, false, kW, kUnits>;
    if (back) {
        kern = norm_rotate_units_bwd_kernel<T, kInter, false, kW, kUnits>;
        if constexpr (kUnits == 2) {
            if (a.R == a.N) kern = norm_rotate_units_bwd_kernel<T, kInter, true, kW, kUnits>;
        }
    }
    kern<<<blocks, kNrThreads, 0, s>>>(a);
}
template <typename T, bool kInter> void units_of(const NormArgs &a, unsigned blocks, bool back, cudaStream_t s) {
    if (a.N <= 64) units_launch<T, kInter, 8, 1>(a, blocks, back, s);
    else if (a.N <= 128) units_launch<T, kInter, 16, 1>(a, blocks, back, s);
    else if (a.N <= 256) units_launch<T, kInter, 32, 1>(a, blocks, back, s);
    else units_launch<T, kInter, 32, 2>(a, blocks, back, s);
}
int groups_of_block(int N) { return kNrThreads / (N <= 64 ? 8 : N <= 128 ? 16 : 32); }

template <typename T>
void fwd_launch(NormArgs a, int64_t tokens, int il, cudaStream_t s) {
    TraceScope tr(s, kTrNormRotate);
    const int64_t rows = tokens * a.G;
    if (units_fit(a.N, a.R)) {
        split_groups(&a, tokens, 1 << 30);
        const int64_t per_block = groups_of_block(a.N), blocks = (a.items + per_block - 1) / per_block, most = 148 * (a.N <= 256 ? 2 : 1);
        (il ? units_of<T, true> : units_of<T, false>)(a, (unsigned)(blocks < most ? blocks : most), false, s);
        return;
    }
    norm_rotate_kernel<T><<<(unsigned)((rows + kNrWarps - 1) / kNrWarps), 32 * kNrWarps, 0, s>>>(
        (const T *)a.B, (const T *)a.C, a.wB, a.wC, a.freq, a.pos, (T *)a.Bo, (T *)a.Co, rows, a.L, a.G, a.N, a.R, a.eps, il);
}

// Returns the rows of weight partials it leaves in a.part (no more than bwd_warps).
template <typename T>
int64_t bwd_launch(NormArgs a, int64_t tokens, int il, cudaStream_t s) {
    TraceScope tr(s, kTrNormRotateBwd);
    const int64_t rows = tokens * a.G;
    if (units_fit(a.N, a.R)) {
        // at most 32 rows of a lane group and 32 groups behind a running sum;
        // fewer items each while that leaves the SMs fewer than two blocks
        split_groups(&a, tokens, 32);
        const int64_t per_block = groups_of_block(a.N), wave = 148 * 2 * per_block;
        int64_t each = (a.items + wave - 1) / wave;
        if (each * a.per > 32) each = 32 / a.per;
        a.turns_each = (int)each;
        const int64_t blocks = (a.items + per_block * each - 1) / (per_block * each);
        (il ? units_of<T, true> : units_of<T, false>)(a, (unsigned)blocks, true, s);
        return blocks;
    }
    const int64_t warps = bwd_warps(rows);
    norm_rotate_bwd_kernel<T><<<(unsigned)((warps + kNrWarps - 1) / kNrWarps), 32 * kNrWarps, 0, s>>>(
        (const T *)a.B, (const T *)a.C, a.wB, a.wC, a.freq, a.pos, (const T *)a.dBo, (const T *)a.dCo, (T *)a.Bo, (T *)a.Co,
        a.part, rows, warps, a.L, a.G, a.N, a.R, a.eps, il);
    return warps;
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
    ssd::NormArgs a = {};
    a.B = B; a.C = C; a.wB = weight_B; a.wC = weight_C; a.freq = inv_freq; a.pos = positions;
    a.Bo = B_out; a.Co = C_out; a.L = seqlen; a.G = (int)ngroups; a.N = (int)state_dim; a.R = (int)rot_dim; a.eps = eps;
    (in_dtype == SSD_BF16 ? ssd::fwd_launch<__nv_bfloat16> : ssd::fwd_launch<float>)(a, batch * seqlen, interleaved, s);
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
    ssd::NormArgs a = {};
    a.B = B; a.C = C; a.dBo = dB_out; a.dCo = dC_out; a.wB = weight_B; a.wC = weight_C; a.freq = inv_freq;
    a.pos = positions; a.Bo = dB; a.Co = dC; a.part = part; a.L = seqlen; a.G = (int)ngroups; a.N = (int)state_dim;
    a.R = (int)rot_dim; a.eps = eps;
    const int64_t sums = (in_dtype == SSD_BF16 ? ssd::bwd_launch<__nv_bfloat16> : ssd::bwd_launch<float>)(
        a, batch * seqlen, interleaved, s);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = ssd::column_sum(part, dweight_B, nullptr, sums, 2 * state_dim, 2 * state_dim, s, dweight_C, state_dim);
    return e == cudaSuccess ? SSD_OK : (ssd_status)ssd::record_cuda_error(e);
}

}  // extern "C"
