// The gated linear recurrence, one decay per channel: scan, backward, step.
//   r = sigmoid(r_raw), g = sigmoid(g_raw), u = c softplus(lam) r, a = e^-u,
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) g_t x_t
// Written with om = a - 1 (which keeps its relative accuracy where a is near 1,
// the long memories):  h_t = h_{t-1} + (om h_{t-1} + beta g x),
// beta = sqrt(-om (2 + om)).
//
// One pass over the data.  A CTA takes a chunk of tokens by 64 channels; a
// warp 8 or 16 consecutive tokens, a lane two channels.  A warp folds its tokens
// into a segment (A, H), which makes A h + H of the state h entering it, and
// forward keeps that of every token, so the state that arrives later finishes
// them independently.  Segments join in a fixed order, inside the CTA through
// shared memory and across chunks through the workspace (hand_on and gather
// below).  So x and the gates are read once and y is written once, where a
// first pass over the chunks' totals would read the inputs twice; and the
// order of every sum is fixed by the sizes alone, whichever CTA runs first.
//
// A CTA lives for many tiles: the rows of the tile after next are on their way
// to shared memory (TMA where rows start on 16 bytes, 4-byte asynchronous
// copies else), and the ticket of the one behind is drawn, while a tile is
// worked on, so neither is waited for.  The last warp does this between the
// two barriers of a tile, where all wait for the chunk before; a warp of its
// own would cost the others a fifth of their registers.
//
// What bounds it: HBM (8 bytes an element of bf16 forward, 14 backward) comes
// next to the issue slots: 30 instructions an element forward and 70 backward,
// 20 and 49 of them arithmetic, at half the issue rate, since two CTAs of an SM
// take all of its registers and both wait between a tile's two halves.
// Measured on B200s: 65536 x 5120 bf16 forward 0.616 to 0.635 ms (0.67 to 0.65 of
// HBM), backward 1.38 ms (0.52); 65536 x 2560 fp32 0.523 ms (0.79) and 1.03 ms (0.70).
#include <math.h>

#include <initializer_list>
#include <type_traits>

#include "../../include/ssd.h"
#include "ssd_common.cuh"
#include "ssd_f2.cuh"
#include "ssd_internal.h"
#include "ssd_tc.cuh"
#include "ssd_tmap.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

constexpr int kGatedChunk = 64;   // tokens between chunk states
constexpr int kTileCh = 64;       // channels of a CTA: two a lane
// Tokens of a CTA and of a warp: what a warp keeps in registers.  16 tokens of
// a warp halve the joins against 8 and fit 128 registers; stages of fp32 rows
// leave two CTAs of an SM room for 64 tokens each.
template <typename T> constexpr int kFwdChunk = sizeof(T) == 2 ? 128 : 64;
template <typename T> constexpr int kFwdSeg = kFwdChunk<T> / 8;
constexpr int kFwdWarps = 8;
constexpr int kBwdChunk = 64, kBwdSeg = 8, kBwdWarps = kBwdChunk / kBwdSeg;
constexpr int kGroup = 16;        // chunks a look-back joins before it needs the state of the group before
static_assert(kBwdChunk == kGatedChunk && kFwdChunk<float> % kGatedChunk == 0 && kFwdChunk<__nv_bfloat16> % kGatedChunk == 0,
              "chunk states at chunk ends");
constexpr float kLog2e = 1.4426950408889634f;

// The special functions as the hardware has them, numbers below float32's
// normal range taken as 0: the library forms rescale around that range, which
// more than doubled this file's instructions (123 an element of the scan,
// against 50) and moves nothing here.  Each is within 2 roundings of a float32 of its
// argument; the exponentials' arguments, raw * log2(e), are rounded before, which
// moves a gate by up to |raw| roundings (10 at a gate of -10, shut to 5e-5).
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Down to the smallest number: decays, which come times u in the gradients.
__device__ __forceinline__ float ex2_whole(float v) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// sqrt(q), 0 at 0
__device__ __forceinline__ float root(float q) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(q));
    return r;
}

__device__ __forceinline__ float get(f2 v, int i) { return i ? hi(v) : lo(v); }
__device__ __forceinline__ void put(f2 &v, int i, float x) { v = i ? two(lo(v), x) : two(x, hi(v)); }
// Both gates' sigmoids share one reciprocal: 1 / (1 + e1) = (1 + e2) / ((1 +
// e1)(1 + e2)).  Where an exponential is large (a gate shut) the product could
// overflow, so each has its own there; kOpen is the share below which the
// packed path leaves a warp to this one.
constexpr float kOpen = 1e-12f;
__device__ __forceinline__ void sigmoids_of(float er, float eg, float &r, float &g) {
    const float a = __fadd_rn(1.0f, er), b = __fadd_rn(1.0f, eg), both = rcp(a * b);
    const bool open = both > kOpen;
    r = open ? b * both : rcp(a);
    g = open ? a * both : rcp(b);
}
// The least of three, NaN if one is: a NaN gate leaves the packed path too, where it
// would reach the other gate through their reciprocal (and so, backward, the
// gradients of all tokens before).
__device__ __forceinline__ float least_of(float a, float b, float c) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %2, %3;\n\tmin.NaN.f32 %0, %1, t;\n\t}" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float exp_of_gate(float raw) { return ex2(raw * -kLog2e); }

// a - 1 = e^-u - 1 for u >= 0, to its own relative accuracy: u times the
// polynomial of least relative error (1.4e-8; 0.5 of 2^-24 with its
// coefficients rounded) below kNear, the exponential above.
constexpr float kNear = 0.35f;
constexpr float kP1 = -1.0f, kP2 = 0.49999812f, kP3 = -0.16662432f, kP4 = 0.04132745f, kP5 = -0.00720496f;
__device__ __forceinline__ float loss_of(float u) {
    float p = fmaf(u, kP5, kP4);
    p = fmaf(u, p, kP3);
    p = fmaf(u, p, kP2);
    p = fmaf(u, p, kP1);
    return u < kNear ? u * p : ex2(u * -kLog2e) - 1.0f;
}
__device__ __forceinline__ f2 loss_near(f2 u) {
    f2 p = fma(u, two(kP5), two(kP4));
    p = fma(u, p, two(kP3));
    p = fma(u, p, two(kP2));
    p = fma(u, p, two(kP1));
    return mul(u, p);
}
// a, from u and a - 1.  (Sums here and in the paths that are not packed are spelt
// so that no product is drawn into them: how rows lie in memory picks the
// kernel, and must not pick the bits.)
__device__ __forceinline__ float decay_of(float om, float u) { return u < kNear ? __fadd_rn(1.0f, om) : ex2_whole(u * -kLog2e); }
// a^2 - 1
__device__ __forceinline__ float less_square(float om) { return om * __fadd_rn(2.0f, om); }
__device__ __forceinline__ f2 less_square(f2 om) { return mul(om, add(om, two(2.0f))); }

// u a^2 / (1 - a^2) = u / (e^2u - 1), which is finite where the gate shuts
// and 1 - a^2 goes to 0: 1/2 - u/2 + u^2 q(u^2) below kNear, q the polynomial
// of least relative error of (1/6 - u^2/90 + ...), 3.6e-8 of it.
constexpr float kQ0 = 0.16666666f, kQ1 = -0.011110234f, kQ2 = 0.0010390305f;
__device__ __forceinline__ float input_slope(float u, float om) {
    const float v = u * u;
    const float near = fmaf(v, fmaf(v, fmaf(v, kQ2, kQ1), kQ0), fmaf(u, -0.5f, 0.5f));
    if (u < kNear) return near;
    const float a = decay_of(om, u);
    return a == 0.0f ? 0.0f : u * a * a * rcp(-less_square(om));
}
__device__ __forceinline__ f2 input_slope_near(f2 u) {
    const f2 v = mul(u, u);
    return fma(v, fma(v, fma(v, two(kQ2), two(kQ1)), two(kQ0)), fma(u, two(-0.5f), two(0.5f)));
}

template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }


// ---- segments of two channels: the state after one is a h + h0 (a < 0: a
// document starts inside, nothing of the state before it reaches the end)
struct Segment {
    f2 a, h;
};

// `first`, then `s`; kCuts: a document may start in either
template <bool kCuts> __device__ __forceinline__ Segment joined(const Segment &first, const Segment &s) {
    Segment r = {mul(first.a, s.a), fma(s.a, first.h, s.h)};
    if (kCuts) {
        const bool cut = lo(s.a) < 0.0f;
        if (cut) r.h = s.h;
        if (cut || lo(first.a) < 0.0f) r.a = two(-1.0f);
    }
    return r;
}
template <bool kCuts> __device__ __forceinline__ f2 after(const Segment &s, f2 h) {
    return kCuts && lo(s.a) < 0.0f ? s.h : fma(s.a, h, s.h);
}
__device__ __forceinline__ Segment segment_of(ulonglong2 v) { return Segment{v.x, v.y}; }
__device__ __forceinline__ ulonglong2 packed(const Segment &s) { return make_ulonglong2(s.a, s.h); }

// What the chunks of a row and channel tile hand on, in the workspace: zeros
// when the kernel starts.  A segment is written as one 16-byte word, whose
// first float is never all zero bits, so a reader needs no flag beside it and
// the writer no fence.
struct Handoff {
    unsigned *status, *ticket;
    float4 *seg;              // [b, chunks, tiles, 32]: a chunk's segment, two channels a lane
    float4 *state;            // [b, groups, tiles, 32]: the state after a group's last chunk (as h of a segment)
    int chunks, groups, tiles;
    long long budget;         // clock cycles before a wait gives up
};

__device__ __forceinline__ void hand_on(float4 *to, const Segment &s) {
    const f2 a = lo(s.a) == 0.0f ? two(-0.0f, hi(s.a)) : s.a;
    asm volatile("{\n\t.reg .b128 v;\n\tmov.b128 v, {%1, %2};\n\tst.relaxed.gpu.global.b128 [%0], v;\n\t}" ::"l"(to),
                 "l"(a), "l"(s.h)
                 : "memory");
}
// false: not there yet
__device__ __forceinline__ bool look(const float4 *from, Segment &s) {
    asm volatile("{\n\t.reg .b128 v;\n\tld.relaxed.gpu.global.b128 v, [%2];\n\tmov.b128 {%0, %1}, v;\n\t}"
                 : "=l"(s.a), "=l"(s.h)
                 : "l"(from)
                 : "memory");
    return (uint32_t)s.a != 0u;
}

// The state entering chunk c (0 is the first in scan order) is the state that
// the last chunk of the group of kGroup before has handed on, with the
// segments of the chunks between: a chain of chunks / kGroup hops, and the
// same sums in the same order on every run.  Warp `warp` waits for the
// segments of two of those chunks and leaves them joined in s_prev[warp], one
// warp the state in s_in (`first`: the state before chunk 0); the caller has
// all warps meet before `entering`.  A CTA waits only for tickets below its
// own, so for CTAs that run already.
template <int kWarps, bool kCuts>
__device__ __forceinline__ void gather(const Handoff &w, int b, int c, int tile, f2 first, ulonglong2 (*s_prev)[32],
                                       f2 *s_in, volatile int *abort) {
    static_assert(2 * kWarps == kGroup, "two chunks a warp");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = c / kGroup, pos = c % kGroup;
    const bool for_state = warp == kWarps - 2 && group > 0;
    const int mine = min(2, pos - 2 * warp);
    if (warp == kWarps - 2 && group == 0) s_in[lane] = first;
    if (mine <= 0 && !for_state) return;
    const float4 *from = &w.seg[(((int64_t)b * w.chunks + group * kGroup + 2 * warp) * w.tiles + tile) * 32 + lane];
    const float4 *st = &w.state[(((int64_t)b * w.groups + group - 1) * w.tiles + tile) * 32 + lane];
    Segment s0, s1, before;
    bool got0 = mine < 1, got1 = mine < 2, got = !for_state;
    const long long t0 = clock64();
    for (;;) {
        if (!got0) got0 = look(from, s0);
        if (!got1) got1 = look(from + (int64_t)w.tiles * 32, s1);
        if (!got) got = look(st, before);
        if (__all_sync(0xffffffffu, got0 && got1 && got)) break;
        const bool late = *abort || clock64() - t0 > w.budget;
        if (__any_sync(0xffffffffu, late)) {
            *abort = 1;
            break;
        }
    }
    if (mine > 0) s_prev[warp][lane] = packed(mine > 1 ? joined<kCuts>(s0, s1) : s0);
    if (for_state) s_in[lane] = before.h;
}

// The state entering chunk c, once all warps have gathered.
template <bool kCuts> __device__ __forceinline__ f2 entering(int c, const ulonglong2 (*s_prev)[32], const f2 *s_in) {
    const int lane = threadIdx.x & 31, pairs = (c % kGroup + 1) / 2;
    f2 h = s_in[lane];
#pragma unroll 4
    for (int j = 0; j < pairs; ++j) h = after<kCuts>(segment_of(s_prev[j][lane]), h);
    return h;
}

// ---- how a tile's rows come to shared memory
enum Source {
    kTma,      // rows start on 16 bytes
    kAsync,    // on 4 bytes (fp32, or bf16 in pairs): asynchronous copies of 4 bytes
    kOdd       // bf16 on single elements: the same copies from the word a row starts in, so it lands 0 or 1 elements further on
};

// Two channels of a token's staged row: adjacent ones where rows start on pairs
// of elements (kPair), else 32 apart.
template <typename T, bool kPair> __device__ __forceinline__ f2 two_of(const T *row, int lane) {
    if constexpr (!kPair) {
        return two(to_f(row[lane]), to_f(row[lane + 32]));
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t u = reinterpret_cast<const uint32_t *>(row)[lane];
        return two(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    } else {
        return reinterpret_cast<const f2 *>(row)[lane];
    }
}
// The other way, to a staged row (kTma) or the tensor's.
template <typename T, Source kSource, bool kPair>
__device__ __forceinline__ void store_two(T *staged, T *row, int lane, f2 v, bool in0, bool in1) {
    if constexpr (kSource == kTma) {
        if constexpr (sizeof(T) == 2) reinterpret_cast<__nv_bfloat162 *>(staged)[lane] = __floats2bfloat162_rn(lo(v), hi(v));
        else reinterpret_cast<f2 *>(staged)[lane] = v;
    } else if constexpr (!kPair) {
        if (in0) row[lane] = from_f<T>(lo(v));
        if (in1) row[lane + 32] = from_f<T>(hi(v));
    } else if (in1) {
        if constexpr (sizeof(T) == 2) reinterpret_cast<__nv_bfloat162 *>(row)[lane] = __floats2bfloat162_rn(lo(v), hi(v));
        else reinterpret_cast<f2 *>(row)[lane] = v;
    }
}

// Whether an element lies in the upper half of its word.
__device__ __forceinline__ unsigned odd_of(const void *p, int64_t elements) {
    return ((unsigned)(reinterpret_cast<uintptr_t>(p) >> 1) + (unsigned)elements) & 1u;
}

struct ScanShape {
    int64_t L, D, ldx, ldg, lddg;
    float c;
    int rows;             // batch
};

// ---- the tiles of a CTA.  All rows and channel tiles of a chunk come before
// the next chunk's, by ticket: a CTA that waits for a chunk before its own
// waits for one that has been taken before, and that is being worked on or
// comes first among what its CTA has taken.
struct Tile {
    int c, tile, b;              // chunk in scan order (-1: no more), channel tile, row
    unsigned starts[16];         // per warp: its tokens that start a document
    float rate[kTileCh];         // c softplus(lam)
};

constexpr int kMostTensors = 4, kMostOut = 3;
struct Inputs {
    const void *p[kMostTensors];   // x, r_raw, g_raw, dy
    int64_t ld[kMostTensors];
};
struct Maps {
    CUtensorMap m[kMostTensors], out[kMostOut];   // boxes of a CTA's tokens in, of a warp's out
};

// kTensors x kTokens rows of 64 channels per stage.  Tile `it` of the CTA is
// described in tiles[it % 4] and lands in stage it % kStages.
template <typename T, Source kSource, int kTensors, int kTokens, int kWarps, int kStages> struct Ring {
    static constexpr uint32_t kRow = kTileCh * sizeof(T) + (kSource == kOdd ? 4 : 0), kPart = kTokens * kRow;
    static constexpr int kPitch = kRow / sizeof(T);
    static constexpr uint32_t kStage = kTensors * kPart;
    static constexpr int kSeg = kTokens / kWarps;
    static constexpr size_t kBytes = 128 + kStages * kStage + 4 * sizeof(Tile) + kStages * 8 + 16;
    unsigned char *data;
    Tile *tiles;
    uint64_t *full;
    volatile int *abort;
    __device__ __forceinline__ explicit Ring(unsigned char *raw) {
        data = raw + (-tc::smem_u32(raw) & 127u);
        full = reinterpret_cast<uint64_t *>(data + kStages * kStage);
        tiles = reinterpret_cast<Tile *>(full + kStages);
        abort = reinterpret_cast<volatile int *>(tiles + 4);
    }
    __device__ __forceinline__ T *row(int stage, int tensor, int token) const {
        return reinterpret_cast<T *>(data + stage * kStage + tensor * kPart + token * kRow);
    }

    // The ticket of the CTA's tile `it` (last warp).
    __device__ __forceinline__ unsigned draw(const Handoff &w, int it) const {
        if (w.chunks == 1) return blockIdx.x + (unsigned)it * gridDim.x;
        return (threadIdx.x & 31) == 0 ? atomicAdd(w.ticket, 1u) : 0u;
    }

    // Describes tile `it` from its ticket (last warp), but for its rates, whose
    // lam it loads.  kBack: chunks are taken from the last to the first.
    template <bool kBack>
    __device__ __forceinline__ float2 describe(int it, unsigned taken, const Handoff &w, const ScanShape &s, const float *lam,
                                               const int32_t *ids) const {
        const int lane = threadIdx.x & 31;
        taken = __shfl_sync(0xffffffffu, taken, 0);
        Tile &t = tiles[it % 4];
        const unsigned plane = (unsigned)s.rows * (unsigned)w.tiles, total = plane * (unsigned)w.chunks;
        if (taken >= total) {
            if (lane == 0) t.c = -1;
            return make_float2(0.0f, 0.0f);
        }
        const int c = (int)(taken / plane);
        const unsigned r = taken - (unsigned)c * plane;
        const int b = (int)(r / (unsigned)w.tiles), tile = (int)(r - (unsigned)b * (unsigned)w.tiles);
        const int64_t t0 = (int64_t)(kBack ? w.chunks - 1 - c : c) * kTokens, d0 = (int64_t)tile * kTileCh;
        float l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t d = d0 + lane + 32 * i;
            l[i] = d < s.D ? lam[d] : -INFINITY;   // past the last channel: nothing decays
        }
#pragma unroll
        for (int j = 0; ids && j < kTokens / 32; ++j) {
            const int64_t at = t0 + j * 32 + lane;
            bool start = false;
            if (at > 0 && at < s.L) start = ids[(int64_t)b * s.L + at] != ids[(int64_t)b * s.L + at - 1];
            const unsigned word = __ballot_sync(0xffffffffu, start);
            if (lane < 32 / kSeg) t.starts[j * (32 / kSeg) + lane] = word >> (lane * kSeg) & ((1u << kSeg) - 1u);
        }
        if (lane == 0) {
            t.c = c;
            t.tile = tile;
            t.b = b;
        }
        return make_float2(l[0], l[1]);
    }
    // The rest of the description.
    __device__ __forceinline__ void rates(int it, float2 l, const ScanShape &s) const {
        const int lane = threadIdx.x & 31;
        Tile &t = tiles[it % 4];
        t.rate[lane] = s.c * softplus_f(l.x);
        t.rate[lane + 32] = s.c * softplus_f(l.y);
    }

    // Starts the copies of tensors kFirst .. kLast - 1 of tile `it` into stage st,
    // which nobody reads any more (all warps).
    template <bool kBack, int kFirst, int kLast>
    __device__ __forceinline__ void copy(int it, int st, const Inputs &in, const Maps &maps, const Handoff &w, const ScanShape &s) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (kSource == kTma && warp != kWarps - 1) return;
        const Tile &t = tiles[it % 4];
        if (t.c < 0) return;
        const int64_t t0 = (int64_t)(kBack ? w.chunks - 1 - t.c : t.c) * kTokens, row0 = (int64_t)t.b * s.L + t0;
        const int64_t d0 = (int64_t)t.tile * kTileCh;
        if (kSource == kTma) {
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&full[st], (kLast - kFirst) * kPart);
#pragma unroll
                for (int k = kFirst; k < kLast; ++k)
                    tc::tma_load_3d(data + st * kStage + k * kPart, &maps.m[k], &full[st], (int)d0, (int)t0, t.b);
            }
            return;
        }
        // the warp's own rows, one 4-byte copy a lane: half a row of fp32, a row
        // of bf16 pairs; zeros past the last channel
        constexpr int kPer = kTileCh * sizeof(T) / 128, kElems = 4 / sizeof(T);
        const int64_t left = s.L - t0 - warp * kSeg;
        const int n = left < 0 ? 0 : left < kSeg ? (int)left : kSeg;
        if (kSource == kOdd && n > 0) {
            const int here = (int)(s.D - d0 < kTileCh ? s.D - d0 : kTileCh);
#pragma unroll
            for (int k = kFirst; k < kLast; ++k) {
                // row r starts in the lower or upper half of a word, all alike or by turns; the
                // words from there on, none that holds nothing of the row
                const T *src = static_cast<const T *>(in.p[k]) + (row0 + warp * kSeg) * in.ld[k] + d0;
                const unsigned first = (unsigned)(reinterpret_cast<uintptr_t>(src) >> 1) & 1u, turn = (unsigned)in.ld[k] & 1u;
                const uint32_t dst = tc::smem_u32(data + st * kStage + k * kPart + warp * kSeg * kRow);
                const T *from = src + (2 * lane - 1 < here ? 2 * lane : 0);
                const uint32_t even = 2 * lane < here ? 4 : 0, odd = 2 * lane - 1 < here ? 4 : 0;
#pragma unroll
                for (int r = 0; r < kSeg; ++r) {
                    if (r >= n) break;
                    const unsigned half = first ^ (r & turn);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + r * kRow + lane * 4), "l"(from - half),
                                 "r"(half ? odd : even)
                                 : "memory");
                    from += in.ld[k];
                }
                // the last element of a row that starts in an upper half has a word of its own: lane r, row r
                if (here == kTileCh && lane < n && (first ^ (lane & turn)))
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + lane * kRow + kTileCh * 2),
                                 "l"(src + lane * in.ld[k] + kTileCh - 1)
                                 : "memory");
            }
        } else if (n > 0) {
#pragma unroll
            for (int k = kFirst; k < kLast; ++k) {
                const T *from[kPer];
                uint32_t size[kPer];
#pragma unroll
                for (int h = 0; h < kPer; ++h) {
                    const int e = (h * 32 + lane) * kElems;
                    const bool there = d0 + e < s.D;
                    from[h] = static_cast<const T *>(in.p[k]) + (row0 + warp * kSeg) * in.ld[k] + d0 + (there ? e : 0);
                    size[h] = there ? 4 : 0;
                }
                const uint32_t dst = tc::smem_u32(data + st * kStage + k * kPart + warp * kSeg * kRow) + lane * 4;
#pragma unroll
                for (int r = 0; r < kSeg; ++r) {
                    if (r >= n) break;
#pragma unroll
                    for (int h = 0; h < kPer; ++h) {
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + r * kRow + h * 128), "l"(from[h]),
                                     "r"(size[h])
                                     : "memory");
                        from[h] += in.ld[k];
                    }
                }
            }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&full[st])) : "memory");
    }

    // Before the first tile: barriers, three tiles described, two on their way.
    // Returns the ticket of the fourth (last warp).
    template <bool kBack>
    __device__ __forceinline__ unsigned start(const Inputs &in, const Maps &maps, const Handoff &w, const ScanShape &s,
                                              const float *lam, const int32_t *ids) const {
        unsigned next = 0;
        if (threadIdx.x == 32 * (kWarps - 1)) {
            for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[i], (kSource == kTma ? 1 : 32 * kWarps) * (kBack ? 1 : 2));
            *abort = 0;
            tc::fence_mbar_init();
        }
        auto copies = [&](int it) {
            copy<kBack, 0, kBack ? kTensors : 1>(it, it, in, maps, w, s);
            if (!kBack) copy<kBack, 1, kTensors>(it, it, in, maps, w, s);
        };
        if (threadIdx.x >> 5 == kWarps - 1) {
            // one ticket after the other: the tiles that the CTAs work on at a time
            // are then neighbours, and neighbours wait for one another (two at once doubled
            // the time of 64k x 1024)
            const float2 l0 = describe<kBack>(0, draw(w, 0), w, s, lam, ids);
            __syncwarp();
            if (kSource == kTma) copies(0);
            const float2 l1 = describe<kBack>(1, draw(w, 1), w, s, lam, ids);
            __syncwarp();
            if (kSource == kTma) copy<kBack, kBack ? 0 : 1, kTensors>(1, 1, in, maps, w, s);
            rates(0, l0, s);
            rates(1, l1, s);
            rates(2, describe<kBack>(2, draw(w, 2), w, s, lam, ids), s);
            next = draw(w, 3);
        }
        __syncthreads();
        if (kSource != kTma) {
            copies(0);
            copy<kBack, kBack ? 0 : 1, kTensors>(1, 1, in, maps, w, s);
        }
        return next;
    }
    // Between the barriers of tile `it`.  Backward: the stage of the tile before
    // is free.  Forward, with two stages: the gates of this tile are read and
    // make room for the tile after next, x's place (where y leaves from) is free
    // in the tile before.
    template <bool kBack>
    __device__ __forceinline__ float2 ahead(int it, int st, unsigned &next, const Inputs &in, const Maps &maps, const Handoff &w,
                                          const ScanShape &s, const float *lam, const int32_t *ids) const {
        if (kBack) {
            copy<kBack, 0, kTensors>(it + 2, st == 0 ? 2 : st - 1, in, maps, w, s);
        } else {
            copy<kBack, 0, 1>(it + 1, st ^ 1, in, maps, w, s);
            copy<kBack, 1, kTensors>(it + 2, st, in, maps, w, s);
        }
        float2 l = make_float2(0.0f, 0.0f);
        if (threadIdx.x >> 5 == kWarps - 1) {
            l = describe<kBack>(it + 3, next, w, s, lam, ids);
            next = draw(w, it + 4);
        }
        return l;   // for `rates`
    }
    // Waits for the tile in stage st; false: the wait gave up.
    __device__ __forceinline__ bool arrived(int st, uint32_t parity, long long budget) const {
        return tc::mbar_wait_abortable(&full[st], parity, budget, abort);
    }
};

// All warps meet; whether all of them say yes.
template <int kWarps> __device__ __forceinline__ bool all_warps(bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)yes), "n"(32 * kWarps)
        : "memory");
    return r != 0;
}
template <int kWarps> __device__ __forceinline__ void all_warps() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
}

// The end of a CTA: after a wait that gave up, let the copies in flight land
// (about a millisecond) before the shared memory goes away.
__device__ __forceinline__ void leave(volatile int *abort, unsigned *status) {
    __syncthreads();
    if (*abort) {
        if (threadIdx.x == 0) atomicOr(status, kStatusTimeout);
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 21)) {
        }
    }
}

// ---- forward
constexpr int kFwdCtas = 2;                                          // per SM
// (three stages of fp32 rows are 192 KB, of odd bf16 rows just above half an SM's)
template <typename T, Source kSource> constexpr int kBwdCtas = sizeof(T) == 2 && kSource != kOdd ? 2 : 1;
template <typename T, Source kSource> using FwdRing = Ring<T, kSource, 3, kFwdChunk<T>, kFwdWarps, 2>;
// the stage of a tile is read until its end, so three
template <typename T, Source kSource> using BwdRing = Ring<T, kSource, 4, kBwdChunk, kBwdWarps, 3>;

// kPacked: there are document ids (without them the kernel is smaller and spills less)
template <typename T, Source kSource, bool kPair, bool kPacked>
__global__ void __launch_bounds__(32 * kFwdWarps, kFwdCtas)
gated_scan_kernel(const __grid_constant__ Maps maps, Inputs src, const float *__restrict__ lam,
                  const float *__restrict__ init, const int32_t *__restrict__ ids, T *__restrict__ y,
                  float *__restrict__ fin, float *__restrict__ states, ScanShape s, Handoff w) {
    constexpr int kSeg = kFwdSeg<T>, kWarps = kFwdWarps;
    using R = FwdRing<T, kSource>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ ulonglong2 s_seg[2][kWarps][32], s_prev[kWarps][32];
    __shared__ f2 s_in[32];
    const R ring(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (w.chunks == 1 && blockIdx.x == 0 && threadIdx.x == 0) *w.status = 0;
    unsigned next = ring.template start<false>(src, maps, w, s, lam, ids);
    for (int it = 0;; ++it) {
        const int st = it & 1;
        const Tile &t = ring.tiles[it % 4];
        const int c = t.c, tile = t.tile, b = t.b;
        if (c < 0) break;
        const bool alive = ring.arrived(st, (uint32_t)(it >> 1) & 1u, w.budget);
        const int64_t d0 = (int64_t)tile * kTileCh + (kPair ? 2 * lane : lane), d1 = d0 + (kPair ? 1 : 32);
        const bool in0 = d0 < s.D, in1 = d1 < s.D;
        const int64_t t0 = (int64_t)c * kFwdChunk<T> + warp * kSeg, row0 = b * s.L;
        const int n = s.L <= t0 ? 0 : s.L - t0 < kSeg ? (int)(s.L - t0) : kSeg;
        const bool whole = n == kSeg;
        const unsigned starts = kPacked ? t.starts[warp] : 0u;
        const float k[2] = {t.rate[kPair ? 2 * lane : lane], t.rate[kPair ? 2 * lane + 1 : lane + 32]};

        // what token j's state is of the one entering this warp: A[j] h + H[j]
        f2 A[kSeg], H[kSeg];
        Segment seg;
        const T *px = ring.row(st, 0, warp * kSeg), *pr = ring.row(st, 1, warp * kSeg), *pg = ring.row(st, 2, warp * kSeg);
        const unsigned odd_x = odd_of(src.p[0], (row0 + t0) * s.ldx), odd_r = odd_of(src.p[1], (row0 + t0) * s.ldg),
                       odd_g = odd_of(src.p[2], (row0 + t0) * s.ldg);
        auto row_of = [&](const T *p, int j) {
            if (kSource != kOdd) return p + j * R::kPitch;
            return p + j * R::kPitch + (p == px ? odd_x ^ (j & (unsigned)s.ldx & 1u) : (p == pr ? odd_r : odd_g) ^ (j & (unsigned)s.ldg & 1u));
        };
        // (zeros past the last channel: what else lies in its word belongs to others)
        auto take = [&](const T *p, int j) {
            const f2 v = two_of<T, kPair>(row_of(p, j), lane);
            return kSource == kOdd ? two(in0 ? lo(v) : 0.0f, in1 ? hi(v) : 0.0f) : v;
        };
        // the common warp: all of its tokens there, every u near (a rate bounds its
        // u) and, seen on the way, no gate shut
        bool easy = whole && __all_sync(0xffffffffu, k[0] < kNear && k[1] < kNear);
        auto fold = [&](auto with_starts) {
            constexpr bool kStarts = decltype(with_starts)::value;
            const f2 one = two(1.0f), kk = two(k[0], k[1]);
            f2 a = one, h = two(0.0f);
            float least = 1.0f;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                const f2 er = mul(take(pr, j), two(-kLog2e));
                const f2 eg = mul(take(pg, j), two(-kLog2e));
                const f2 x = take(px, j);
                const f2 p = add(two(ex2(lo(er)), ex2(hi(er))), one), q = add(two(ex2(lo(eg)), ex2(hi(eg))), one);
                const f2 pq = mul(p, q), both = two(rcp(lo(pq)), rcp(hi(pq)));
                least = least_of(least, lo(both), hi(both));
                const f2 om = loss_near(mul(kk, mul(q, both))), z = less_square(om);
                const f2 in = mul(two(root(-lo(z)), root(-hi(z))), mul(mul(p, both), x));
                if (kStarts && (starts >> j & 1)) a = h = two(0.0f);
                H[j] = h = add(h, fma(om, h, in));
                A[j] = a = fma(om, a, a);
            }
            seg = Segment{kStarts ? two(-1.0f) : a, h};
            easy = __all_sync(0xffffffffu, least > kOpen);
        };
        if (easy) {
            if (kPacked && starts) fold(std::bool_constant<kPacked>{});
            else fold(std::false_type{});
        }
        if (!easy) {
            f2 a = two(1.0f), h = two(0.0f);
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (j < n) {
                    const f2 vr = take(pr, j);
                    const f2 vg = take(pg, j);
                    const f2 vx = take(px, j);
                    if (starts >> j & 1) a = h = two(0.0f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float r, g;
                        sigmoids_of(exp_of_gate(get(vr, i)), exp_of_gate(get(vg, i)), r, g);
                        const float u = k[i] * r, om = loss_of(u), hb = get(h, i);
                        put(h, i, __fadd_rn(hb, fmaf(om, hb, root(-less_square(om)) * (g * get(vx, i)))));
                        put(a, i, decay_of(om, u) * get(a, i));
                    }
                }
                A[j] = a;
                H[j] = h;
            }
            seg = Segment{starts ? two(-1.0f) : a, h};
        }
        ulonglong2 (*segs)[32] = s_seg[it & 1];
        segs[warp][lane] = packed(seg);
        if (kSource == kTma && lane == 0) tc::tma_store_wait_read();   // of the tile before
        if (!all_warps<kWarps>(alive && !*ring.abort)) break;
        const float2 l = ring.template ahead<false>(it, st, next, src, maps, w, s, lam, ids);

        // the segments of the CTA's own warps and of the chunks before, in order
        f2 h = two(0.0f);
        auto join = [&] {
            if (init && c < kGroup && (w.chunks == 1 || warp == kWarps - 2))
                h = two(in0 ? init[b * s.D + d0] : 0.0f, in1 ? init[b * s.D + d1] : 0.0f);
            if (w.chunks > 1) {
                if (warp == 0 && c + 1 < w.chunks && c % kGroup + 1 < kGroup) {
                    Segment all = segment_of(segs[0][lane]);
#pragma unroll
                    for (int j = 1; j < kWarps; ++j) all = joined<kPacked>(all, segment_of(segs[j][lane]));
                    hand_on(&w.seg[(((int64_t)b * w.chunks + c) * w.tiles + tile) * 32 + lane], all);
                }
                gather<kWarps, kPacked>(w, b, c, tile, h, s_prev, s_in, ring.abort);
                if (warp == kWarps - 1) ring.rates(it + 3, l, s);
                all_warps<kWarps>();
                h = entering<kPacked>(c, s_prev, s_in);
            } else if (warp == kWarps - 1) {
                ring.rates(it + 3, l, s);
            }
#pragma unroll
            for (int j = 0; j < kWarps - 1; ++j) {
                if (j == warp) break;
                h = after<kPacked>(segment_of(segs[j][lane]), h);
            }
            if (w.chunks > 1 && warp == kWarps - 1 && c + 1 < w.chunks && c % kGroup + 1 == kGroup)
                hand_on(&w.state[(((int64_t)b * w.groups + c / kGroup) * w.tiles + tile) * 32 + lane],
                        Segment{two(1.0f), after<kPacked>(seg, h)});
        };
        join();

        // y takes x's place in shared memory on its way out
        T *py = y + (row0 + t0) * s.D + (int64_t)tile * kTileCh, *sy = ring.row(st, 0, warp * kSeg);
        const f2 h_in = h;
        f2 now = h_in;
        if (whole && starts == 0) {
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                now = fma(A[j], h_in, H[j]);
                store_two<T, kSource, kPair>(sy + j * kTileCh, py + j * s.D, lane, now, in0, in1);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kSeg; ++j)
                if (j < n) {
                    now = starts & ((2u << j) - 1u) ? H[j] : fma(A[j], h_in, H[j]);
                    store_two<T, kSource, kPair>(sy + j * kTileCh, py + j * s.D, lane, now, in0, in1);
                }
        }
        if (kSource == kTma) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
                tc::tma_store_3d(&maps.out[0], sy, tile * kTileCh, (int)t0, b);
                tc::tma_store_commit();
            }
        }
        if (n > 0) {
            const int64_t end = t0 + n;   // one past this warp's last token
            if (states && (end % kGatedChunk == 0 || end == s.L)) {
                float *o = states + (b * ((s.L + kGatedChunk - 1) / kGatedChunk) + (end - 1) / kGatedChunk) * s.D;
                if (in0) o[d0] = lo(now);
                if (in1) o[d1] = hi(now);
            }
            if (fin && end == s.L) {
                if (in0) fin[b * s.D + d0] = lo(now);
                if (in1) fin[b * s.D + d1] = hi(now);
            }
        }
    }
    if (kSource == kTma && lane == 0) tc::tma_store_wait_read();   // the last tile's, before the shared memory goes
    leave(ring.abort, w.status);
}

// ---- backward: chunks of 64 tokens from the last to the first.  The states
// inside a chunk come from the one entering it (the forward's chunk states);
// the gradient's recurrence runs the other way over the same decays:
//   dh_t = dy_t + c_{t+1},   c_t = a_t dh_t (nothing past a document start)
//   dx = dh beta g,  dg_raw = dh beta x g (1 - g)
//   p = dh (u a h_{t-1} - u a^2/beta g x)      (u times d/d log a)
//   dr_raw = -(1 - r) p,  dlam = -sigmoid(lam)/softplus(lam) sum p
// (u/beta stays finite where the gate shuts and beta goes to 0.)
template <typename T, Source kSource, bool kPair, bool kPacked>
__global__ void __launch_bounds__(32 * kBwdWarps, kBwdCtas<T, kSource>)
gated_bwd_kernel(const __grid_constant__ Maps maps, Inputs src, const float *__restrict__ lam,
                 const float *__restrict__ init, const int32_t *__restrict__ ids, const float *__restrict__ states,
                 const float *__restrict__ dfin, T *__restrict__ dx, T *__restrict__ dr, T *__restrict__ dg,
                 float *__restrict__ part, float *__restrict__ dinit, ScanShape s, Handoff w) {
    constexpr int kSeg = kBwdSeg, kWarps = kBwdWarps;
    using R = BwdRing<T, kSource>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ ulonglong2 s_fwd[kWarps][32], s_rev[kWarps][32], s_prev[kWarps][32];
    __shared__ f2 s_in[32], s_sum[kWarps][32];
    const R ring(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (w.chunks == 1 && blockIdx.x == 0 && threadIdx.x == 0) *w.status = 0;
    unsigned next = ring.template start<true>(src, maps, w, s, lam, ids);
    // the sums of p of the tile before, which wait in s_sum until all warps meet
    float *sums = nullptr;
    bool sum0 = false, sum1 = false;
    auto store_sums = [&] {
        if (warp != kWarps / 2 || !sums) return;
        f2 v = s_sum[0][lane];
#pragma unroll
        for (int j = 1; j < kWarps; ++j) v = add(v, s_sum[j][lane]);
        if (sum0) sums[0] = -lo(v);
        if (sum1) sums[kPair ? 1 : 32] = -hi(v);
    };
    int st = 0;
    uint32_t parity = 0;
    for (int it = 0;; ++it) {
        const Tile &t = ring.tiles[it % 4];
        const int back = t.c, tile = t.tile, b = t.b;
        if (back < 0) break;
        const bool alive = ring.arrived(st, parity, w.budget);
        const int c = w.chunks - 1 - back;
        const int64_t d0 = (int64_t)tile * kTileCh + (kPair ? 2 * lane : lane), d1 = d0 + (kPair ? 1 : 32);
        const bool in0 = d0 < s.D, in1 = d1 < s.D;
        const int64_t t0 = (int64_t)c * kBwdChunk + warp * kSeg, row0 = b * s.L;
        const int n = s.L <= t0 ? 0 : s.L - t0 < kSeg ? (int)(s.L - t0) : kSeg;
        const bool whole = n == kSeg;
        const unsigned starts = kPacked ? t.starts[warp] : 0u;
        const float k[2] = {t.rate[kPair ? 2 * lane : lane], t.rate[kPair ? 2 * lane + 1 : lane + 32]};
        const float *from = c > 0 ? states + ((int64_t)b * w.chunks + c - 1) * s.D : init ? init + b * s.D : nullptr;
        f2 hh = two(from && in0 ? from[d0] : 0.0f, from && in1 ? from[d1] : 0.0f);
        const T *px = ring.row(st, 0, warp * kSeg), *pr = ring.row(st, 1, warp * kSeg), *pg = ring.row(st, 2, warp * kSeg);
        const T *py = ring.row(st, 3, warp * kSeg);
        const int64_t at = row0 + t0, dt = (int64_t)tile * kTileCh;
        const unsigned odd_x = odd_of(src.p[0], at * s.ldx), odd_r = odd_of(src.p[1], at * s.ldg), odd_g = odd_of(src.p[2], at * s.ldg),
                       odd_y = odd_of(src.p[3], at * s.D);
        auto row_of = [&](const T *p, int j) {
            if (kSource != kOdd) return p + j * R::kPitch;
            const unsigned first = p == px ? odd_x : p == pr ? odd_r : p == pg ? odd_g : odd_y;
            return p + j * R::kPitch + (first ^ (j & (unsigned)(p == px ? s.ldx : p == py ? s.D : s.ldg) & 1u));
        };
        // (zeros past the last channel: what else lies in its word belongs to others)
        auto take = [&](const T *p, int j) {
            const f2 v = two_of<T, kPair>(row_of(p, j), lane);
            return kSource == kOdd ? two(in0 ? lo(v) : 0.0f, in1 ? hi(v) : 0.0f) : v;
        };

        // per token -r, a - 1 and beta g; the state this warp makes of 0, and the
        // same products from the last token to the first.  g waits in shared memory
        // where the lane's gates were: 128 registers have no room for it.
        T *sr = ring.row(st, 1, warp * kSeg), *sg = ring.row(st, 2, warp * kSeg);
        f2 nr[kSeg], om[kSeg], bg[kSeg];
        auto keep_g = [&](int j, f2 v) {
            if constexpr (sizeof(T) == 4 && kPair) {
                reinterpret_cast<f2 *>(sr + j * R::kPitch)[lane] = v;
            } else {
                reinterpret_cast<float *>(sr + j * R::kPitch)[lane] = lo(v);
                reinterpret_cast<float *>((sizeof(T) == 4 ? sr + 32 : sg) + j * R::kPitch)[lane] = hi(v);
            }
        };
        auto kept_g = [&](int j) -> f2 {
            if constexpr (sizeof(T) == 4 && kPair) return reinterpret_cast<const f2 *>(sr + j * R::kPitch)[lane];
            else
                return two(reinterpret_cast<const float *>(sr + j * R::kPitch)[lane],
                           reinterpret_cast<const float *>((sizeof(T) == 4 ? sr + 32 : sg) + j * R::kPitch)[lane]);
        };
        Segment seg, rev;
        bool easy = whole && __all_sync(0xffffffffu, k[0] < kNear && k[1] < kNear);
        const f2 one = two(1.0f), nk = two(-k[0], -k[1]);
        if (easy) {
            f2 g[kSeg];
            float least = 1.0f;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                const f2 er = mul(take(pr, j), two(-kLog2e));
                const f2 eg = mul(take(pg, j), two(-kLog2e));
                const f2 p = add(two(ex2(lo(er)), ex2(hi(er))), one);
                const f2 nq = fma(two(ex2(lo(eg)), ex2(hi(eg))), two(-1.0f), two(-1.0f));
                const f2 pq = mul(p, nq), both = two(rcp(-lo(pq)), rcp(-hi(pq)));
                least = least_of(least, lo(both), hi(both));
                nr[j] = mul(nq, both);
                g[j] = mul(p, both);
            }
            easy = __all_sync(0xffffffffu, least > kOpen);
            auto fold = [&](auto with_starts) {
                constexpr bool kStarts = decltype(with_starts)::value;
                f2 a = one, sh = two(0.0f), rh = two(0.0f);
#pragma unroll
                for (int j = 0; j < kSeg; ++j) {
                    keep_g(j, g[j]);
                    om[j] = loss_near(mul(nk, nr[j]));
                    const f2 z = less_square(om[j]);
                    bg[j] = mul(two(root(-lo(z)), root(-hi(z))), g[j]);
                    if (kStarts && (starts >> j & 1)) sh = two(0.0f);
                    sh = add(sh, fma(om[j], sh, mul(bg[j], take(px, j))));
                    a = fma(om[j], a, a);
                }
#pragma unroll
                for (int j = kSeg - 1; j >= 0; --j) {
                    const f2 dh = add(take(py, j), rh);
                    rh = kStarts && (starts >> j & 1) ? two(0.0f) : fma(om[j], dh, dh);
                }
                if (kStarts) a = two(-1.0f);
                seg = Segment{a, sh};
                rev = Segment{a, rh};
            };
            if (easy) {
                if (kPacked && starts) fold(std::bool_constant<kPacked>{});
                else fold(std::false_type{});
            }
        }
        if (!easy) {
            float sum[2] = {0.0f, 0.0f};
            f2 sh = two(0.0f), rh = two(0.0f);
#pragma unroll
            for (int j = 0; j < kSeg; ++j)
                if (j < n) {
                    const f2 vr = take(pr, j);
                    const f2 vg = take(pg, j);
                    const f2 vx = take(px, j);
                    if (starts >> j & 1) sh = two(0.0f);
                    f2 g = 0;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float r1, g1;
                        sigmoids_of(exp_of_gate(get(vr, i)), exp_of_gate(get(vg, i)), r1, g1);
                        const float u = k[i] * r1, o = loss_of(u), b1 = root(-less_square(o)) * g1, hb = get(sh, i);
                        sum[i] = __fadd_rn(sum[i], u);
                        put(nr[j], i, -r1);
                        put(g, i, g1);
                        put(om[j], i, o);
                        put(bg[j], i, b1);
                        put(sh, i, __fadd_rn(hb, fmaf(o, hb, b1 * get(vx, i))));
                    }
                    if (kSource == kOdd) __syncwarp();   // lanes' places for g are others' raw gates here
                    keep_g(j, g);
                }
#pragma unroll
            for (int j = kSeg - 1; j >= 0; --j)
                if (j < n) {
                    const f2 dh = add(take(py, j), rh);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        put(rh, i, starts >> j & 1 ? 0.0f : decay_of(get(om[j], i), -k[i] * get(nr[j], i)) * get(dh, i));
                }
            const f2 a = starts ? two(-1.0f) : two(ex2_whole(-sum[0] * kLog2e), ex2_whole(-sum[1] * kLog2e));
            seg = Segment{a, sh};
            rev = Segment{a, rh};
        }
        s_fwd[warp][lane] = packed(seg);
        s_rev[warp][lane] = packed(rev);
        if (kSource == kTma && lane == 0) tc::tma_store_wait_read();   // of the tile before
        if (!all_warps<kWarps>(alive && !*ring.abort)) break;
        const float2 l = ring.template ahead<true>(it, st, next, src, maps, w, s, lam, ids);

        // the state entering this warp, and the gradient from the warps and chunks
        // after it
        f2 cc = two(0.0f);
        auto join = [&] {
            if (warp == 0 && back + 1 < w.chunks && back % kGroup + 1 < kGroup) {
                Segment all = segment_of(s_rev[kWarps - 1][lane]);
#pragma unroll
                for (int j = kWarps - 2; j >= 0; --j) all = joined<kPacked>(all, segment_of(s_rev[j][lane]));
                hand_on(&w.seg[(((int64_t)b * w.chunks + back) * w.tiles + tile) * 32 + lane], all);
            }
            if (dfin && back < kGroup && warp == kWarps - 2)
                cc = two(in0 ? dfin[b * s.D + d0] : 0.0f, in1 ? dfin[b * s.D + d1] : 0.0f);
            gather<kWarps, kPacked>(w, b, back, tile, cc, s_prev, s_in, ring.abort);
            store_sums();
#pragma unroll
            for (int j = 0; j < kWarps - 1; ++j) {
                if (j == warp) break;
                hh = after<kPacked>(segment_of(s_fwd[j][lane]), hh);
            }
            Segment later = {two(1.0f), two(0.0f)};
#pragma unroll
            for (int j = kWarps - 1; j > 0; --j) {
                if (j == warp) break;
                later = joined<kPacked>(later, segment_of(s_rev[j][lane]));
            }
            if (warp == kWarps - 1) ring.rates(it + 3, l, s);
            all_warps<kWarps>();
            cc = after<kPacked>(later, entering<kPacked>(back, s_prev, s_in));
            if (warp == 0 && back + 1 < w.chunks && back % kGroup + 1 == kGroup)
                hand_on(&w.state[(((int64_t)b * w.groups + back / kGroup) * w.tiles + tile) * 32 + lane],
                        Segment{two(1.0f), after<kPacked>(rev, cc)});
        };
        join();

        T *ox = dx + at * s.D + dt, *orr = dr + at * s.lddg + dt, *og = dg + at * s.lddg + dt;
        // the gradients take the inputs' places in shared memory on their way out
        T *sx = ring.row(st, 0, warp * kSeg);
        f2 prev[kSeg], total = two(0.0f);   // total: of -p
        auto finish = [&](auto with_starts) {
            constexpr bool kStarts = decltype(with_starts)::value;
#pragma unroll
            for (int j = 0; j < kSeg; ++j) {
                if (kStarts && (starts >> j & 1)) hh = two(0.0f);
                prev[j] = hh;
                hh = add(hh, fma(om[j], hh, mul(bg[j], take(px, j))));
            }
#pragma unroll
            for (int j = kSeg - 1; j >= 0; --j) {
                const f2 in = mul(bg[j], take(px, j));
                const f2 dh = add(take(py, j), cc);
                const f2 g = kept_g(j);   // before dr takes its place
                const f2 nu = mul(two(k[0], k[1]), nr[j]);
                cc = kStarts && (starts >> j & 1) ? two(0.0f) : fma(om[j], dh, dh);
                const f2 din = mul(dh, in);
                // -p / dh = u a^2/(1 - a^2) in - u a h_{t-1}
                const f2 f = input_slope_near(mul(nk, nr[j]));
                const f2 np = mul(fma(mul(nu, add(om[j], one)), prev[j], mul(f, in)), dh);
                total = add(total, np);
                store_two<T, kSource, kPair>(sx + j * kTileCh, ox + j * s.D, lane, mul(dh, bg[j]), in0, in1);
                store_two<T, kSource, kPair>(sr + j * kTileCh, orr + j * s.lddg, lane, fma(nr[j], np, np), in0, in1);
                store_two<T, kSource, kPair>(sg + j * kTileCh, og + j * s.lddg, lane, fma(mul(g, two(-1.0f)), din, din), in0, in1);
            }
        };
        if (easy) {
            if (kPacked && starts) finish(std::bool_constant<kPacked>{});
            else finish(std::false_type{});
        } else {
#pragma unroll
            for (int j = 0; j < kSeg; ++j)
                if (j < n) {
                    if (starts >> j & 1) hh = two(0.0f);
                    prev[j] = hh;
                    hh = add(hh, fma(om[j], hh, mul(bg[j], take(px, j))));
                }
#pragma unroll
            for (int j = kSeg - 1; j >= 0; --j)
                if (j < n) {
                    const f2 in = mul(bg[j], take(px, j));
                    const f2 dh = add(take(py, j), cc);
                    const f2 g = kept_g(j);
                    f2 vr = 0, vg = 0;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float r1 = -get(nr[j], i), u = k[i] * r1, o = get(om[j], i), a = decay_of(o, u), d1 = get(dh, i);
                        const float ua = a == 0.0f ? 0.0f : u * a;   // (u may be infinite)
                        const float np = d1 * fmaf(-ua, get(prev[j], i), input_slope(u, o) * get(in, i));
                        put(total, i, __fadd_rn(get(total, i), np));
                        put(vr, i, fmaf(-r1, np, np));
                        put(vg, i, d1 * get(in, i) * __fsub_rn(1.0f, get(g, i)));
                        put(cc, i, starts >> j & 1 ? 0.0f : a * d1);
                    }
                    store_two<T, kSource, kPair>(sx + j * kTileCh, ox + j * s.D, lane, mul(dh, bg[j]), in0, in1);
                    store_two<T, kSource, kPair>(sr + j * kTileCh, orr + j * s.lddg, lane, vr, in0, in1);
                    store_two<T, kSource, kPair>(sg + j * kTileCh, og + j * s.lddg, lane, vg, in0, in1);
                }
        }
        if (kSource == kTma) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n > 0) {
                tc::tma_store_3d(&maps.out[0], sx, tile * kTileCh, (int)t0, b);
                tc::tma_store_3d(&maps.out[1], sr, tile * kTileCh, (int)t0, b);
                tc::tma_store_3d(&maps.out[2], sg, tile * kTileCh, (int)t0, b);
                tc::tma_store_commit();
            }
        }
        s_sum[warp][lane] = total;
        sums = part + ((int64_t)b * w.chunks + c) * s.D + d0;
        sum0 = in0;
        sum1 = in1;
        if (dinit && c == 0 && warp == 0) {
            if (in0) dinit[b * s.D + d0] = lo(cc);
            if (in1) dinit[b * s.D + d1] = hi(cc);
        }
        if (++st == 3) {
            st = 0;
            parity ^= 1u;
        }
    }
    if (kSource == kTma && lane == 0) tc::tma_store_wait_read();   // the last tile's, before the shared memory goes
    all_warps<kWarps>();
    store_sums();
    leave(ring.abort, w.status);
}

// ---- one token
template <typename T>
__global__ void __launch_bounds__(128)
gated_step_kernel(const T *__restrict__ x, const T *__restrict__ rr, const T *__restrict__ gr,
                  const float *__restrict__ lam, float *__restrict__ state, T *__restrict__ y, int64_t D, int64_t ldx,
                  int64_t ldg, float c) {
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (d >= D) return;
    float r, g;
    sigmoids_of(exp_of_gate(to_f(rr[b * ldg + d])), exp_of_gate(to_f(gr[b * ldg + d])), r, g);
    const float om = loss_of(c * softplus_f(lam[d]) * r);
    float h = state[b * D + d];
    h += fmaf(om, h, root(-less_square(om)) * (g * to_f(x[b * ldx + d])));
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

int64_t chunks_of(int64_t L, int in_dtype, int backward) {
    const int q = backward ? kBwdChunk : in_dtype == SSD_BF16 ? kFwdChunk<__nv_bfloat16> : kFwdChunk<float>;
    return (L + q - 1) / q;
}

// The workspace: status and ticket, the segments and states of the chunks
// (zeroed with them), and the backward's sums of p per chunk.
struct Regions {
    Handoff w;
    float *part;
    size_t zeroed, total;
};

Regions regions_of(void *workspace, int64_t b, int64_t L, int64_t D, int in_dtype, int backward) {
    Regions r = {};
    const int64_t chunks = chunks_of(L, in_dtype, backward), groups = (chunks + kGroup - 1) / kGroup;
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
    r.w.budget = wait_budget(kFaultGated);
    if (chunks > 1) {
        r.w.seg = reinterpret_cast<float4 *>(take((size_t)(b * chunks * tiles) * 32 * sizeof(float4)));
        r.w.state = reinterpret_cast<float4 *>(take((size_t)(b * groups * tiles) * 32 * sizeof(float4)));
        r.zeroed = at;
    }
    if (backward) r.part = reinterpret_cast<float *>(take((size_t)(b * chunks * D) * sizeof(float)));
    r.total = at;
    return r;
}

size_t workspace_bytes_of(int64_t b, int64_t L, int64_t D, int in_dtype, int backward) {
    return regions_of(nullptr, b, L, D, in_dtype, backward).total;
}

// Clears the hand-off before a call of several chunks.  (Under the test fault the
// tickets of the first chunk's tiles are given out to nobody.)
cudaError_t clear_handoff(const Regions &r, int64_t b, cudaStream_t s) {
    cudaError_t e = cudaMemsetAsync(r.w.status, 0, r.zeroed, s);
    if (e == cudaSuccess && test_fault(kFaultGated))
        e = cudaMemsetAsync(r.w.ticket, (int)(b * r.w.tiles < 255 ? b * r.w.tiles : 255), 1, s);
    return e;
}

struct FwdArgs {
    Inputs in;
    const float *lam, *init;
    const int32_t *ids;
    void *y;
    float *fin, *states;
};
struct GradArgs {
    const float *dfin;
    void *dx, *dr, *dg;
    float *part, *dinit;
};

// CTAs that run at once (per_sm of an SM), and the kernel's shared memory allowed, once per device.
template <auto kKern> cudaError_t slots_of(int per_sm, size_t smem, int *slots) {
    static int cached[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!cached[dev]) {
        if ((e = cudaFuncSetAttribute(kKern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess) return e;
        int sms = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        cached[dev] = sms * per_sm;
    }
    *slots = cached[dev];
    return cudaSuccess;
}

// The map of a tensor [rows, L, D] for TMA: false where it cannot be (rows not
// on 16 bytes, sizes beyond a map's).
template <typename T> bool map_of(CUtensorMap *map, const void *p, int64_t ld, const ScanShape &s, int tokens) {
    const uint64_t row = (uint64_t)ld * sizeof(T), all = row * (uint64_t)s.L;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) || row % 16 || all >= (1ull << 40)) return false;
    const uint64_t dims[3] = {(uint64_t)s.D, (uint64_t)s.L, (uint64_t)s.rows}, strides[2] = {row, all};
    const uint32_t box[3] = {(uint32_t)kTileCh, (uint32_t)tokens, 1};
    return tmap_encode_3d_plain(map, p, sizeof(T) == 2 ? kTmapBF16 : kTmapF32, dims, strides, box);
}

// Pairs of elements are aligned in every tensor (and D is even).
template <typename T>
bool pairs_of(const Inputs &in, int tensors, int64_t D, std::initializer_list<const void *> outs, int64_t ld_out) {
    if (D % 2 || ld_out % 2) return false;
    for (const void *p : outs)
        if (reinterpret_cast<uintptr_t>(p) % (2 * sizeof(T))) return false;
    for (int k = 0; k < tensors; ++k)
        if (reinterpret_cast<uintptr_t>(in.p[k]) % (2 * sizeof(T)) || in.ld[k] % 2) return false;
    return true;
}

template <typename T, Source kSource, bool kPair, bool kPacked>
cudaError_t scan_launch_of(const FwdArgs &a, const Maps &maps, const ScanShape &s, const Handoff &w, int64_t tiles, cudaStream_t st) {
    constexpr auto kern = &gated_scan_kernel<T, kSource, kPair, kPacked>;
    constexpr size_t smem = FwdRing<T, kSource>::kBytes;
    int slots = 0;
    const cudaError_t e = slots_of<kern>(kFwdCtas, smem, &slots);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(tiles < slots ? tiles : slots), 32 * kFwdWarps, smem, st>>>(
        maps, a.in, a.lam, a.init, a.ids, (T *)a.y, a.fin, a.states, s, w);
    return cudaGetLastError();
}

template <typename T, Source kSource, bool kPair>
cudaError_t scan_launch(const FwdArgs &a, const Maps &maps, const ScanShape &s, const Handoff &w, int64_t tiles, cudaStream_t st) {
    return a.ids ? scan_launch_of<T, kSource, kPair, true>(a, maps, s, w, tiles, st)
                 : scan_launch_of<T, kSource, kPair, false>(a, maps, s, w, tiles, st);
}

template <typename T> cudaError_t scan_of(const FwdArgs &a, const ScanShape &s, const Handoff &w, cudaStream_t st) {
    const int64_t tiles = (int64_t)s.rows * w.chunks * w.tiles;
    const bool pair = pairs_of<T>(a.in, 3, s.D, {a.y}, s.D);
    Maps maps;
    bool tma = pair && map_of<T>(&maps.out[0], a.y, s.D, s, kFwdSeg<T>);
    for (int i = 0; i < 3; ++i) tma = tma && map_of<T>(&maps.m[i], a.in.p[i], a.in.ld[i], s, kFwdChunk<T>);
    if (tma) return scan_launch<T, kTma, true>(a, maps, s, w, tiles, st);
    if (pair) return scan_launch<T, kAsync, true>(a, maps, s, w, tiles, st);
    if constexpr (sizeof(T) == 4) return scan_launch<T, kAsync, false>(a, maps, s, w, tiles, st);
    else return scan_launch<T, kOdd, false>(a, maps, s, w, tiles, st);
}

template <typename T, Source kSource, bool kPair, bool kPacked>
cudaError_t bwd_launch_of(const FwdArgs &a, const GradArgs &d, const Maps &maps, const ScanShape &s, const Handoff &w, int64_t tiles,
                       cudaStream_t st) {
    constexpr auto kern = &gated_bwd_kernel<T, kSource, kPair, kPacked>;
    constexpr size_t smem = BwdRing<T, kSource>::kBytes;
    int slots = 0;
    const cudaError_t e = slots_of<kern>(kBwdCtas<T, kSource>, smem, &slots);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(tiles < slots ? tiles : slots), 32 * kBwdWarps, smem, st>>>(
        maps, a.in, a.lam, a.init, a.ids, a.states, d.dfin, (T *)d.dx, (T *)d.dr, (T *)d.dg, d.part, d.dinit, s, w);
    return cudaGetLastError();
}

template <typename T, Source kSource, bool kPair>
cudaError_t bwd_launch(const FwdArgs &a, const GradArgs &d, const Maps &maps, const ScanShape &s, const Handoff &w, int64_t tiles,
                       cudaStream_t st) {
    return a.ids ? bwd_launch_of<T, kSource, kPair, true>(a, d, maps, s, w, tiles, st)
                 : bwd_launch_of<T, kSource, kPair, false>(a, d, maps, s, w, tiles, st);
}

template <typename T>
cudaError_t bwd_of(const FwdArgs &a, const GradArgs &d, const ScanShape &s, const Handoff &w, cudaStream_t st) {
    const int64_t tiles = (int64_t)s.rows * w.chunks * w.tiles;
    const bool pair = pairs_of<T>(a.in, 4, s.D, {d.dx, d.dr, d.dg}, s.lddg);
    Maps maps;
    const void *out[3] = {d.dx, d.dr, d.dg};
    bool tma = pair;
    for (int i = 0; i < 3; ++i) tma = tma && map_of<T>(&maps.out[i], out[i], i ? s.lddg : s.D, s, kBwdSeg);
    for (int i = 0; i < 4; ++i) tma = tma && map_of<T>(&maps.m[i], a.in.p[i], a.in.ld[i], s, kBwdChunk);
    if (tma) return bwd_launch<T, kTma, true>(a, d, maps, s, w, tiles, st);
    if (pair) return bwd_launch<T, kAsync, true>(a, d, maps, s, w, tiles, st);
    if constexpr (sizeof(T) == 4) return bwd_launch<T, kAsync, false>(a, d, maps, s, w, tiles, st);
    else return bwd_launch<T, kOdd, false>(a, d, maps, s, w, tiles, st);
}

}  // namespace
}  // namespace ssd

extern "C" {

SSD_API ssd_status ssd_gated_scan_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int in_dtype, int backward,
                                                 size_t *bytes) {
    if (!bytes || (backward != 0 && backward != 1)) return SSD_ERR_INVALID_ARG;
    const ssd_status st = ssd::check_sizes(batch, seqlen, dim, in_dtype);
    if (st == SSD_OK) *bytes = ssd::workspace_bytes_of(batch, seqlen, dim, in_dtype, backward);
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
    if (!workspace || workspace_bytes < ssd::workspace_bytes_of(batch, seqlen, dim, in_dtype, 0)) return SSD_ERR_WORKSPACE;
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
    const ssd::Regions r = ssd::regions_of(workspace, batch, seqlen, dim, in_dtype, 0);
    // with one chunk nothing is handed on, and the kernel clears the status itself
    if (r.w.chunks > 1 && (e = ssd::clear_handoff(r, batch, s)) != cudaSuccess)
        return (ssd_status)ssd::record_cuda_error(e);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedScan);
        const ssd::FwdArgs a = {{{x, r_raw, g_raw, nullptr}, {ld_x, ld_gate, ld_gate, 0}}, lam, init_state, seq_idx, y,
                                final_state, chunk_states};
        const ssd::ScanShape sh = {seqlen, dim, ld_x, ld_gate, 0, decay_scale, (int)batch};
        e = (in_dtype == SSD_BF16 ? ssd::scan_of<__nv_bfloat16> : ssd::scan_of<float>)(a, sh, r.w, s);
    }
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
    if (!workspace || workspace_bytes < ssd::workspace_bytes_of(batch, seqlen, dim, in_dtype, 1)) return SSD_ERR_WORKSPACE;
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
    const ssd::Regions r = ssd::regions_of(workspace, batch, seqlen, dim, in_dtype, 1);
    if (r.w.chunks > 1 && (e = ssd::clear_handoff(r, batch, s)) != cudaSuccess)
        return (ssd_status)ssd::record_cuda_error(e);
    {
        ssd::TraceScope tr(s, ssd::kTrGatedBwd);
        const ssd::FwdArgs a = {{{x, r_raw, g_raw, dy}, {ld_x, ld_gate, ld_gate, dim}}, lam, init_state, seq_idx, nullptr,
                                nullptr, const_cast<float *>(chunk_states)};
        const ssd::GradArgs d = {dfinal_state, dx, dr_raw, dg_raw, r.part, dinit_state};
        const ssd::ScanShape sh = {seqlen, dim, ld_x, ld_gate, ld_dgate, decay_scale, (int)batch};
        e = (in_dtype == SSD_BF16 ? ssd::bwd_of<__nv_bfloat16> : ssd::bwd_of<float>)(a, d, sh, r.w, s);
    }
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
