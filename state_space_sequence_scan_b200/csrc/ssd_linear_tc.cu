// The projections' products on the tensor cores (bf16 operands, or fp32 ones in
// three bf16 parts; fp32 accumulators in TMEM):  D[m, n] = sum_k A(m, k) B(n, k), with the epilogue
// of ssd_linear.h.  Either operand may run along k in memory ("K-major", the
// forward's x and W) or along its own rows ("MN-major": the backward's W, dz
// and x, which need no transposed copy).
//
// A pair of CTAs (a cluster of two, cta_group::2) owns a tile of 256 x BN:
// each loads 128 rows of A and BN/2 of B by TMA into a ring of stages of 64 k,
// one thread of the first CTA issues the MMAs of both (M = 256), and each CTA
// keeps 128 rows of the accumulator in its TMEM.  The pair halves what a tile
// reads of B: at 256 x 256 a CTA moves 32 KB per 128 x 256 x 64 products, and
// it is the L2 that would bound a tile of one CTA (48 KB).  The grid is
// persistent; accumulators are double-buffered, so the eight epilogue warps
// store a tile while the next one is multiplied.  Measured: 8192 x 5120 x 2560 in
// 138 to 145 us, 0.86 of the tensor pipe's cycles, 0.90 to 0.94 of the measured cuBLAS rate.
//
// fp32 operands (kTerms 6).  v = hi + mid + lo, each the nearest bf16 of what
// is left, which is all 24 bits of values from 2^-110 on (below, lo would need less
// than bf16's smallest number); of the nine products of two such sums the
// three smallest, together at most 2^-24 of the whole, are left out.  The tensor cores cut a
// sum's low bits at every step, so a sum is taken in segments of 512 k, its
// smallest products first, and the segments are added in float32 registers:
// 1024^3 then is 4.7e-7 off (relative, in the mean square), cuBLAS's float32
// product 5.7e-7; one segment of all k was 7e-6 off at K 6144.  Measured: 2048 x 2560 x
// 2560 in 190 us, 22 of them the split.  The segments cost the epilogue a read of the accumulator each,
// under the next one's products.
#include <cuda.h>

#include <initializer_list>

#include "ssd_internal.h"
#include "ssd_linear.h"
#include "ssd_tc.cuh"
#include "ssd_tmap.h"
#include "ssd_trace.h"

namespace ssd {
namespace {

using namespace tc;

constexpr int kLtM = 256;                      // rows of a pair's tile
constexpr int kLtK = 64;                       // k per stage: one 128-byte swizzle row
constexpr int kLtEpiWarps = 8;
constexpr int kLtTmaWarp = 8, kLtMmaWarp = 9;
constexpr int kLtThreads = 32 * 10;
// Stages of a segment.  The tensor cores cut a sum's low bits at every step of 16 k,
// so long sums are taken in segments, added in float32 registers: fp32 operands'
// always, in 512 k; those of bf16 products in up to 1024 k where the result is fp32
// (one of 8192 k was 9e-6 off in the mean square, 3.5e-5 with positive values, 32768 k
// 4e-5 and 2e-4; so 1e-6 and 2e-6, as float32 sums in order), and where it is bf16 from 65536 k on, when
// the cuts come near that rounding (a gradient over 1M rows was 0.0021 off, 0.0017
// being the store's).  8192 x 5120 x 2560 takes 140 us to fp32 in one, 168 in segments
// of 1024 and 206 of 512: the stores of a tile have to end under two segments of the next.
constexpr int kLtSegParts = 8, kLtSegBf16 = 16;
constexpr int64_t kLtLongK = 65536;
constexpr int kLtGroupM = 8;                   // row tiles walked together: what a wave reads stays in L2

template <int BN> struct LtStages { static constexpr int value = BN >= 192 ? 6 : BN == 160 ? 7 : 8; };
// TMEM columns of both accumulators: a power of two
template <int BN> constexpr int lt_columns() { return BN <= 64 ? 128 : BN <= 128 ? 256 : 512; }
constexpr uint32_t kLtABytes = 128 * kLtK * 2;
template <int BN> constexpr uint32_t lt_b_bytes() { return (BN / 2) * kLtK * 2; }
template <int BN> constexpr size_t lt_smem() {
    return 1024 + (size_t)LtStages<BN>::value * (kLtABytes + lt_b_bytes<BN>()) + 256 + kLtEpiWarps * 32 * 33 * 4;
}

struct LtShape {
    int M, N, ksteps;          // ksteps: stages of the whole k
    int mt, nt, splits, per;   // tiles, parts of k, stages of a part
    float *part;               // [splits, M, N] fp32 sums when splits > 1
    int out_f32, vec;          // vec: rows of out start on 16 bytes
    int clear;                 // the status word is this launch's to clear
    int seg, planeA, planeB;   // kSegs: stages of a segment; kTerms 2 and 6: rows between the parts of an operand
    int fault;                 // the test fault: arrivals on the first stage that never come (1)
    long long budget;          // clock cycles before a wait gives up
};

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// 2-D tiled load whose completion is counted on a barrier of either CTA of the pair
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const void *tmap, uint32_t cluster_bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(cluster_bar)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued before have completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// One thread of a converged warp.  The compiler knows that it is one, and issues
// tcgen05 and TMA instructions straight from uniform registers; under a test of
// the lane number it loops over the threads that might be there, and a step of
// 64 k cost 556 cycles instead of 287 (256 x 128 tiles).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
// As mbar_wait_abortable, with acquire over the cluster (the other CTA's arrivals).
__device__ __forceinline__ bool wait_cluster(uint64_t *bar, uint32_t parity, long long budget, volatile int *abort) {
    if (try_wait_cluster(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
        if (try_wait_cluster(bar, parity)) return true;
        if (*abort) return false;
        if (clock64() - t0 > budget) {
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void tile_of(int t, const LtShape &s, int &split, int &mi, int &ni) {
    const int plane = s.mt * s.nt;
    split = t / plane;
    const int r = t - split * plane, group = r / (kLtGroupM * s.nt);
    const int first = group * kLtGroupM, gm = min(s.mt - first, kLtGroupM), rr = r - group * kLtGroupM * s.nt;
    mi = first + rr % gm;
    ni = rr / gm;
}

__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's 32 x 32 values, lane r holding row r, leave through shared memory so
// that a store covers whole pieces of rows: 8 rows of 64 bytes (bf16) or 4 of
// 128 (fp32) where rows start on 16 bytes, else one row.  (Each lane storing
// its own row made an unaligned 2560 x 5118 gradient 8 times slower.)
constexpr int kLtPitch = 33;

template <typename T, int kN> __device__ __forceinline__ void get_vec(const T *p, float (&v)[kN]);
template <> __device__ __forceinline__ void get_vec<float, 4>(const float *p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
template <> __device__ __forceinline__ void get_vec<__nv_bfloat16, 8>(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo(w[i]);
        v[2 * i + 1] = bf16hi(w[i]);
    }
}
__device__ __forceinline__ void put_vec(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <int kN> __device__ __forceinline__ void put_vec(__nv_bfloat16 *p, const float (&v)[kN]) {
    uint32_t w[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) w[i] = pack_bf2(v[2 * i], v[2 * i + 1]);
    if constexpr (kN == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// rows m .. m + 31, columns n .. n + 31, those there are: bias, activation, residual, store
template <typename TO, bool kPart>
__device__ __forceinline__ void store_block(const float *v, int64_t m, int n, const LinearEpilogue &ep, const LtShape &s, float *part,
                                            int lane) {
    TO *out = kPart ? reinterpret_cast<TO *>(part) : static_cast<TO *>(ep.out);
    const TO *res = static_cast<const TO *>(ep.residual);
    // the operands' type: bf16, or fp32 (then TO is too)
    __nv_bfloat16 *pre = ep.pre_f32 ? nullptr : static_cast<__nv_bfloat16 *>(ep.preact);
    float *pre32 = ep.pre_f32 ? static_cast<float *>(ep.preact) : nullptr;
    const int rows = s.M - m < 32 ? (int)(s.M - m) : 32;
    if (s.vec && s.N - n >= 32) {
        constexpr int kN = 16 / sizeof(TO), kLanes = 32 / kN;   // lanes of a row
        const int r0 = lane / kLanes, c = lane % kLanes * kN;
#pragma unroll
        for (int i = 0; i < 32 / (32 / kLanes); ++i) {
            const int r = r0 + i * (32 / kLanes);
            if (r >= rows) break;
            const int64_t at = (m + r) * s.N + n + c;
            float z[kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) z[j] = v[r * kLtPitch + c + j];
            if (!kPart) {
                if (ep.bias) {
#pragma unroll
                    for (int j = 0; j < kN; j += 4) {
                        const float4 b = __ldg(reinterpret_cast<const float4 *>(ep.bias + n + c + j));
                        z[j] += b.x; z[j + 1] += b.y; z[j + 2] += b.z; z[j + 3] += b.w;
                    }
                }
                if (pre) put_vec<kN>(pre + at, z);
                if constexpr (kN == 4) {
                    if (pre32) put_vec(pre32 + at, z);
                }
                if (ep.act != SSD_ACT_NONE) {
#pragma unroll
                    for (int j = 0; j < kN; ++j) z[j] = linear_act<TO>(z[j], ep.act);
                }
                if (res) {
                    float q[kN];
                    get_vec<TO, kN>(res + at, q);
#pragma unroll
                    for (int j = 0; j < kN; ++j) z[j] += q[j];
                }
            }
            put_vec(out + at, z);
        }
        return;
    }
    if (lane >= s.N - n) return;
    const float b = !kPart && ep.bias ? ep.bias[n + lane] : 0.0f;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
        const int64_t at = (m + r) * s.N + n + lane;
        float z = v[r * kLtPitch + lane];
        if (!kPart) {
            if (ep.bias) z += b;
            if (pre) pre[at] = __float2bfloat16_rn(z);
            if (pre32) pre32[at] = z;
            z = linear_act<TO>(z, ep.act);
            if (res) z += to_f(res[at]);
        }
        out[at] = linear_from_f<TO>(z);
    }
}

// The products of two parts each, smallest first: 3 lo, 2 mid, 1 hi with zeros
// in the place of infinities and NaN, 0 hi (an infinity meets the other's first
// part only, never a zero that is not there in fp32).
__device__ __forceinline__ int part_of_a(int term) { return 0x012123 >> (4 * term) & 15; }
__device__ __forceinline__ int part_of_b(int term) { return 0x021321 >> (4 * term) & 15; }

// kTerms 1: A B;  2: (A0 + A1) B, A1's products first;  6: the products of two
// operands in three parts each.  kSegs: sums in segments of s.seg stages, added in
// registers (up to 192 columns: those of 256 would not fit).
template <int BN, bool AMN, bool BMN, int kTerms, bool kSegs>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLtThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, LinearEpilogue ep,
                 LtShape s, unsigned *status) {
    constexpr int S = LtStages<BN>::value;
    constexpr uint32_t kB = lt_b_bytes<BN>(), kStage = kLtABytes + kB;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S * kStage);   // the first CTA's: a stage has landed in both
    uint64_t *empty = full + S;                                         // each CTA's: its stage may be refilled
    uint64_t *acc_full = empty + S, *acc_empty = acc_full + 2;          // accumulators; acc_empty the first CTA's
    uint32_t *slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *abort = reinterpret_cast<volatile int *>(slot + 1);
    float *staged = reinterpret_cast<float *>(smem + S * kStage + 256);   // per epilogue warp 32 x 32
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, tiles = s.mt * s.nt * s.splits;

    if (warp == kLtMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(lt_columns<BN>())
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], i == 0 ? 1 + s.fault : 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * kLtEpiWarps);
        }
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&ta);
        tma_prefetch_desc(&tb);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_launch_dependents();      // the join
    pdl_wait_prerequisites();     // the split that made the operands
    if (s.clear && blockIdx.x == 0 && tid == 0) *status = 0;   // (a wait takes seconds to give up and set it)

    if (warp == kLtTmaWarp) {
        if (elect_one()) {
            int it = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                int split, mi, ni;
                tile_of(t, s, split, mi, ni);
                const int m0 = mi * kLtM + (int)rank * 128, n0 = ni * BN + (int)rank * (BN / 2);
                const int k_end = min(s.ksteps, (split + 1) * s.per), seg = kSegs ? s.seg : s.per;
                for (int k0 = split * s.per; ok && k0 < k_end; k0 += seg) {
                    const int len = min(seg, k_end - k0);
                    for (int i = 0; i < len * kTerms; ++i, ++it) {
                        const int term = kTerms == 1 ? 0 : i / len, k = (k0 + i - term * len) * kLtK;
                        const int ra = kTerms == 1 ? 0 : (kTerms == 2 ? 1 - term : part_of_a(term)) * s.planeA, rb = kTerms <= 2 ? 0 : part_of_b(term) * s.planeB;
                        const int st = it % S;
                        if (!(ok = wait_cluster(&empty[st], ((uint32_t)(it / S) & 1u) ^ 1u, s.budget, abort))) break;
                        const uint32_t bar = at_rank(smem_u32(&full[st]), 0);
                        if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kStage);
                        const uint32_t a = smem_u32(smem + st * kStage), b = a + kLtABytes;
                        if (AMN) {
                            load_2d_pair(a, &ta, bar, m0, k + ra);
                            load_2d_pair(a + 8192, &ta, bar, m0 + 64, k + ra);
                        } else {
                            load_2d_pair(a, &ta, bar, k, m0 + ra);
                        }
                        if (BMN) {
#pragma unroll
                            for (int q = 0; q < BN / 128; ++q) load_2d_pair(b + 8192 * q, &tb, bar, n0 + 64 * q, k + rb);
                        } else {
                            load_2d_pair(b, &tb, bar, k, n0 + rb);
                        }
                    }
                }
            }
        }
    } else if (warp == kLtMmaWarp) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = idesc_bf16(kLtM, BN, AMN, BMN);
            // 16 k further on: 32 bytes along a swizzled row, or 16 rows of 128 bytes
            constexpr uint32_t stepA = (AMN ? 2048u : 32u) >> 4, stepB = (BMN ? 2048u : 32u) >> 4;
            int it = 0, at = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                int split, mi, ni;
                tile_of(t, s, split, mi, ni);
                const int k_end = min(s.ksteps, (split + 1) * s.per), seg = kSegs ? s.seg : s.per;
                for (int k0 = split * s.per; ok && k0 < k_end; k0 += seg, ++at) {
                    const int buf = at & 1, steps = min(seg, k_end - k0) * kTerms;
                    if (!(ok = wait_cluster(&acc_empty[buf], ((uint32_t)(at >> 1) & 1u) ^ 1u, s.budget, abort))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * (lt_columns<BN>() / 2);
                    for (int i = 0, first = 1; i < steps; ++i, ++it) {
                        const int st = it % S;
                        if (!(ok = wait_cluster(&full[st], (uint32_t)(it / S) & 1u, s.budget, abort))) break;
                        tc_fence_after();
                        const uint32_t a = smem_u32(smem + st * kStage), b = a + kLtABytes;
                        const uint64_t da = sdesc_sw128(a, AMN ? 8192 : 16, 1024), db = sdesc_sw128(b, BMN ? 8192 : 16, 1024);
#pragma unroll
                        for (int q = 0; q < kLtK / 16; ++q) {
                            mma_pair(d, da + q * stepA, db + q * stepB, idesc, first ? 0u : 1u);
                            first = 0;
                        }
                        commit_pair(&empty[st]);
                    }
                    if (ok) commit_pair(&acc_full[buf]);
                }
            }
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;
        float *mine = staged + warp * 32 * kLtPitch;
        int at = 0;
        bool ok = true;
        for (int t = pair; ok && t < tiles; t += pairs) {
            int split, mi, ni;
            tile_of(t, s, split, mi, ni);
            const int64_t m = (int64_t)mi * kLtM + rank * 128 + quarter * 32;
            auto leave = [&](int c, const float (&v)[32]) {
                if (m >= s.M || (int64_t)ni * BN + 32 * c >= s.N) return;
                const int n = ni * BN + 32 * c;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 32; ++i) mine[lane * kLtPitch + i] = v[i];
                __syncwarp();
                if (s.splits > 1)
                    store_block<float, true>(mine, m, n, ep, s, s.part + (int64_t)split * s.M * s.N, lane);
                else if (s.out_f32) store_block<float, false>(mine, m, n, ep, s, nullptr, lane);
                else store_block<__nv_bfloat16, false>(mine, m, n, ep, s, nullptr, lane);
            };
            // waits for the accumulator, hands each 32 columns on, lets it be refilled
            auto drain = [&](auto &&take) {
                const int buf = at & 1;
                ok = __all_sync(0xffffffffu, wait_cluster(&acc_full[buf], (uint32_t)(at >> 1) & 1u, s.budget, abort));
                if (!ok) return;
                ++at;
                tc_fence_after();
                const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + buf * (lt_columns<BN>() / 2);
                take(src);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(at_rank(smem_u32(&acc_empty[buf]), 0));
            };
            if constexpr (!kSegs) {
                drain([&](uint32_t src) {
#pragma unroll 1
                    for (int c = half; c < BN / 32; c += 2) {
                        if (m >= s.M || (int64_t)ni * BN + 32 * c >= s.N) break;
                        float v[32];
                        tmem_ld32(src + 32 * c, v);
                        leave(c, v);
                    }
                });
            } else {
                constexpr int kMine = (BN / 32 + 1) / 2;   // pieces of 32 columns of a warp (one less with an odd number, half 1)
                float sum[kMine][32];
#pragma unroll
                for (int c = 0; c < kMine; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c][i] = 0.0f;
                const int k_end = min(s.ksteps, (split + 1) * s.per);
                for (int k0 = split * s.per; ok && k0 < k_end; k0 += s.seg)
                    drain([&](uint32_t src) {
#pragma unroll
                        for (int c = 0; c < kMine; ++c) {
                            if (BN / 32 % 2 && half + 2 * c >= BN / 32) break;
                            float v[32];
                            tmem_ld32(src + 32 * (half + 2 * c), v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) sum[c][i] += v[i];
                        }
                    });
                if (ok) {
#pragma unroll
                    for (int c = 0; c < kMine; ++c) {
                        if (BN / 32 % 2 && half + 2 * c >= BN / 32) break;
                        leave(half + 2 * c, sum[c]);
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        // let the copies and MMAs in flight end (about a millisecond) before
        // the shared memory and the accumulators go away
        if (tid == 0) atomicOr(status, kStatusTimeout);
        const long long t0 = clock64();
        while (clock64() - t0 < (1ll << 21)) {
        }
    }
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == kLtMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(lt_columns<BN>()) : "memory");
}

// Rows of `cols` bf16 copied to rows of `groups` times 8, zeros behind: a warp
// takes 256 elements of a row, read by twos where rows start on pairs, else one by one
// (side by side, so whole sectors), and written 16 bytes a lane.
__global__ void __launch_bounds__(256)
linear_pad_kernel(const unsigned short *__restrict__ src, uint4 *__restrict__ dst, int64_t rows, int cols, int groups) {
    __shared__ __align__(16) unsigned short s_row[8][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = (groups + 31) / 32;
    const int64_t item = (int64_t)blockIdx.x * 8 + warp, row = item / pieces;
    const int c0 = (int)(item - row * pieces) * 256;
    if (row >= rows) return;
    const unsigned short *from = src + row * cols + c0;
    if (cols % 2 == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 2 * (i * 32 + lane);
            reinterpret_cast<uint32_t *>(s_row[warp])[i * 32 + lane] =
                c0 + c < cols ? __ldg(reinterpret_cast<const uint32_t *>(from + c)) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s_row[warp][i * 32 + lane] = c0 + i * 32 + lane < cols ? __ldg(from + i * 32 + lane) : 0;
    }
    __syncwarp();
    if (c0 / 8 + lane < groups) dst[row * groups + c0 / 8 + lane] = reinterpret_cast<const uint4 *>(s_row[warp])[lane];
}

// fp32 matrices in bf16 parts: planes of `up` rows of `ld` elements (both
// multiples of 64, zeros behind the matrix) hold hi, hi with zeros for
// infinities and NaN, mid, lo.  A warp takes 256 elements of a row: read side by
// side (rows start anywhere), written 16 bytes a lane.  Bound by HBM, 12 bytes a
// value.
struct SplitOf {
    const float *src;
    __nv_bfloat16 *dst;
    int64_t rows, up;
    int cols, ld;
};
__device__ __forceinline__ void split_piece(const SplitOf &a, unsigned item, __nv_bfloat16 (*s_part)[256]) {
    const int lane = threadIdx.x & 31;
    const unsigned pieces = (unsigned)(a.ld + 255) / 256u, row = item / pieces;
    const int c0 = (int)(item - row * pieces) * 256;
    const bool there = row < a.rows;
    const float *src = a.src + (int64_t)row * a.cols + c0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = there && c0 + i * 32 + lane < a.cols ? __ldg(src + i * 32 + lane) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool finite = fabsf(v[i]) <= 3.402823466e38f;
        __nv_bfloat16 hi = __float2bfloat16_rn(v[i]);
        // (the largest floats would round to infinity)
        if (finite && __hisinf(hi)) hi = __float2bfloat16_rz(v[i]);
        const float rest = finite ? v[i] - __bfloat162float(hi) : 0.0f;
        const __nv_bfloat16 mid = __float2bfloat16_rn(rest);
        s_part[0][i * 32 + lane] = hi;
        s_part[1][i * 32 + lane] = finite ? hi : __float2bfloat16_rn(0.0f);
        s_part[2][i * 32 + lane] = mid;
        s_part[3][i * 32 + lane] = __float2bfloat16_rn(rest - __bfloat162float(mid));
    }
    __syncwarp();
    if (c0 + 8 * lane >= a.ld) return;
    __nv_bfloat16 *dst = a.dst + (int64_t)row * a.ld + c0 + 8 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4 *>(dst + k * a.up * a.ld) = reinterpret_cast<const uint4 *>(s_part[k])[lane];
}
__global__ void __launch_bounds__(256)
linear_split_kernel(const __grid_constant__ SplitOf a, const __grid_constant__ SplitOf b, unsigned items_a, unsigned items) {
    __shared__ __align__(16) __nv_bfloat16 s_part[8][4][256];
    pdl_launch_dependents();
    const unsigned item = blockIdx.x * 8u + (threadIdx.x >> 5);
    if (item >= items) return;
    if (item < items_a) split_piece(a, item, s_part[threadIdx.x >> 5]);
    else split_piece(b, item - items_a, s_part[threadIdx.x >> 5]);
}

int64_t up64(int64_t v) { return (v + 63) / 64 * 64; }

struct Plan {
    int bn, splits, per;
};

// The tile width and the parts of k, by an estimate of the cycles: a pair
// takes 310 for 256 x 128 x 64 and 600 for 256 x 256 x 64, measured with all
// SMs at it, and never less than about 235 (the copies); a tile costs about
// 1500 more (fill, last stores); joining parts costs a launch and 8 bytes a
// value.  Widths between the powers of two fill the last wave (1024 x 5120: 128
// tiles of 160 in two waves, where 80 of 256 leave most of the second empty); an
// operand along its own rows comes in boxes of 64, so 128 and 256 there, and
// 128 takes about 345 (dx of 8192 x 5120 x 2560: 165 us with 128, 154 with 256).
Plan plan_of(int64_t M, int64_t N, int64_t K, bool b_mn, int terms, bool segs, double *cycles = nullptr) {
    const int64_t ksteps = (K + kLtK - 1) / kLtK, pairs = 74;
    Plan best = {256, 1, (int)ksteps};
    double least = 1e300;
    for (int bn : {256, 224, 192, 160, 128, 96, 64}) {
        if ((b_mn && bn % 128) || (terms == 6 && bn != 128) || (segs && bn > 192)) continue;
        const int64_t tiles = (M + kLtM - 1) / kLtM * ((N + bn - 1) / bn);
        const double step = terms * (b_mn && bn == 128 && terms <= 2 ? 345 : 20 + 2.27 * bn > 235 ? 20 + 2.27 * bn : 235);
        for (int want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            const int64_t per = (ksteps + want - 1) / want, splits = (ksteps + per - 1) / per;
            if (want > 1 && (splits != want || per < (terms == 6 ? 1 : 4) || (tiles >= pairs && !(segs && terms <= 2)))) continue;
            const double waves = (double)((tiles * splits + pairs - 1) / pairs);
            double t = waves * ((double)per * step + 1500);
            if (splits > 1) t += 4000 + (double)M * N * splits * 8 / 3500;
            if (t < least) {
                least = t;
                best = {bn, (int)splits, (int)per};
            }
        }
    }
    if (cycles) *cycles = least;
    return best;
}

template <int BN, bool AMN, bool BMN, int kTerms = 1, bool kSegs = kTerms == 6>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const LinearEpilogue &ep, const LtShape &s,
                   unsigned *status, cudaStream_t st) {
    auto kern = linear_tc_kernel<BN, AMN, BMN, kTerms, kSegs>;
    static int sms[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!sms[dev]) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)lt_smem<BN>())) != cudaSuccess)
            return e;
        int n = 0;
        if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        sms[dev] = n;
    }
    const int tiles = s.mt * s.nt * s.splits, pairs = tiles < sms[dev] / 2 ? tiles : sms[dev] / 2;
    return linear_launch(kern, (unsigned)(2 * pairs), kLtThreads, lt_smem<BN>(), kTerms == 6, st, ta, tb, ep, s, status);
}

// The map of an operand with `rows` rows of `cols` contiguous elements, ld apart.
bool map_of(CUtensorMap *map, const void *p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, strides[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64u, (uint32_t)box_rows};
    return tmap_encode_2d(map, p, kTmapBF16, dims, strides, box);
}

}  // namespace

size_t linear_tc_part_bytes(int64_t M, int64_t N, int64_t K, bool b_mn, int terms) {
    size_t most = 0;   // whether the output is fp32 is not known here
    for (const bool segs : {false, true}) {
        const Plan p = plan_of(M, N, K, b_mn, terms, segs);
        const size_t n = p.splits > 1 ? align256((size_t)(M * N) * p.splits * sizeof(float)) : 0;
        if (n > most) most = n;
    }
    return most;
}

cudaError_t linear_pad(const void *src, void *dst, int64_t rows, int64_t cols, cudaStream_t s) {
    const int64_t groups = (cols + 7) / 8, items = rows * ((groups + 31) / 32);
    linear_pad_kernel<<<(unsigned)((items + 7) / 8), 256, 0, s>>>((const unsigned short *)src, (uint4 *)dst, rows, (int)cols,
                                                                  (int)groups);
    return cudaGetLastError();
}

cudaError_t linear_tc(const void *A, int64_t lda, bool a_mn, const void *B, int64_t ldb, bool b_mn,
                      const LinearEpilogue &ep, int out_f32, int64_t M, int64_t N, int64_t K, void *part, unsigned *status,
                      bool clear, cudaStream_t st, int terms, int64_t plane) {
    const bool segs = K > (out_f32 ? kLtSegBf16 * kLtK : kLtLongK);
    const Plan p = plan_of(M, N, K, b_mn, terms, segs);
    LtShape s = {};
    s.M = (int)M; s.N = (int)N; s.ksteps = (int)((K + kLtK - 1) / kLtK);
    s.mt = (int)((M + kLtM - 1) / kLtM); s.nt = (int)((N + p.bn - 1) / p.bn);
    s.splits = p.splits; s.per = p.per;
    s.part = static_cast<float *>(part);
    s.out_f32 = out_f32; s.vec = N % 8 == 0; s.clear = clear;
    s.fault = test_fault(kFaultLinear); s.budget = wait_budget(kFaultLinear);
    CUtensorMap ta, tb;
    const int count = (p.per + kLtSegBf16 - 1) / kLtSegBf16;
    s.seg = (p.per + count - 1) / count;   // segments of equal length
    const int64_t more = (terms - 1) * plane;   // rows in front of the last part
    s.planeA = (int)plane;
    if (!(a_mn ? map_of(&ta, A, K + more, M, lda, 64) : map_of(&ta, A, M + more, K, lda, 128)) ||
        !(b_mn ? map_of(&tb, B, K, N, ldb, 64) : map_of(&tb, B, N, K, ldb, p.bn / 2)))
        return cudaErrorInvalidValue;
    TraceScope tr(st, kTrLinear);
    cudaError_t e;
    if (segs) {
        if (terms == 2) e = a_mn ? launch<128, true, true, 2, true>(ta, tb, ep, s, status, st) : launch<128, false, true, 2, true>(ta, tb, ep, s, status, st);
        else if (b_mn) e = a_mn ? launch<128, true, true, 1, true>(ta, tb, ep, s, status, st) : launch<128, false, true, 1, true>(ta, tb, ep, s, status, st);
        else if (p.bn == 192) e = launch<192, false, false, 1, true>(ta, tb, ep, s, status, st);
        else if (p.bn == 160) e = launch<160, false, false, 1, true>(ta, tb, ep, s, status, st);
        else if (p.bn == 128) e = launch<128, false, false, 1, true>(ta, tb, ep, s, status, st);
        else if (p.bn == 96) e = launch<96, false, false, 1, true>(ta, tb, ep, s, status, st);
        else e = launch<64, false, false, 1, true>(ta, tb, ep, s, status, st);
    } else if (terms == 2) {
        if (p.bn == 256) e = a_mn ? launch<256, true, true, 2>(ta, tb, ep, s, status, st) : launch<256, false, true, 2>(ta, tb, ep, s, status, st);
        else e = a_mn ? launch<128, true, true, 2>(ta, tb, ep, s, status, st) : launch<128, false, true, 2>(ta, tb, ep, s, status, st);
    } else if (b_mn) {
        if (p.bn == 256) e = a_mn ? launch<256, true, true>(ta, tb, ep, s, status, st) : launch<256, false, true>(ta, tb, ep, s, status, st);
        else e = a_mn ? launch<128, true, true>(ta, tb, ep, s, status, st) : launch<128, false, true>(ta, tb, ep, s, status, st);
    } else {
        switch (p.bn) {
            case 256: e = launch<256, false, false>(ta, tb, ep, s, status, st); break;
            case 224: e = launch<224, false, false>(ta, tb, ep, s, status, st); break;
            case 192: e = launch<192, false, false>(ta, tb, ep, s, status, st); break;
            case 160: e = launch<160, false, false>(ta, tb, ep, s, status, st); break;
            case 128: e = launch<128, false, false>(ta, tb, ep, s, status, st); break;
            case 96: e = launch<96, false, false>(ta, tb, ep, s, status, st); break;
            default: e = launch<64, false, false>(ta, tb, ep, s, status, st); break;
        }
    }
    if (e == cudaSuccess && p.splits > 1)
        e = out_f32 ? linear_join<float>(s.part, ep, M, N, p.splits, st)
                    : linear_join<__nv_bfloat16>(s.part, ep, M, N, p.splits, st);
    return e;
}

// ---- fp32 operands in parts
bool linear_parts_pay(int64_t M, int64_t N, int64_t K, bool b_mn, double other_cycles) {
    // (below 64 k the 24 steps that a stage of 64 takes could cut more off a sum than its own roundings do)
    if (M >= (1ll << 28) || N >= (1ll << 28) || K >= (1ll << 28) || K < 64) return false;
    double cycles = 0;
    plan_of(M, N, K, b_mn, 6, true, &cycles);
    // the split's launch and its traffic: 12 bytes a value at 3500 a cycle; set-up of the kernel
    return cycles + 12000 + 12.0 * (double)(M * K + N * K) / 3500 < other_cycles;
}

size_t linear_parts_bytes(int64_t rows, int64_t cols) { return align256((size_t)(4 * up64(rows)) * up64(cols) * 2); }

size_t linear_parts_sum_bytes(int64_t M, int64_t N, int64_t K, bool b_mn) {
    const Plan p = plan_of(M, N, K, b_mn, 6, true);
    return p.splits > 1 ? align256((size_t)(M * N) * p.splits * sizeof(float)) : 0;
}

cudaError_t linear_parts(const float *a, int64_t a_rows, int64_t a_cols, void *a_parts, const float *b, int64_t b_rows, int64_t b_cols,
                         void *b_parts, cudaStream_t st) {
    auto of = [](const float *src, int64_t rows, int64_t cols, void *dst) {
        return SplitOf{src, static_cast<__nv_bfloat16 *>(dst), rows, up64(rows), (int)cols, (int)up64(cols)};
    };
    const SplitOf ga = of(a, a_rows, a_cols, a_parts), gb = of(b, b_rows, b_cols, b_parts);
    const unsigned na = a ? (unsigned)(ga.up * ((ga.ld + 255) / 256)) : 0, nb = b ? (unsigned)(gb.up * ((gb.ld + 255) / 256)) : 0;
    if (na + nb == 0) return cudaSuccess;
    linear_split_kernel<<<(na + nb + 7) / 8, 256, 0, st>>>(ga, gb, na, na + nb);
    return cudaGetLastError();
}

cudaError_t linear_tc_parts(const void *A, bool a_mn, const void *B, bool b_mn, const LinearEpilogue &ep, int64_t M, int64_t N, int64_t K,
                            void *part, unsigned *status, bool clear, cudaStream_t st) {
    const Plan p = plan_of(M, N, K, b_mn, 6, true);
    LtShape s = {};
    s.M = (int)M; s.N = (int)N; s.ksteps = (int)((K + kLtK - 1) / kLtK);
    s.mt = (int)((M + kLtM - 1) / kLtM); s.nt = (int)((N + p.bn - 1) / p.bn);
    s.splits = p.splits; s.per = p.per;
    s.part = static_cast<float *>(part);
    s.out_f32 = 1; s.vec = N % 8 == 0; s.clear = clear;
    s.fault = test_fault(kFaultLinear); s.budget = wait_budget(kFaultLinear);
    s.seg = kLtSegParts;
    s.planeA = (int)up64(a_mn ? K : M);
    s.planeB = (int)up64(b_mn ? K : N);
    CUtensorMap ta, tb;
    const int64_t la = up64(a_mn ? M : K), lb = up64(b_mn ? N : K);
    if (!map_of(&ta, A, 4ll * s.planeA, la, la, a_mn ? 64 : 128) || !map_of(&tb, B, 4ll * s.planeB, lb, lb, b_mn ? 64 : p.bn / 2))
        return cudaErrorInvalidValue;
    TraceScope tr(st, kTrLinear);
    cudaError_t e = a_mn ? launch<128, true, true, 6>(ta, tb, ep, s, status, st)
                    : b_mn ? launch<128, false, true, 6>(ta, tb, ep, s, status, st)
                           : launch<128, false, false, 6>(ta, tb, ep, s, status, st);
    if (e == cudaSuccess && p.splits > 1) e = linear_join<float>(s.part, ep, M, N, p.splits, st);
    return e;
}

}  // namespace ssd
