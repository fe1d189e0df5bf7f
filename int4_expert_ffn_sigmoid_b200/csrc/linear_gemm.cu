// Dense projection with int4 weights and group scales for more tokens than
// the weight-streaming kernel takes: a tcgen05 GEMM with the weights as its M
// side.
//
//   D[128 weight rows][kN tokens] += A[128][128 columns] x[kN][128 columns]^T
//
// per stage, accumulated in tensor memory over all columns (of this CTA's
// share).  A is built in tensor memory from the packed codes: the converter
// warps turn a row's codes into bf16 and multiply them by the row's group
// scale.  x enters as it is, by TMA.
//
// Two forms.  One part: each weight is rounded once to bf16 (2^-8 of it at
// most; the codes 0, 1, 2, 4 and 8 times a bf16 scale are exact).  Two parts
// (kRest): what that rounding left is a second bf16 matrix and each step takes
// a second MMA, which holds a weight to 2^-15.  Two parts are taken for up to
// eight tokens, where weight streaming is as good and a token's accuracy should
// not hang on its company, and under MOE_FULL_WEIGHTS.  They cost 64 tokens x
// 6144 x 6144 13.5 -> 19.7 us, 512 x 4096 x 6144 22.6 -> 38.7, 16 x 6144 x 2048 6.3
// -> 10.6: the MMAs' pace.  One part is the default for more tokens because a
// bf16 output rounds as much again (relative L2 error 1.66e-3; the weights'
// rounding adds 1.2e-3 with bf16 scales to 1.7e-3 with f32 ones).
//
// Few row tiles: a cluster of up to eight CTAs shares a tile's columns; each
// leaves its part in shared memory and sums all parts of the chunks of eight
// tokens c = rank mod size, rank 0's first, the same every time.
//
// Roles (864 threads, one CTA per SM): warps 0-23 convert (in groups that take
// the stages in turn) and then read the accumulators out; warps 24 and 25
// issue the TMA loads of the codes and of x, warp 26 the MMAs.  Every wait is
// bounded; a CTA whose wait gave up (never, in a correct run) stores NaN.  Under
// MOE_TEST_STALL the first CTA's codes stop half way.
//
// What bounds it.  64 tokens x 6144 x 6144: 13.9 us (3.4 at the copy rate): the
// MMAs' pace over the stages of one CTA, 96 of the 148 SMs (48 row tiles in
// clusters of two), and the start and end of a launch.  512 x 4096 x 6144:
// 22.5 us, 1.15 PFLOP/s: in its 24 stages a CTA's MMAs run at their full rate
// (1024 cycles each, 13 us); the first stage's loads and conversion, the
// cluster's exchange and the output take the rest, and 20 SMs have no tile.
#include <cooperative_groups.h>
#include <cuda.h>

#include "group_stream.cuh"
#include "moe_tc.h"

namespace moe {
namespace {

constexpr int kRows = 128, kStageK = 128;
constexpr int kConvWarps = 24, kThreads = 32 * (kConvWarps + 3);
constexpr int kWarpW = kConvWarps, kWarpX = kConvWarps + 1, kWarpMma = kConvWarps + 2;
constexpr int kTmemCols = 512;
constexpr int kWBytes = kRows * kStageK / 2;
constexpr long long kWait = kBulkWaitCycles;

// kRest: a second A matrix with what the rounding of the weights left.
template <int kN, bool kRest>
struct Geo {
    static constexpr int kACols = kRest ? 128 : 64;  // tensor memory columns of an A stage
    // Stages of x and of A go together: the one commit after a stage's MMAs
    // frees both.  The codes have a deeper ring of their own.
    static constexpr int kXBytes = kN * kStageK * 2;
    static constexpr int kStages = kRest || kN == 256 ? 3 : kN == 128 ? 4 : 6;
    static constexpr int kWStages = kN == 256 ? 3 : 6;
    // Converter warps: kGroups take the stages in turn; of a stage's two
    // 64-column halves a warp takes both (kSplit = 1: less to do per stage, and
    // more stages under way) or one (2: where shared memory holds few stages).
    static constexpr int kSplit = kRest || kN >= 128 ? 2 : 1;
    static constexpr int kGroups = kConvWarps / (4 * kSplit);
    // A barrier's phase is told apart by its parity alone, so nobody may wait
    // for a phase before the one ahead of it is over.  A slot of the code ring
    // is always the same group's, which has then seen the phase before; a
    // stage's `empty` is waited for by groups that have written a stage after
    // the one it frees.
    static_assert(kWStages % kGroups == 0 && kGroups <= kStages, "phases");
    static constexpr int kACol0 = kN == 256 ? 256 : 128;  // D before it
    static constexpr int kRing = kStages * kXBytes + kWStages * kWBytes;
    // over half of an SM's: two CTAs there would wait on each other's tensor memory
    static constexpr int kSmem = kRing + 1024 > 116 * 1024 ? kRing + 1024 : 116 * 1024;
    static_assert(kN <= kACol0 && kACol0 + kStages * kACols <= kTmemCols, "tensor memory");
    static_assert(kN * kRows * 4 <= kRing, "the f32 tile fits the rings");
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16, bf16 operands, f32 accumulators, both K-major
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// True on one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(0xffffffffu, bar_try(bar, parity))) return true;
    if (__all_sync(0xffffffffu, bar_wait_or_abort(bar, parity, kWait, abort))) return true;
    *abort = 1;
    return false;
}

__device__ __forceinline__ void st_tmem32(uint32_t at, const uint32_t (&o)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(at),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]), "r"(o[9]),
        "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15]), "r"(o[16]), "r"(o[17]), "r"(o[18]),
        "r"(o[19]), "r"(o[20]), "r"(o[21]), "r"(o[22]), "r"(o[23]), "r"(o[24]), "r"(o[25]), "r"(o[26]), "r"(o[27]),
        "r"(o[28]), "r"(o[29]), "r"(o[30]), "r"(o[31])
        : "memory");
}
__device__ __forceinline__ void st_tmem16(uint32_t at, const uint32_t (&o)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(at),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]), "r"(o[9]),
        "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
        : "memory");
}
__device__ __forceinline__ void ld_tmem8(uint32_t at, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// The bf16 parts of a scale, each in both halves of a word.
struct ScaleParts {
    __nv_bfloat162 hi, lo;
};
template <bool kLow>
__device__ __forceinline__ ScaleParts split_scale(uint32_t raw, int stype) {
    if (!kLow) {  // bf16 scales
        const uint32_t two = __byte_perm(raw, 0, 0x1010);
        const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&two);
        return {s, s};
    }
    const float s = stype == kScaleF32    ? __uint_as_float(raw)
                    : stype == kScaleBf16 ? __uint_as_float(raw << 16)
                                          : __half2float(__ushort_as_half((unsigned short)raw));
    ScaleParts p;
    p.hi = __float2bfloat162_rn(s);
    p.lo = __float2bfloat162_rn(s - __low2float(p.hi));
    return p;
}

// Eight codes times a scale: four words of bf16 pairs in column order.
// kLow: the scale has a low part.  kRest: to r what o lacks, c s_hi - o exactly
// (a multiple of s_hi's last place, at most eight of them), then + c s_lo rounded
// to bf16.  The scale's two parts and r's rounding are off by 2^-16 of the weight
// at most each (together by 1.03 times that over two million scales and all codes).
template <bool kLow, bool kRest>
__device__ __forceinline__ void dequant8(uint32_t w, const ScaleParts& s, uint32_t* o, uint32_t* r) {
    const uint32_t w4 = w >> 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // int4x8_to_16 with the sign flip folded into the mask's operation: 128 + 8 + c, minus 136
        const uint32_t t = (__byte_perm(w, w4, j | ((4 + j) << 8)) & 0x000f000fu) ^ 0x43084308u;
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                         __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308)));
        const __nv_bfloat162 h = kLow ? __hfma2(v, s.hi, __hmul2(v, s.lo)) : __hmul2(v, s.hi);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
        if (kRest) {
            const __nv_bfloat162 l = __hfma2(v, s.lo, __hfma2(v, s.hi, __hneg2(h)));
            r[j] = *reinterpret_cast<const uint32_t*>(&l);
        }
    }
}

// A ring's slot and the parity of its phase, stepped instead of divided out:
// the loading and MMA warps share their schedulers with six converter warps
// each, and every instruction of theirs waits its turn.
template <int kSlots>
struct Slot {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void step(int by = 1) {
        s += by;
        if (s >= kSlots) {
            s -= kSlots;
            ph ^= 1;
        }
    }
};

struct GemmPlan {
    int stages;  // 128-column stages of a row
    int row_tiles;
};

template <int kN, bool kLow, bool kRest>
__global__ void __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearArgs a,
                       GemmPlan p) {
    namespace cg = cooperative_groups;
    using G = Geo<kN, kRest>;
    constexpr int kACols = G::kACols;
    static_assert(kLow || !kRest, "the rest is taken with both parts of the scale");
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ uint64_t w_full[G::kWStages], w_empty[G::kWStages], x_full[G::kStages], a_full[G::kStages], empty[G::kStages], done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort, s_never;
    volatile int* abort = &s_abort;
    // warp-uniform to the compiler too: the MMA warp's descriptors then live in uniform registers
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    cg::cluster_group cluster = cg::this_cluster();
    const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const uint32_t ring = (smem_addr(dsm) + 1023u) & ~1023u;
    uint8_t* ring_p = dsm + (ring - smem_addr(dsm));
    const int tile = blockIdx.x / size, row0 = (tile % p.row_tiles) * kRows, tok0 = (tile / p.row_tiles) * kN;
    const int st0 = (int)((long long)p.stages * rank / size), st1 = (int)((long long)p.stages * (rank + 1) / size);
    const int n = st1 - st0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < G::kWStages; ++i) {
            bar_init(w_full + i, 1);
            bar_init(w_empty + i, 4 * G::kSplit);  // a group's converter warps
        }
        for (int i = 0; i < G::kStages; ++i) {
            bar_init(x_full + i, 1);
            bar_init(a_full + i, 4 * G::kSplit);
            bar_init(empty + i, 1);  // the MMAs' commit
        }
        bar_init(&done_bar, 1);
        s_abort = s_never = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    uint8_t* const xring = ring_p;
    uint8_t* const wring = ring_p + G::kStages * G::kXBytes;
    if (warp == kWarpW) {
        const bool leader = elect_one();
        Slot<G::kWStages> w;
        const int upto = a.stall && blockIdx.x == 0 ? n / 2 : n;
        int i = 0;
        for (int x = st0 * (kStageK / 2); i < upto; ++i, x += kStageK / 2) {  // weights do not depend on the kernel before this one
            if (i >= G::kWStages && !warp_wait(w_empty + w.s, w.ph ^ 1u, abort)) break;
            if (leader) {
                refill_fence();
                bar_expect_tx(w_full + w.s, kWBytes);
                tma_tile(wring + w.s * kWBytes, &map_w, w_full + w.s, x, row0);
            }
            w.step();
        }
        if (upto < n) {  // every other role waits for the rest
            stall_on_unset_flag(&s_never, kStallCycles);
            *abort = 1;
        }
        // every copy lands before the CTA's shared memory is reused or goes away
        for (int j = i > G::kWStages ? i - G::kWStages : 0; j < i; ++j)
            bar_wait(w_full + j % G::kWStages, (j / G::kWStages) & 1, kWait);
    } else if (warp == kWarpX) {
        const bool leader = elect_one();
        pdl_wait();
        pdl_release();
        Slot<G::kStages> t;
        int i = 0;
        for (int x = st0 * kStageK; i < n; ++i, x += kStageK) {
            if (i >= G::kStages && !warp_wait(empty + t.s, t.ph ^ 1u, abort)) break;
            if (leader) {
                uint8_t* to = xring + t.s * G::kXBytes;
                bar_expect_tx(x_full + t.s, G::kXBytes);
                tma_tile(to, &map_x, x_full + t.s, x, tok0);
                tma_tile(to + G::kXBytes / 2, &map_x, x_full + t.s, x + 64, tok0);
            }
            t.step();
        }
        for (int j = i > G::kStages ? i - G::kStages : 0; j < i; ++j)
            bar_wait(x_full + j % G::kStages, (j / G::kStages) & 1, kWait);
    } else if (warp == kWarpMma) {
        // The whole warp runs the loop and one lane issues: under a divergent
        // `lane == 0` every operand of an MMA is first moved to a uniform
        // register (16 MMAs took 1130 cycles to issue, against 560).
        constexpr uint32_t idesc = idesc_bf16(kRows, kN);
        const bool leader = elect_one();
        Slot<G::kStages> t;
        for (int i = 0; i < n; ++i, t.step()) {
            const bool ready = bar_try(x_full + t.s, t.ph) & bar_try(a_full + t.s, t.ph);
            if (!__all_sync(0xffffffffu, ready) && !(warp_wait(x_full + t.s, t.ph, abort) && warp_wait(a_full + t.s, t.ph, abort)))
                break;
            fence_after();
            const uint64_t b0 = desc_sw128(ring + t.s * G::kXBytes);
            const uint32_t acol = tmem + G::kACol0 + t.s * kACols;
            if (leader) {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t b = b0 + ((kb * (G::kXBytes / 2) + kk * 32) >> 4);
                        mma_ts(tmem, acol + kb * 32 + kk * 8, b, idesc, (i | kb | kk) != 0);
                        if (kRest) mma_ts(tmem, acol + 64 + kb * 32 + kk * 8, b, idesc, 1);
                    }
                commit(empty + t.s);
            }
            __syncwarp();
        }
        if (leader) commit(&done_bar);  // all MMAs issued are complete
    } else {
        // warp (group, half, quarter): rows 32 quarter .. + 31 (lane = row) of
        // the stages i = group mod kGroups, its half or both
        constexpr int kHalves = 2 / G::kSplit;
        const int quarter = warp & 3, half0 = G::kSplit == 2 ? (warp >> 2) & 1 : 0, group = warp / (4 * G::kSplit);
        const int row = min(row0 + quarter * 32 + lane, a.N - 1);
        const int r = quarter * 32 + lane;
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + G::kACol0 + half0 * 32;
        const uint32_t wrow = smem_addr(wring) + r * 64;
        const int esh = a.stype == kScaleF32 ? 2 : 1;
        const char* srow = static_cast<const char*>(a.scales) + (((size_t)row * a.G) << esh);
        const bool two = a.gshift == 5;  // two scales for 64 columns
        uint32_t raw[kHalves][2];
        auto load_scales = [&](int i) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u == 1 && !two) continue;
                    const int k = (st0 + i) * kStageK + (half0 + h) * 64 + 32 * u;
                    const char* p = srow + (min(k >> a.gshift, a.G - 1) << esh);
                    raw[h][u] = kLow && a.stype == kScaleF32 ? __ldg(reinterpret_cast<const uint32_t*>(p))
                                                             : (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p));
                }
        };
#pragma unroll
        for (int h = 0; h < kHalves; ++h) raw[h][0] = raw[h][1] = 0;
        if (group < n) load_scales(group);
        Slot<G::kStages> t;
        Slot<G::kWStages> w;
        t.step(group);
        w.step(group);
        for (int i = group; i < n; i += G::kGroups, t.step(G::kGroups), w.step(G::kGroups)) {
            const int s = t.s, sw = w.s;
            ScaleParts sp[kHalves][2];
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                sp[h][0] = split_scale<kLow>(raw[h][0], a.stype);
                sp[h][1] = two ? split_scale<kLow>(raw[h][1], a.stype) : sp[h][0];
            }
            if (i + G::kGroups < n) load_scales(i + G::kGroups);
            const uint32_t full_ph = w.ph, free_ph = t.ph ^ 1u;
            // usually both are ready: one round trip to the barriers, not two
            const bool ready = bar_try(w_full + sw, full_ph) & bar_try(empty + s, free_ph);
            if (!__all_sync(0xffffffffu, ready) &&
                !(warp_wait(w_full + sw, full_ph, abort) && warp_wait(empty + s, free_ph, abort)))
                break;
            fence_after();
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                auto codes = [&](int u) {  // 16-byte chunk 2 half + u of the row's 64 bytes (64-byte swizzle)
                    return lds128(wrow + sw * kWBytes + (((2 * (half0 + h) + u) ^ ((r >> 1) & 3)) << 4));
                };
                if constexpr (kRest) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t o[16], l[16];
                        const uint4 v = codes(u);
                        dequant8<kLow, true>(v.x, sp[h][u], o, l);
                        dequant8<kLow, true>(v.y, sp[h][u], o + 4, l + 4);
                        dequant8<kLow, true>(v.z, sp[h][u], o + 8, l + 8);
                        dequant8<kLow, true>(v.w, sp[h][u], o + 12, l + 12);
                        st_tmem16(at + s * kACols + h * 32 + 16 * u, o);
                        st_tmem16(at + s * kACols + 64 + h * 32 + 16 * u, l);
                    }
                } else {
                    uint32_t o[32];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 v = codes(u);
                        dequant8<kLow, false>(v.x, sp[h][u], o + 16 * u, nullptr);
                        dequant8<kLow, false>(v.y, sp[h][u], o + 16 * u + 4, nullptr);
                        dequant8<kLow, false>(v.z, sp[h][u], o + 16 * u + 8, nullptr);
                        dequant8<kLow, false>(v.w, sp[h][u], o + 16 * u + 12, nullptr);
                    }
                    st_tmem32(at + s * kACols + h * 32, o);
                }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(a_full + s);
                bar_arrive(w_empty + sw);
            }
        }
    }
    pdl_wait();  // for every thread that reads add or writes out below (the loading warp has waited: a no-op there)
    __syncwarp();

    // Output u of this CTA (a cluster's rank owns the chunks of eight tokens c =
    // rank mod size): one token's 128 rows, a warp each, four rows a lane.  The
    // loops below are short and rolled: they run once, and code fetched cold
    // costs more than it does.
    constexpr int kChunks = kN / 8, kBatch = 2;
    const int own = (kChunks - rank + size - 1) / size * 8;
    auto token_of = [&](int u) { return (u >> 3) * size * 8 + rank * 8 + (u & 7); };  // of the CTA's tile
    const int row = row0 + 4 * lane;
    const bool four = row + 3 < a.N;
    const bool add4 = four && a.lda % 4 == 0 && reinterpret_cast<uintptr_t>(a.add) % 8 == 0;
    const bool out4 = four && a.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(a.out) % (a.out_f32 ? 16 : 8) == 0;
    auto load_add = [&](int u) {  // four bf16
        const int t = tok0 + token_of(u);
        uint2 o = make_uint2(0, 0);
        if (u >= own || t >= a.T) return o;
        const unsigned short* p = reinterpret_cast<const unsigned short*>(a.add) + t * a.lda + row;
        if (add4) return __ldcg(reinterpret_cast<const uint2*>(p));
        if (row < a.N) o.x = __ldcg(p);
        if (row + 1 < a.N) o.x |= (uint32_t)__ldcg(p + 1) << 16;
        if (row + 2 < a.N) o.y = __ldcg(p + 2);
        if (four) o.y |= (uint32_t)__ldcg(p + 3) << 16;
        return o;
    };
    uint2 plus[kBatch] = {};  // on its way while the last MMAs run
    bool all = false;
    if (warp < kConvWarps) {
        if (a.add)
#pragma unroll
            for (int e = 0; e < kBatch; ++e) plus[e] = load_add(warp + e * kConvWarps);
        const bool ok = bar_wait(&done_bar, 0, kWait) && *abort == 0 && n > 0;
        all = __all_sync(0xffffffffu, ok) != 0;
        fence_after();
    }
    __syncthreads();  // every copy has landed: the rings are free
    // The tile to shared memory, [token][row].
    float* tile_sum = reinterpret_cast<float*>(ring_p);
    if (warp < kConvWarps) {
        const int quarter = warp & 3;
#pragma unroll 1
        for (int c = warp >> 2; c < kChunks; c += kConvWarps / 4) {
            float v[8];
            ld_tmem8(tmem + ((uint32_t)(quarter * 32) << 16) + 8 * c, v);
#pragma unroll
            for (int u = 0; u < 8; ++u) tile_sum[(c * 8 + u) * kRows + quarter * 32 + lane] = all ? v[u] : __int_as_float(0x7fc00000);
        }
        fence_before();
    }
    __syncthreads();
    // Tensor memory is freed before any wait on another CTA.
    if (warp == kWarpMma) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
    }
    if (size > 1) cluster.sync();
    if (warp < kConvWarps) {
#pragma unroll 1
        for (int u0 = warp; u0 < own; u0 += kBatch * kConvWarps) {
            float4 y[kBatch];
            uint2 next[kBatch] = {};
            if (a.add)
#pragma unroll
                for (int e = 0; e < kBatch; ++e) next[e] = load_add(u0 + (kBatch + e) * kConvWarps);
#pragma unroll
            for (int e = 0; e < kBatch; ++e) y[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int q = 0; q < size; ++q) {
                const float* from = (size > 1 ? cluster.map_shared_rank(tile_sum, q) : tile_sum) + 4 * lane;
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    const int u = u0 + e * kConvWarps;
                    if (u >= own) continue;
                    const float4 v = *reinterpret_cast<const float4*>(from + token_of(u) * kRows);
                    y[e].x += v.x;
                    y[e].y += v.y;
                    y[e].z += v.z;
                    y[e].w += v.w;
                }
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int u = u0 + e * kConvWarps, t = tok0 + token_of(u);
                if (u < own && t < a.T) {
                    float o[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
                    if (a.add) {
                        o[0] += bf16lo(plus[e].x);
                        o[1] += bf16hi(plus[e].x);
                        o[2] += bf16lo(plus[e].y);
                        o[3] += bf16hi(plus[e].y);
                    }
                    if (a.out_f32) {
                        float* to = static_cast<float*>(a.out) + t * a.ldo + row;
                        if (out4) {
                            *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (row + i < a.N) to[i] = o[i];
                        }
                    } else {
                        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + t * a.ldo + row;
                        if (out4) {
                            const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
                            *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                                       *reinterpret_cast<const uint32_t*>(&hi));
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (row + i < a.N) to[i] = __float2bfloat16_rn(o[i]);
                        }
                    }
                }
                plus[e] = next[e];
            }
        }
    }
    if (size > 1) cluster.sync();  // no CTA is gone while another reads its tile
}

template <int kN, bool kLow, bool kRest>
cudaError_t launch(const LinearArgs& a, int dev, int size, cudaStream_t stream) {
    auto* k = linear_gemm_kernel<kN, kLow, kRest>;
    using G = Geo<kN, kRest>;
    static std::atomic<int> set[64];
    if (!set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
        if (e != cudaSuccess) return e;
        set[dev] = 1;
    }
    GemmPlan p;
    p.stages = (a.K + kStageK - 1) / kStageK;
    p.row_tiles = (a.N + kRows - 1) / kRows;
    CUtensorMap mw, mx;
    if (!encode_tensor_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w, a.K / 2, a.N, kStageK / 2, kRows,
                              CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_tensor_map_rows(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.T, (uint64_t)a.ldx * 2, 64, kN,
                                CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((long long)p.row_tiles * ((a.T + kN - 1) / kN) * size));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = G::kSmem;
    c.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, k, mw, mx, a, p);
}

// CTAs of a cluster size that run at once, of any of the kernels (one an SM).
struct Capacity {
    std::atomic<int> ctas[9];  // [1] = 0: not asked yet; written last
};
cudaError_t capacity(int dev, const Capacity** out) {
    static Capacity caps[64];
    Capacity& cap = caps[dev];
    *out = &cap;
    if (cap.ctas[1] > 0) return cudaSuccess;
    auto* k = linear_gemm_kernel<256, true, false>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<256, false>::kSmem);
    for (int s = 8; s >= 1 && e == cudaSuccess; --s) {
        int n = 0;
        cudaLaunchConfig_t c = {};
        c.gridDim = dim3(s);
        c.blockDim = dim3(kThreads);
        c.dynamicSmemBytes = Geo<256, false>::kSmem;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = s;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        c.attrs = &at;
        c.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, k, &c);
        cap.ctas[s] = n * s;
    }
    return e;
}

// Time of a CTA, in 10 ns: its stages one after another, its start and end, a
// cluster's exchange, and what a launch takes that leaves the next one less
// than half of the SMs to start on while it runs.  Fitted (8 % r.m.s.) to 1330
// measured launches of 11 shapes from 256 x 1024 to 12288 x 2048, 20 to 512
// tokens, each tile width and cluster size, one after another on a stream.  With
// weights in two parts a stage takes 1.7 times as long (1141 launches), and the
// same costs choose within 2 % of the best on average, 33 % at worst.
struct TileCost {
    int tokens, stage, fixed;
};
constexpr TileCost kTiles[] = {{16, 36, 160}, {32, 36, 184}, {64, 36, 257}, {128, 39, 379}, {256, 56, 648}};
constexpr int kExchange = 53, kExchangeCta = 29, kCrowd = 200;

template <bool kLow>
cudaError_t launch_rounded(const LinearArgs& a, int tokens, int dev, int size, cudaStream_t stream) {
    switch (tokens) {
        case 16: return launch<16, kLow, false>(a, dev, size, stream);
        case 32: return launch<32, kLow, false>(a, dev, size, stream);
        case 64: return launch<64, kLow, false>(a, dev, size, stream);
        case 128: return launch<128, kLow, false>(a, dev, size, stream);
        default: return launch<256, kLow, false>(a, dev, size, stream);
    }
}

cudaError_t launch_rest(const LinearArgs& a, int tokens, int dev, int size, cudaStream_t stream) {
    switch (tokens) {
        case 16: return launch<16, true, true>(a, dev, size, stream);
        case 32: return launch<32, true, true>(a, dev, size, stream);
        case 64: return launch<64, true, true>(a, dev, size, stream);
        default: return launch<128, true, true>(a, dev, size, stream);
    }
}

}  // namespace

// Tokens of a tile and CTAs of a cluster: the least time of the CTAs' waves by
// the costs above, which is within 2 % of the best of all on average (35 % at
// worst).  Few rows and many tokens go to narrow tiles, each converting the
// weights again, many rows to wide ones.  Against the narrowest tile that holds
// T (up to 256), us: 64 tokens x 1024 x 1024 3.7 and 6.2, 256 4.3 and 11.2, 300 x
// 6144 x 6144 27 and 39, 40 x 2048 x 8192 9.4 and 12.5.
cudaError_t launch_linear_gemm(const LinearArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const Capacity* cap;
    if ((e = capacity(dev, &cap)) != cudaSuccess) return e;
    const int stages = (a.K + kStageK - 1) / kStageK;
    const bool rest = a.full || a.T <= kStreamTok;
    int tokens = 0, size = 1;
    long long best = 0;
    for (const TileCost& c : kTiles) {
        if ((c.tokens >= 2 * a.T && c.tokens > 16) || (rest && c.tokens > 128)) break;
        const long long tiles = (long long)((a.N + kRows - 1) / kRows) * ((a.T + c.tokens - 1) / c.tokens);
        for (int s = 1; s <= 8 && s <= stages; ++s) {
            if (cap->ctas[s] == 0) continue;
            const long long ctas = tiles * s, waves = (ctas + cap->ctas[s] - 1) / cap->ctas[s];
            const long long cost = waves * ((stages + s - 1) / s * c.stage + c.fixed + (s > 1 ? kExchange + kExchangeCta * s : 0)) +
                                   (2 * ctas > cap->ctas[1] ? kCrowd : 0);
            if (tokens == 0 || cost < best) {
                tokens = c.tokens;
                size = s;
                best = cost;
            }
        }
    }
    if (rest) return launch_rest(a, tokens, dev, size, stream);
    return a.stype == kScaleBf16 ? launch_rounded<false>(a, tokens, dev, size, stream)
                                 : launch_rounded<true>(a, tokens, dev, size, stream);
}

}  // namespace moe
