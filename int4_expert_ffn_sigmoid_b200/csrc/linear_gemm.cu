// Dense projection with int4 weights and group scales for more tokens than
// the weight-streaming kernel takes in a pass: a tcgen05 GEMM with the weights
// as its M side.
//
//   D[128 weight rows][kN tokens] += A[128][128 columns] x[kN][128 columns]^T
//
// per stage, accumulated in tensor memory over all columns (of this CTA's
// share).  A is built in tensor memory from the packed codes: 16 converter
// warps turn a row's codes into bf16 and multiply them by the row's group
// scale.  A bf16 product alone would round every weight by up to 2^-9, as much
// as the output's own rounding; the rest goes into a second bf16 matrix,
//   hi = bf16(c s),  lo = bf16(c s - hi)        (exact to 2^-16 of the weight)
// and each k step takes two MMAs, hi x + lo x.  The second MMA is free until
// the tensor pipe bounds the kernel (a few hundred tokens), and x enters as it
// is, by TMA.  A scale of 24 or 11 bits is itself split in two bf16 parts.
//
// Few row tiles: a cluster of up to eight CTAs shares a tile's columns, sums
// its parts in shared memory (rank c % size takes tokens 8 c .. 8 c + 7) and
// stores them; in the same order every time.
//
// Roles (576 threads, one CTA per SM): warps 0-15 convert (groups of eight
// take alternate stages) and then read the accumulators out; warp 16 issues
// the TMA loads, warp 17 the MMAs.  Every wait is bounded; a CTA whose wait
// gave up (never, in a correct run) stores NaN.
#include <cooperative_groups.h>
#include <cuda.h>

#include "group_stream.cuh"
#include "moe_tc.h"

namespace moe {
namespace {

constexpr int kRows = 128, kStageK = 128;
constexpr int kConvWarps = 16, kThreads = 32 * (kConvWarps + 2);
constexpr int kAStages = 3, kACols = 128, kACol0 = 128;  // tensor memory: D in columns 0-127, then the A stages
constexpr int kTmemCols = 512;
constexpr int kWBytes = kRows * kStageK / 2;
constexpr long long kWait = kBulkWaitCycles;

template <int kN>
struct Geo {
    static constexpr int kXBytes = kN * kStageK * 2;
    static constexpr int kStage = kWBytes + kXBytes;
    static constexpr int kStages = kN == 128 ? 4 : kN == 64 ? 6 : 8;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kRing + 1024 + 512;
    // the cluster's partial sums reuse the ring: chunks of 8 tokens, rounded up per rank
    static_assert((kN / 8 + 7) * 8 * kRows * 4 <= kRing, "partial sums fit the ring");
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
__device__ __forceinline__ ScaleParts split_scale(uint32_t raw, int stype) {
    const float s = stype == kScaleF32   ? __uint_as_float(raw)
                    : stype == kScaleBf16 ? __uint_as_float(raw << 16)
                                          : __half2float(__ushort_as_half((unsigned short)raw));
    ScaleParts p;
    p.hi = __float2bfloat162_rn(s);
    p.lo = __float2bfloat162_rn(s - __low2float(p.hi));
    return p;
}

// Eight codes times a scale: four words of bf16 pairs in column order, and
// what they lack.  kLow: the scale has a low part.
template <bool kLow>
__device__ __forceinline__ void dequant8(uint32_t w, const ScaleParts& s, uint32_t* hi, uint32_t* lo) {
    uint32_t c[4];
    int4x8_to_16<true>(w, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&c[j]);
        const __nv_bfloat162 h = __hmul2(v, s.hi);
        __nv_bfloat162 l = __hfma2(v, s.hi, __hneg2(h));  // exact: a 4-bit by an 8-bit value has 12 bits
        if (kLow) l = __hfma2(v, s.lo, l);
        hi[j] = *reinterpret_cast<const uint32_t*>(&h);
        lo[j] = *reinterpret_cast<const uint32_t*>(&l);
    }
}

struct GemmPlan {
    int stages;  // 128-column stages of a row
    int row_tiles;
};

template <int kN, bool kLow>
__global__ void __launch_bounds__(kThreads, 1)
    linear_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LinearArgs a,
                       GemmPlan p) {
    namespace cg = cooperative_groups;
    using G = Geo<kN>;
    extern __shared__ __align__(128) uint8_t dsm[];
    __shared__ uint64_t full[G::kStages], empty[G::kStages], a_full[kAStages], a_empty[kAStages], done_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_abort;
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
        for (int i = 0; i < G::kStages; ++i) {
            bar_init(full + i, 1);
            bar_init(empty + i, 1 + 8);  // the MMAs' commit, a group's converter warps
        }
        for (int i = 0; i < kAStages; ++i) {
            bar_init(a_full + i, 8);
            bar_init(a_empty + i, 1);
        }
        bar_init(&done_bar, 1);
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kConvWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == kConvWarps) {
        if (lane == 0) {
            auto load_w = [&](int i) {
                const int s = i % G::kStages;
                bar_expect_tx(full + s, G::kStage);
                tma_tile(ring_p + s * G::kStage, &map_w, full + s, (st0 + i) * (kStageK / 2), row0);
            };
            auto load_x = [&](int i) {
                const int s = i % G::kStages;
                uint8_t* x = ring_p + s * G::kStage + kWBytes;
                tma_tile(x, &map_x, full + s, (st0 + i) * kStageK, tok0);
                tma_tile(x + G::kXBytes / 2, &map_x, full + s, (st0 + i) * kStageK + 64, tok0);
            };
            // the weights do not depend on the kernel before this one, x does
            const int early = n < G::kStages ? n : G::kStages;
            for (int i = 0; i < early; ++i) load_w(i);
            pdl_wait();
            pdl_release();
            int issued = early;
            for (int i = 0; i < early; ++i) load_x(i);
            for (int i = early; i < n; ++i) {
                if (*abort || !bar_wait_or_abort(empty + i % G::kStages, (i / G::kStages - 1) & 1, kWait, abort)) {
                    *abort = 1;
                    break;
                }
                load_w(i);
                load_x(i);
                ++issued;
            }
            // every copy lands before the CTA's shared memory is reused or goes away
            for (int i = issued > G::kStages ? issued - G::kStages : 0; i < issued; ++i)
                bar_wait(full + i % G::kStages, (i / G::kStages) & 1, kWait);
        }
    } else if (warp == kConvWarps + 1) {
        // The whole warp runs the loop and one lane issues: under a divergent
        // `lane == 0` every operand of an MMA is first moved to a uniform
        // register (a stage of 16 MMAs took 1680 cycles, against LATER).
        constexpr uint32_t idesc = idesc_bf16(kRows, kN);
        const bool leader = elect_one();
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int s = i % G::kStages, sa = i % kAStages;
            // a full A stage implies a landed ring stage for the converters; this warp's MMAs read x themselves
            ok = warp_wait(full + s, (i / G::kStages) & 1, abort) && warp_wait(a_full + sa, (i / kAStages) & 1, abort);
            if (!ok) break;
            fence_after();
            const uint64_t b0 = desc_sw128(ring + s * G::kStage + kWBytes);
            const uint32_t acol = tmem + kACol0 + sa * kACols;
            if (leader) {
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t b = b0 + ((kb * (G::kXBytes / 2) + kk * 32) >> 4);
                        mma_ts(tmem, acol + kb * 32 + kk * 8, b, idesc, (i | kb | kk) != 0);
                        mma_ts(tmem, acol + 64 + kb * 32 + kk * 8, b, idesc, 1);
                    }
                commit(empty + s);
                commit(a_empty + sa);
            }
            __syncwarp();
        }
        if (leader) commit(&done_bar);  // all MMAs issued are complete
    } else {
        // warp (group, half, quarter): rows 32 quarter .. + 31 (lane = row),
        // columns 64 half .. + 63 of the stages i = group mod 2
        const int quarter = warp & 3, half = (warp >> 2) & 1, group = warp >> 3;
        const int row = min(row0 + quarter * 32 + lane, a.N - 1);
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + kACol0 + half * 32;
        const int r = quarter * 32 + lane;
        const bool two = a.gshift == 5;  // two scales for 64 columns
        const size_t s0 = (size_t)row * a.G;
        uint32_t raw[2];
        auto load_scales = [&](int i) {
            const int k = (st0 + i) * kStageK + half * 64;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u == 1 && !two) break;
                const size_t at_s = s0 + min((k + 32 * u) >> a.gshift, a.G - 1);
                raw[u] = a.stype == kScaleF32 ? __ldg(static_cast<const uint32_t*>(a.scales) + at_s)
                                              : (uint32_t)__ldg(static_cast<const unsigned short*>(a.scales) + at_s);
            }
        };
        raw[0] = raw[1] = 0;
        if (group < n) load_scales(group);
        for (int i = group; i < n; i += 2) {
            const int s = i % G::kStages, sa = i % kAStages;
            ScaleParts sp[2];
            sp[0] = split_scale(raw[0], a.stype);
            sp[1] = two ? split_scale(raw[1], a.stype) : sp[0];
            if (i + 2 < n) load_scales(i + 2);
            if (!warp_wait(full + s, (i / G::kStages) & 1, abort)) break;
            uint4 w[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)  // 16-byte chunk 2 half + u of the row's 64 bytes (64-byte swizzle)
                w[u] = lds128(ring + s * G::kStage + r * 64 + (((2 * half + u) ^ ((r >> 1) & 3)) << 4));
            if (!warp_wait(a_empty + sa, ((i / kAStages) & 1) ^ 1u, abort)) break;
            fence_after();
            uint32_t hi[32], lo[32];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                dequant8<kLow>(w[u].x, sp[u], hi + 16 * u, lo + 16 * u);
                dequant8<kLow>(w[u].y, sp[u], hi + 16 * u + 4, lo + 16 * u + 4);
                dequant8<kLow>(w[u].z, sp[u], hi + 16 * u + 8, lo + 16 * u + 8);
                dequant8<kLow>(w[u].w, sp[u], hi + 16 * u + 12, lo + 16 * u + 12);
            }
            st_tmem32(at + sa * kACols, hi);
            st_tmem32(at + sa * kACols + 64, lo);
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            fence_before();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(a_full + sa);
                bar_arrive(empty + s);
            }
        }
    }
    pdl_wait();  // for every thread that reads add or writes out below (the producer has waited: a no-op there)
    __syncwarp();

    // Accumulators to registers: warp (quarter, cgrp): columns 8 c .. + 7, c = cgrp mod 4.
    constexpr int kChunks = kN / 8, kMine = (kChunks + 3) / 4;
    const int quarter = warp & 3, cgrp = warp >> 2;
    float v[kMine][8];
    // What the output rows already hold is loaded while the last MMAs run: at
    // the store, one round trip to memory would follow another.
    uint16_t plus[kMine][8];
    auto inside = [&](int t, int row) { return t < a.T && row < a.N; };
    // a cluster's rank owns the chunks c = rank mod size, thread by thread
    const int own = (kChunks + size - 1 - rank) / size * 8 * kRows;
    auto own_t = [&](int i) { return tok0 + 8 * (i / (8 * kRows) * size + rank) + i / kRows % 8; };
    if (a.add && warp < kConvWarps) {
#pragma unroll
        for (int m = 0; m < kMine; ++m)
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                int t = tok0 + 8 * (cgrp + 4 * m) + u, row = row0 + quarter * 32 + lane;
                bool in = cgrp + 4 * m < kChunks;
                if (size > 1) {  // a rank's share is at most half as many elements
                    const int i = threadIdx.x + (8 * m + u) * 32 * kConvWarps;
                    t = own_t(i);
                    row = row0 + i % kRows;
                    in = i < own;
                }
                plus[m][u] = in && inside(t, row) ? __ldcg(reinterpret_cast<const unsigned short*>(a.add) + t * a.lda + row) : 0;
            }
    }
    if (warp < kConvWarps) {
        const bool ok = bar_wait(&done_bar, 0, kWait) && *abort == 0 && n > 0;
        const bool all = __all_sync(0xffffffffu, ok) != 0;
        fence_after();
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int c = cgrp + 4 * m;
            if (c < kChunks) ld_tmem8(tmem + ((uint32_t)(quarter * 32) << 16) + 8 * c, v[m]);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (!all) v[m][u] = __int_as_float(0x7fc00000);
        }
        fence_before();
    }
    __syncthreads();
    // Tensor memory is freed before any wait on another CTA.
    if (warp == kConvWarps + 1) {
        bar_wait(&done_bar, 0, kWait);
        __syncwarp();
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
    }
    auto store = [&](int t, int row, float y, uint16_t add) {
        if (!inside(t, row)) return;
        if (a.add) y += bf16lo(add);
        if (a.out_f32) static_cast<float*>(a.out)[t * a.ldo + row] = y;
        else static_cast<__nv_bfloat16*>(a.out)[t * a.ldo + row] = __float2bfloat16_rn(y);
    };
    if (size == 1) {
        if (warp < kConvWarps)
#pragma unroll
            for (int m = 0; m < kMine; ++m)
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (cgrp + 4 * m < kChunks)
                        store(tok0 + 8 * (cgrp + 4 * m) + u, row0 + quarter * 32 + lane, v[m][u], plus[m][u]);
        return;
    }
    // [chunk of this rank][source rank][token][row]
    float* part = reinterpret_cast<float*>(ring_p);
    cluster.sync();  // every CTA is through with its ring
    if (warp < kConvWarps)
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int c = cgrp + 4 * m;
            if (c >= kChunks) continue;
            float* to = cluster.map_shared_rank(part, c % size) + ((size_t)(c / size) * size + rank) * 8 * kRows + quarter * 32 + lane;
#pragma unroll
            for (int u = 0; u < 8; ++u) to[u * kRows] = v[m][u];
        }
    cluster.sync();
    if (warp < kConvWarps)
#pragma unroll
        for (int e = 0; e < kMine * 8; ++e) {
            const int i = threadIdx.x + e * 32 * kConvWarps;
            if (i >= own) break;
            float y = 0.f;
            for (int q = 0; q < size; ++q) y += part[((size_t)(i / (8 * kRows) * size + q) * 8 + i / kRows % 8) * kRows + i % kRows];
            store(own_t(i), row0 + i % kRows, y, plus[e / 8][e % 8]);
        }
}

struct Capacity {
    int ctas[9];  // CTAs of a cluster size that run at once (0: not asked yet)
};

template <int kN, bool kLow>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
    auto* k = linear_gemm_kernel<kN, kLow>;
    using G = Geo<kN>;
    static Capacity caps[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t c = {};
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = G::kSmem;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    Capacity& cap = caps[dev];
    if (cap.ctas[1] == 0) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
        for (int s = 8; s >= 1 && e == cudaSuccess; --s) {
            int n = 0;
            at[1].val.clusterDim.x = s;
            c.gridDim = dim3(s);
            c.attrs = at + 1;
            c.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, k, &c);
            cap.ctas[s] = n * s;
        }
        if (e != cudaSuccess) return e;
    }
    GemmPlan p;
    p.stages = (a.K + kStageK - 1) / kStageK;
    p.row_tiles = (a.N + kRows - 1) / kRows;
    const long long tiles = (long long)p.row_tiles * ((a.T + kN - 1) / kN);
    // Columns per cluster: the fewest stages one after another, a CTA's start
    // and end counted as six stages and the cluster's exchange as six more.
    int size = 1;
    long long best = 0;
    for (int s = 1; s <= 8 && s <= p.stages; ++s) {
        if (cap.ctas[s] == 0) continue;
        const long long waves = (tiles * s + cap.ctas[s] - 1) / cap.ctas[s];
        const long long cost = waves * ((p.stages + s - 1) / s + 6 + (s > 1 ? 6 : 0));
        if (s == 1 || cost < best) {
            size = s;
            best = cost;
        }
    }
    CUtensorMap mw, mx;
    if (!encode_tensor_map_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.w, a.K / 2, a.N, kStageK / 2, kRows,
                              CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_tensor_map_rows(&mx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.K, a.T, (uint64_t)a.ldx * 2, 64, kN,
                                CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    at[1].val.clusterDim.x = size;
    c.gridDim = dim3((unsigned)(tiles * size));
    c.stream = stream;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, k, mw, mx, a, p);
}

}  // namespace

cudaError_t launch_linear_gemm(const LinearArgs& a, cudaStream_t stream) {
    const bool low = a.stype != kScaleBf16;
    if (a.T <= 16) return low ? launch<16, true>(a, stream) : launch<16, false>(a, stream);
    if (a.T <= 32) return low ? launch<32, true>(a, stream) : launch<32, false>(a, stream);
    if (a.T <= 64) return low ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
    return low ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
}

}  // namespace moe
