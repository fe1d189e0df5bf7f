// A whole MoE layer for a few tokens, with group-scaled int4 weights, in two
// kernels (three when the router or the gate and up weights are large):
//
//   few_gate_up_kernel  router logits, selection, and h = silu(g) * u of every
//                       touched expert and of the shared one
//   few_down_kernel     the down projections, their weighted sum, the residual
//
// Both read each touched expert's weights once for all its tokens
// (group_stream.cuh) and let the columns of an mma tile be the tokens themselves: token t is
// column pair t % 4 of every expert's product, so the down kernel adds all
// experts of a row up in registers.  Of tokens q and q + 4 the one that picked
// the expert takes the column; a second pass over a weight tile is needed only
// where both did (lane_token; 64 experts of 2560 x 512, 8 of them picked, 8
// tokens: 47.3 us, 49.7 with a pass for each touched half of the tokens).  A
// column without a token is computed and not used.
//
// h is stored as the down kernel's int8 operands: per 32 columns two int8
// parts and a power-of-two scale (2^-15 of the block's largest value), taken
// in f32 from the finished, routing-weighted h.
//
// What bounds it.  256 experts of 6144 x 2048, 8 of them picked, one shared:
// one token 46.8 us (28.1 at the copy rate), five tokens 185.6 us (120.7).  Both
// kernels are held by their instructions (59 and 67 % of the issue slots at
// five tokens, 49 and 33 % of DRAM's peak): about 300 a warp for 16 rows x 256
// columns of the down kernel, of whose time the mma products take 14 % and the
// loads of h 7 %.  64 experts of 1024 x 512, 2 picked, one token: 10.1 us against
// 0.95, none of it bandwidth: the chain logits - exchange - selection (1.0) - first
// routed weights from HBM (1.4) - down (2.4), and two launches.
#include <cooperative_groups.h>

#include "group_stream.cuh"
#include "moe_launch.h"

namespace moe {

constexpr int kFewWarps = 16;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewDepth = 3;
// The down kernel: more warps, shallower rings.  Its units are short and each
// waits for an h from L2, so warps in flight count for more than copies (one
// token and five of 6144 x 2048, 8 of 256 experts: 46.9 and 185.6 us, 48.7 and
// 188.7 with 16 warps and rings of three).
constexpr int kDownWarps = 24, kDownThreads = 32 * kDownWarps, kDownDepth = 2;
constexpr int kFewTileRows = 32;  // h elements of a gate/up tile
constexpr int kFewSmemMax = 227 * 1024;
constexpr int kFewXMax = 98 * 1024;
// CTAs that share the router: a cluster of kFewCluster computes all logits,
// each CTA those of an eighth of the experts, and exchanges them in shared
// memory.  Clusters of eight leave 120 of 148 SMs usable, of four 132, of two
// all (64 experts of 1024 x 512, one, four and eight tokens: 10.1, 11.5 and 16.7;
// 10.5, 11.9 and 17.4; 11.3, 13.2 and 19.5 us).  With router
// weights beyond kFewRouterMax, or gate and up weights beyond kFewWeightsMax
// (elements of h times H), the logits are a kernel of their own in front
// (router_logits_kernel) and every SM takes part in this one.  Logits here and
// in front, us, four tokens:
//   64 x 1024 router, 192 tiles  12.5, 14.5    1040 tiles of H = 1024  29.6, 32.3 (eight tokens)
//   64 x 2048, 272 tiles         17.4, 18.9    1024 tiles of H = 2048  36.8, 35.4
//   64 x 4096, 272 tiles         27.1, 26.7    128 x 4096, 144 tiles   24.3, 20.9
constexpr int kFewCluster = 8;
constexpr int kFewRouterMax = 64 * 4096;
// Columns from which several warps share an expert's logits (six experts of
// 2688 x 1152, five tokens: 30.6 us, 33.5 with one warp each; where the rows are
// short the join costs more: 64 x 1024, one token, 10.1 us and 10.6).
constexpr int kFewShareMin = 2048;
constexpr long long kFewWeightsMax = 40ll << 20;

int few_logit_slices(int H) { return (H / 128 + 2) / 3; }

// Shared memory of a gate/up CTA: rings, two buffers of partial sums, scales and
// int8 parts of x; x itself where the logits are computed here.
constexpr size_t kFewDynMax = kFewSmemMax - 13 * 1024;  // static shared memory comes on top
size_t few_smem(int NT, int T, int H, int x_stride, bool split) {
    const size_t chunks = (H + kChunkK - 1) / kChunkK;
    return (size_t)kFewWarps * kFewDepth * kStageBytes + 2 * (size_t)kFewWarps * 4 * NT * 16 * 4 + chunks * 4 * NT * 4 +
           (size_t)2 * T * x_stride + (split ? 0 : (size_t)2 * T * H);
}
int few_touched(const FewArgs& a) { return a.E < a.T * a.K ? a.E : a.T * a.K; }
int few_tiles(const FewArgs& a) { return a.Is / kFewTileRows + few_touched(a) * (a.I / kFewTileRows); }
// Once true, true for every larger T (a workspace for T tokens serves fewer).
bool few_split_router(const FewArgs& a) {
    const int stride = x_stride<true>((a.H + kChunkK - 1) / kChunkK);
    return a.E * a.H > kFewRouterMax || (long long)few_tiles(a) * kFewTileRows * a.H > kFewWeightsMax ||
           few_smem(a.T <= 4 ? 1 : 2, a.T, a.H, stride, false) > kFewDynMax;
}

__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t b = __float_as_uint(f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}

// Top-K of one token (one warp) from its scores in shared memory: the K
// largest score + bias (NaN as -infinity), ties to the lower expert.  Lane k <
// K returns pick k and its weight.
__device__ __forceinline__ void few_select(const FewArgs& a, const float* scores, const float* bias, int lane, int& out_e,
                                           float& out_w) {
    uint32_t key[kMaxE / 32];
#pragma unroll
    for (int j = 0; j < kMaxE / 32; ++j) {
        const int e = lane + 32 * j;
        const float k = e < a.E ? scores[e] + bias[e] : 0.f;
        key[j] = e < a.E ? ordered(isnan(k) ? -INFINITY : k + 0.0f) : 0;  // + 0: -0 compares as 0; 0: below every key
    }
    int my_e = -1;
    float my_s = 0.f, ssum = 0.f;
#pragma unroll 1
    for (int k = 0; k < a.K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < kMaxE / 32; ++j) best = max(best, key[j]);
        best = __reduce_max_sync(0xffffffffu, best);
        unsigned e = 0x7fffffff;
#pragma unroll
        for (int j = kMaxE / 32 - 1; j >= 0; --j)
            if (key[j] == best) e = lane + 32 * j;
        const int be = (int)__reduce_min_sync(0xffffffffu, e);
#pragma unroll
        for (int j = 0; j < kMaxE / 32; ++j)
            if (lane + 32 * j == be) key[j] = 0;
        const float s = scores[be];
        if (lane == k) {
            my_e = be;
            my_s = s;
        }
        ssum += s;
    }
    topp_picks(a.K, a.topp, a.scale, lane, my_e, my_s, ssum, out_e, out_w);
}

// The token of column pair q in a pass over an expert that `tokens` picked; not
// one of them where the column is unused.
template <int NT>
__device__ __forceinline__ int lane_token(unsigned tokens, int q, int pass) {
    return NT == 1 || (pass == 0 && ((tokens >> q) & 1u)) ? q : q + 4;
}
template <int NT>
__device__ __forceinline__ int token_passes(unsigned tokens) {
    return NT == 1 || !(tokens & (tokens >> 4)) ? 1 : 2;
}

template <int NT, bool kCoarse>
__global__ void __launch_bounds__(kFewThreads, 1) few_gate_up_kernel(FewArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ FewPicks P;
    __shared__ float s_logit[kFewTok][kMaxE];  // logits, then scores
    __shared__ float s_bias[kMaxE];
    __shared__ unsigned s_mask[kMaxE / 32];  // touched experts
    __shared__ float s_weight[kFewMaxU][kFewTok];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int T = a.T, H = a.H, half = H / 2;
    const int chunks = (H + kChunkK - 1) / kChunkK;
    const int xs_bytes = x_stride<kCoarse>(chunks);
    constexpr int kRed = kFewWarps * 4 * NT * 16;
    float* red = reinterpret_cast<float*>(smem + kFewWarps * kFewDepth * kStageBytes);  // [2][warp][4 NT][16]
    float* xs = red + 2 * kRed;                                                         // [chunks][4 NT]
    int8_t* xq = reinterpret_cast<int8_t*>(xs + chunks * 4 * NT);                       // [token][part][xs_bytes]
    const uint32_t ring = smem_addr(smem + warp * (kFewDepth * kStageBytes));

    // Tile i of the layer: 32 h elements, the shared expert's first.  A CTA
    // takes tiles blockIdx.x + k gridDim.x; of a tile, warp (j, sub) = (warp /
    // 4, warp % 4) takes the chunks j, j + 4, ... of gate rows 8 sub .. + 7
    // and the same up rows: mma rows g and g + 8 of a lane are one h element.
    const int sub = warp & 3, j = warp >> 2;
    const int per = j < chunks ? (chunks - j - 1) / 4 + 1 : 0;
    const int shared_tiles = a.Is / kFewTileRows, expert_tiles = a.I / kFewTileRows;
    int known = shared_tiles;  // tiles whose expert is known
    struct Tile {
        const uint8_t* w;
        const void* s;
        size_t row;  // this warp's first gate row in the matrix
        int I, u, i0;
    };
    auto tile = [&](int i) {
        Tile t;
        if (i < shared_tiles) {
            t.u = -1;
            t.i0 = i * kFewTileRows;
            t.I = a.Is;
            t.w = a.sh_w13;
            t.s = a.sh_s13;
            t.row = t.i0 + 8 * sub;
        } else {
            t.u = (i - shared_tiles) / expert_tiles;
            t.i0 = (i - shared_tiles - t.u * expert_tiles) * kFewTileRows;
            t.I = a.I;
            t.w = a.w13;
            t.s = a.s13;
            t.row = (size_t)P.expert[t.u] * 2 * a.I + t.i0 + 8 * sub;
        }
        return t;
    };
    int it = blockIdx.x, ic = j, ahead = 0;  // next copy; stages filled before the picks are known
    uint32_t dst = ring + stage_at(lane);
    const uint32_t dst_end = dst + kFewDepth * kStageBytes;
    const uint8_t* ip[4] = {};
    auto open_tile = [&]() {
        if (it >= known) return;
        const Tile t = tile(it);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (lane >> 3) + 4 * i;
            ip[i] = t.w + (t.row + (r < 8 ? r : t.I + r - 8)) * half + (lane & 7) * 16;
        }
    };
    auto issue = [&]() {
        if (it < known && per > 0) {
            issue_chunk(dst, ip, ic, ic * kChunkK + (lane & 7) * 32 < H);
            dst += kStageBytes;
            if (dst == dst_end) dst -= kFewDepth * kStageBytes;
            ++ahead;
            ic += 4;
            if (ic >= chunks) {
                ic = j;
                it += gridDim.x;
                open_tile();
            }
        }
        cp_async_commit();
    };
    open_tile();
    for (int i = 0; i < kFewDepth; ++i) issue();
    float nxt[4];  // the next chunk's scales, on their way while this one is multiplied
    ScaleRows sr;
    auto open_scales = [&](const Tile& t) {
        sr.open(t.s, t.row + g, t.row + t.I + g, a.G13, a.stype);
        if (per > 0) load_chunk_scales<kCoarse>(nxt, sr, j, a.gshift, a.G13, a.stype, q);
    };
    if ((int)blockIdx.x < shared_tiles) open_scales(tile(blockIdx.x));

    // Before the wait: the router's constants, and the tables' initial state.
    const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int epc = (a.E + size - 1) / size, e_lo = rank * epc, e_hi = min(a.E, e_lo + epc);
    if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started
    if (tid < a.E) s_bias[tid] = __ldg(a.rb + tid);
    if (tid < kMaxE / 32) s_mask[tid] = 0;
    // Unused entries name expert 0 and slot 0: of a workspace that two calls use
    // at once (which is not allowed) the down kernel may read a mix of their
    // tables, and sums that are wrong are better than addresses out of range.
    if (tid < kFewMaxU) P.tokens[tid] = 0, P.expert[tid] = 0;
    if (tid < kFewMaxU * kFewTok) P.slot[tid / kFewTok][tid % kFewTok] = 0;
    static_assert(kFewCluster <= 8, "a lane of eight per CTA");
    static_assert(kFewThreads >= kFewMaxU * kFewTok, "one slot a thread");
    // The dot products of this CTA's experts.  Of eight experts and fewer, with
    // rows of 16 blocks of 128 columns and more, 1 << plog warps share each one's
    // blocks (b_lo .. b_hi - 1 are this warp's); else a warp has experts of its
    // own.  Eight blocks of weights at a time, the next ones on their way.
    int plog = 0;
    while (H >= kFewShareMin && (epc << (plog + 1)) <= kFewWarps) ++plog;
    const int teams = kFewWarps >> plog, part = warp & ((1 << plog) - 1);
    const int b_lo = (H / 128 * part) >> plog, b_hi = (H / 128 * (part + 1)) >> plog;
    float4 wn[8];
    auto load_w = [&](int e, int b) {
        const float4* w = reinterpret_cast<const float4*>(a.rw + (size_t)e * H) + lane;
#pragma unroll
        for (int i = 0; i < 8; ++i) wn[i] = b + i < b_hi ? __ldg(w + (b + i) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    int e = a.lslices > 0 ? e_hi : e_lo + (warp >> plog);
    if (e < e_hi) load_w(e, b_lo);
    // Behind the logits kernel x is final: that kernel let this one start only
    // after its own wait for whatever wrote x.
    if (a.lslices > 0)
        quantize_tokens<kCoarse, true>(a.x, H, H, chunks, T, xq, xs_bytes, xs, 4 * NT, warp, kFewWarps, lane);
    pdl_wait();
    pdl_release();

    // x in shared memory, behind its int8 parts, for the logits
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(xq + 2 * T * xs_bytes);
    if (a.lslices == 0) {
        __nv_bfloat16* xr = const_cast<__nv_bfloat16*>(x);
        for (int i = tid; i < T * H / 8; i += kFewThreads)
            reinterpret_cast<uint4*>(xr)[i] = __ldcg(reinterpret_cast<const uint4*>(a.x) + i);
        __syncthreads();
    }
    if (size > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

    // Router logits of this CTA's experts, to every CTA of the cluster.
    if (a.lslices > 0) {
        for (int i = tid; i < T * a.E; i += kFewThreads) {  // no cluster then: every CTA sums all of them
            const float* l = a.lpart + i;
            float v = 0.f;
            for (int s0 = 0; s0 < a.lslices; s0 += 8) {  // eight loads on their way, whatever the count
                float p[8];
#pragma unroll
                for (int s = 0; s < 8; ++s) p[s] = s0 + s < a.lslices ? __ldcg(l + (size_t)(s0 + s) * T * a.E) : 0.f;
#pragma unroll
                for (int s = 0; s < 8; ++s) v += p[s];
            }
            s_logit[i / a.E][i % a.E] = v;
        }
    } else {
        float acc[4 * NT] = {};
        for (int b = b_lo; e < e_hi;) {
            float4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = wn[i];
            const int e_now = e, nb = min(8, b_hi - b);
            const uint2* xb = reinterpret_cast<const uint2*>(x + b * 128) + lane;
            b += 8;
            const bool last = b >= b_hi;
            if (last) {
                b = b_lo;
                e += teams;
            }
            if (e < e_hi) load_w(e, b);
            auto dot = [&](float& o, const uint2* xt) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint2 xv = i < nb ? xt[i * 32] : make_uint2(0, 0);
                    o = fmaf(bf16lo(xv.x), w[i].x, o);
                    o = fmaf(bf16hi(xv.x), w[i].y, o);
                    o = fmaf(bf16lo(xv.y), w[i].z, o);
                    o = fmaf(bf16hi(xv.y), w[i].w, o);
                }
            };
            // One or two tokens, or all 4 NT of the tile (past the last, it again):
            // independent chains instead of one after another.
            if (T == 1) {
                dot(acc[0], xb);
            } else if (T == 2) {
                dot(acc[0], xb);
                dot(acc[1], xb + H / 4);
            } else {
#pragma unroll
                for (int t = 0; t < 4 * NT; ++t) dot(acc[t], xb + (size_t)min(t, T - 1) * (H / 4));
            }
            if (!last) continue;
            // The 32 lanes' sums, lane pairs 16, 8, 4, 2, 1 apart in turn: for
            // four tokens at once the first two exchanges halve what a lane
            // holds, and lanes 8 t .. 8 t + 7 end with token t.
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float* v = acc + 4 * n;
                const bool up = lane & 16, odd = lane & 8;
                const float a0 = (up ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
                const float a1 = (up ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16);
                float s = (odd ? a1 : a0) + __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                const int t = 4 * n + (lane >> 3);
                if (plog == 0) {
                    if (t < T && (lane & 7) < size) *cluster.map_shared_rank(&s_logit[t][e_now], lane & 7) = s;
                } else if (t < T && (lane & 7) == 0) {
                    red[(((e_now - e_lo) << plog) + part) * kFewTok + t] = s;
                }
                v[0] = v[1] = v[2] = v[3] = 0.f;
            }
        }
        if (plog > 0) {  // added up, and sent to every CTA of the cluster
            __syncthreads();
            const int t = (tid >> 3) & 7, le = tid >> 6;
            static_assert(kFewTok == 8 && kFewCluster == 8 && kFewThreads >= 8 * 64, "a thread per token, rank and expert of eight");
            if (le < e_hi - e_lo && t < T && (tid & 7) < size) {
                float v = 0.f;
                for (int k = 0; k < 1 << plog; ++k) v += red[((le << plog) + k) * kFewTok + t];
                *cluster.map_shared_rank(&s_logit[t][e_lo + le], tid & 7) = v;
            }
        }
    }
    if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // int8 activations, while the cluster's other logits arrive
    if (a.lslices == 0)
        quantize_tokens<kCoarse, false>(x, H, H, chunks, T, xq, xs_bytes, xs, 4 * NT, warp, kFewWarps, lane);
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    __syncthreads();

    // Scores (a short loop: this code runs once a launch and is fetched cold)
    // and picks, a warp a token; then the tables.
    int my_e = -1;
    float my_w = 0.f;
    if (warp < T) {
        float* s = s_logit[warp];
#pragma unroll 2
        for (int i = lane; i < a.E; i += 32) s[i] = 1.0f / (1.0f + expf(-s[i]));
        __syncwarp();
        few_select(a, s_logit[warp], s_bias, lane, my_e, my_w);
        if (lane < a.K) {
            if (my_e >= 0) atomicOr(&s_mask[my_e >> 5], 1u << (my_e & 31));
            if (blockIdx.x == 0) {
                const int i = warp * a.K + lane;
                if (a.topk_idx_out) a.topk_idx_out[i] = my_e;
                if (a.topk_w_out) a.topk_w_out[i] = my_w;
            }
        }
        if (lane >= a.K) my_e = -1;
    }
    __syncthreads();
    if (my_e >= 0) {
        int u = __popc(s_mask[my_e >> 5] & ((1u << (my_e & 31)) - 1));
        for (int i = 0; i < (my_e >> 5); ++i) u += __popc(s_mask[i]);
        P.expert[u] = my_e;
        P.slot[u][warp] = (int8_t)(warp * a.K + lane);
        s_weight[u][warp] = my_w;
        atomicOr(&P.tokens[u], 1u << warp);
    }
    if (tid == kFewThreads - 1) {
        int n = 0;
        for (int i = 0; i < kMaxE / 32; ++i) n += __popc(s_mask[i]);
        P.U = n;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i < (int)(sizeof(FewPicks) / 4); i += kFewThreads)
            reinterpret_cast<int*>(a.picks)[i] = reinterpret_cast<const int*>(&P)[i];
    {  // the routed tiles are known now: fill the ring
        const bool was = it < known;
        known = shared_tiles + P.U * expert_tiles;
        if (!was) open_tile();
        // As many groups again as the first ones held no copy: the group of the
        // n-th stage is then never among the last kFewDepth - 1 when it is read.
        for (int i = ahead; i < kFewDepth; ++i) issue();
    }
    int slot = 0, parity = 0;
    Tile t;
    if ((int)blockIdx.x >= shared_tiles && (int)blockIdx.x < known) open_scales(tile(blockIdx.x));
    if ((int)blockIdx.x < known) t = tile(blockIdx.x);
    for (int i = blockIdx.x; i < known; i += gridDim.x, parity ^= 1) {
        Tile after = t;
        if (per == 0 && i + (int)gridDim.x < known) after = tile(i + gridDim.x);
        const unsigned tokens = t.u < 0 ? (1u << T) - 1 : P.tokens[t.u];
        const int passes = token_passes<NT>(tokens);
        uint32_t xrow[NT];
        const float* xsc[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            xrow[n] = smem_addr(xq + (2 * min(lane_token<NT>(tokens, g >> 1, n), T - 1) + (g & 1)) * xs_bytes);
            xsc[n] = xs + min(lane_token<NT>(tokens, q, n), T - 1);
        }
        float acc[NT][2] = {};
        for (int c = j; c < chunks; c += 4) {
            float sc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) sc[u] = nxt[u];
            scale_values(sc, a.stype);
            if (c + 4 < chunks) load_chunk_scales<kCoarse>(nxt, sr, c + 4, a.gshift, a.G13, a.stype, q);
            else if (i + (int)gridDim.x < known) open_scales(after = tile(i + gridDim.x));
            cp_async_wait<kFewDepth - 1>();
            __syncwarp();
            const uint32_t st = ring + slot * kStageBytes;
            slot = slot == kFewDepth - 1 ? 0 : slot + 1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= passes) break;
                const uint32_t xb[1] = {xrow[n] + c * kChunkK};
                float p[1][2];
                chunk_mma<1, kCoarse>(st, xb, sc, a.gshift, lane, p);
                const float s = xsc[n][c * 4 * NT];
                acc[n][0] = fmaf(p[0][0], s, acc[n][0]);
                acc[n][1] = fmaf(p[0][1], s, acc[n][1]);
            }
            __syncwarp();
            issue();
        }
        float* part = red + parity * kRed;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n > 0 && !((tokens >> q) & 1u)) continue;  // q + 4 had the first pass
            float* o = part + (warp * 4 * NT + lane_token<NT>(tokens, q, n)) * 16;
            o[g] = acc[n][0];
            o[g + 8] = acc[n][1];
        }
        __syncthreads();
        if (warp < T && ((tokens >> warp) & 1u)) {  // a warp per token, a lane per h element
            float gv = 0.f, uv = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float* o = part + ((k * 4 + (lane >> 3)) * 4 * NT + warp) * 16 + (lane & 7);
                gv += o[0];
                uv += o[8];
            }
            float h = silu_mul(gv, uv);
            if (t.u >= 0) h *= s_weight[t.u][warp];
            const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
            // block_scale of the magnitude rounded up to bf16's seven bits
            float s, inv;
            block_scale((m >> 16) + ((m & 0xffffu) != 0), &s, &inv);
            const uint32_t f = fixed16(h, inv);
            // eight columns in the order of lo8 / hi8; the eights of two blocks side by side (a lane's 16 bytes)
            const int at = (t.i0 & ~63) + (lane >> 3) * 16 + ((t.i0 >> 5) & 1) * 8 + ((lane & 1) << 2) + ((lane & 7) >> 1);
            const size_t base = t.u < 0 ? (size_t)T * a.K * 2 * a.I + (size_t)warp * 2 * a.Is
                                        : (size_t)P.slot[t.u][warp] * 2 * a.I;
            a.hq[base + at] = (int8_t)((f + 128) >> 8);
            a.hq[base + t.I + at] = (int8_t)f;
            if (lane == 0)
                a.hs[t.u < 0 ? (T * a.K * a.I + warp * a.Is + t.i0) / 32 : (P.slot[t.u][warp] * a.I + t.i0) / 32] = s * 0x1p-12f;
        }
        t = after;
    }
    cp_async_wait<0>();
}

// One staged chunk of w2 times one tile of four tokens: a block of 32 columns
// at a time, its sum times the token's own scale of the block (hv), the blocks
// of a scale group together times the rows' scales.
template <bool kCoarse>
__device__ __forceinline__ void down_mma(uint32_t stage, const uint4 (&x)[4], const float4 (&h4)[2], const float (&sc)[4],
                                         int gshift, int lane, float (&t)[2]) {
    const float hv[8] = {h4[0].x, h4[0].y, h4[0].z, h4[0].w, h4[1].x, h4[1].y, h4[1].z, h4[1].w};
    const int g = lane >> 2, q = lane & 3, quad = lane & 28;
    const uint32_t row = stage + g * 128 + (seg_perm(g) << 4) + q * 4;
    float u0 = 0.f, u8 = 0.f;
    t[0] = t[1] = 0.f;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint32_t at = row ^ (b << 4);
        const uint32_t wa = lds32(at), wb = lds32(at + 1024);
        const uint32_t a[4] = {lo8(wa), lo8(wb), hi8(wa), hi8(wb)};
        int d[4];
        mma_s8_first(d, a, (b & 1) ? x[b >> 1].z : x[b >> 1].x, (b & 1) ? x[b >> 1].w : x[b >> 1].y);
        u0 = fmaf((float)(d[0] * 256 + d[1]), hv[b], u0);
        u8 = fmaf((float)(d[2] * 256 + d[3]), hv[b], u8);
        const bool fine = !kCoarse && gshift == 5;
        if (kCoarse ? (b & 3) == 3 : fine || (b & 1)) {
            const int from = quad | (kCoarse ? b >> 2 : fine ? b & 3 : b >> 1);
            t[0] = fmaf(u0, __shfl_sync(0xffffffffu, fine ? sc[b >> 2] : sc[0], from), t[0]);
            t[1] = fmaf(u8, __shfl_sync(0xffffffffu, fine ? sc[2 + (b >> 2)] : sc[2], from), t[1]);
            u0 = u8 = 0.f;
        }
    }
}

struct Unit {  // 24 bytes: up to 2080 of them beside the rings (I = Is = 8192, 64 experts)
    const uint8_t* w;
    const char* s;
    int16_t u, I, G;
    uint8_t c, tokens;
};
static_assert(sizeof(Unit) == 24, "packed");

// Down projection of whole output tiles: 16 rows, the shared expert and all
// touched ones as one long sum, its chunks (units) dealt out to the CTA's
// warps: unit v to warp v mod kDownWarps, the shared expert's chunks first.
template <int NT, bool kCoarse>
__global__ void __launch_bounds__(kDownThreads, 1) few_down_kernel(FewArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ FewPicks P;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int T = a.T;
    constexpr int kRed = kDownWarps * 4 * NT * 16;
    float* red = reinterpret_cast<float*>(smem + kDownWarps * kDownDepth * kStageBytes);  // [2][warp][4 NT][16]
    const uint32_t ring = smem_addr(smem + warp * (kDownDepth * kStageBytes));
    const int Cs = (a.Is + kChunkK - 1) / kChunkK, Ci = (a.I + kChunkK - 1) / kChunkK;
    const int tiles = a.H / 16;
    int units = Cs;  // units of a tile, as far as they are known
    bool all = false;

    // Where unit v is, worked out once for all tiles: the byte of its first
    // code in the first row of w2 (or sh_w2), its first scale, the columns of
    // its row, its h, the tokens.  [units], behind the partial sums.
    Unit* list = reinterpret_cast<Unit*>(red + 2 * kRed);
    auto describe = [&](int v) {
        Unit d;
        const bool sh = v < Cs;
        const int u = sh ? -1 : (v - Cs) / Ci, c = sh ? v : v - Cs - u * Ci;
        // in range whatever the table holds (see few_gate_up_kernel)
        const size_t row = sh ? 0 : (size_t)min((unsigned)P.expert[u], (unsigned)a.E - 1) * a.H;
        d.I = (int16_t)(sh ? a.Is : a.I);
        d.G = (int16_t)(sh ? a.Gs2 : a.G2);
        d.w = (sh ? a.sh_w2 : a.w2) + row * (d.I / 2) + c * (kChunkK / 2);
        d.s = static_cast<const char*>(sh ? a.sh_s2 : a.s2) + ((row * d.G) << (a.stype == kScaleF32 ? 2 : 1));
        d.u = (int16_t)u;
        d.c = (uint8_t)c;
        d.tokens = (uint8_t)(sh ? (1u << T) - 1 : max(P.tokens[u], 1u));
        return d;
    };
    for (int v = tid; v < Cs; v += kDownThreads) list[v] = describe(v);
    __syncthreads();

    int iv = warp, it = blockIdx.x, ahead = 0;  // next copy: unit and tile; stages filled before the picks are known
    uint32_t dst = ring + stage_at(lane);
    const uint32_t dst_end = dst + kDownDepth * kStageBytes;
    auto issue = [&]() {
        if (it < tiles && iv < units) {
            const Unit& d = list[iv];
            const int half = d.I / 2;
            const uint8_t* ip[4];
            ip[0] = d.w + (size_t)(it * 16 + (lane >> 3)) * half + (lane & 7) * 16;
#pragma unroll
            for (int i = 1; i < 4; ++i) ip[i] = ip[i - 1] + 4 * half;
            issue_chunk(dst, ip, 0, d.c * kChunkK + (lane & 7) * 32 < d.I);
            dst += kStageBytes;
            if (dst == dst_end) dst -= kDownDepth * kStageBytes;
            ++ahead;
            iv += kDownWarps;
            if (all && iv >= units) {
                iv = warp;
                it += gridDim.x;
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < kDownDepth; ++i) issue();
    // The rows' scales come from HBM and are loaded a unit ahead; h comes from L2.
    float nsc[4];
    const int esh = a.stype == kScaleF32 ? 2 : 1;
    auto load_scales = [&](int v, int i) {
        const Unit& d = list[v];
        ScaleRows sr;
        sr.p0 = d.s + (((i * 16 + g) * d.G) << esh);
        sr.p8 = sr.p0 + ((8 * d.G) << esh);
        load_chunk_scales<kCoarse>(nsc, sr, d.c, a.gshift, d.G, a.stype, q);
    };
    if (warp < Cs && (int)blockIdx.x < tiles) load_scales(warp, blockIdx.x);

    pdl_wait();
    pdl_release();
    for (int i = tid; i < (int)(sizeof(FewPicks) / 4); i += kDownThreads)
        reinterpret_cast<int*>(&P)[i] = __ldcg(reinterpret_cast<const int*>(a.picks) + i);
    __syncthreads();
    units = Cs + max(min(P.U, min(a.E, T * a.K)), 0) * Ci;
    for (int v = Cs + tid; v < units; v += kDownThreads) list[v] = describe(v);
    __syncthreads();
    all = true;
    if (iv >= units && warp < units) {
        iv = warp;
        it += gridDim.x;
    }
    for (int i = ahead; i < kDownDepth; ++i) issue();  // see few_gate_up_kernel

    const int8_t* hq_shared = a.hq + (size_t)T * a.K * 2 * a.I;
    const float* hs_shared = a.hs + T * a.K * a.I / 32;
    int slot = 0, parity = 0;
    // This lane's B row (the token of column pair g / 2, part g % 2) and the
    // block scales of its D columns (column pair q).  A column without a token
    // takes the first token's: its sums are not used.
    auto load_h = [&](const Unit& d, unsigned tokens, int n, uint4 (&x)[4], float4 (&hv)[2]) {
        const int any = __ffs((int)tokens) - 1;
        int sb = lane_token<NT>(tokens, g >> 1, n), sd = lane_token<NT>(tokens, q, n);
        if (!((tokens >> sb) & 1u)) sb = any;
        if (!((tokens >> sd) & 1u)) sd = any;
        if (d.u >= 0) {
            sb = P.slot[d.u][sb];
            sd = P.slot[d.u][sd];
        }
        const uint4* xp = reinterpret_cast<const uint4*>((d.u < 0 ? hq_shared : a.hq) + (2 * sb + (g & 1)) * d.I + d.c * kChunkK) + q;
        const float4* hp = reinterpret_cast<const float4*>((d.u < 0 ? hs_shared : a.hs) + (sd * d.I + d.c * kChunkK) / 32);
        x[0] = __ldcg(xp);
        x[1] = __ldcg(xp + 4);
        hv[0] = __ldcg(hp);
        if (d.c * kChunkK + 128 < d.I) {
            x[2] = __ldcg(xp + 8);
            x[3] = __ldcg(xp + 12);
            hv[1] = __ldcg(hp + 1);
        } else {  // half a chunk: the rest of the stage is not its row's
            x[2] = x[3] = make_uint4(0, 0, 0, 0);
            hv[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    if (warp >= Cs && warp < units && (int)blockIdx.x < tiles) load_scales(warp, blockIdx.x);
    for (int i = blockIdx.x; i < tiles; i += gridDim.x, parity ^= 1) {
        float acc[NT][2] = {};
        for (int v = warp; v < units; v += kDownWarps) {
            const Unit& d = list[v];
            const unsigned tokens = d.tokens;
            uint4 x[4];
            float4 hv[2];
            const int passes = token_passes<NT>(tokens);
            load_h(d, tokens, 0, x, hv);
            float sc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) sc[u] = nsc[u];
            if (v + kDownWarps < units) load_scales(v + kDownWarps, i);
            else if (i + (int)gridDim.x < tiles) load_scales(warp, i + gridDim.x);
            scale_values(sc, a.stype);
            cp_async_wait<kDownDepth - 1>();
            __syncwarp();
            const uint32_t st = ring + slot * kStageBytes;
            slot = slot == kDownDepth - 1 ? 0 : slot + 1;
#pragma unroll 1
            for (int n = 0;;) {
                float t[2];
                down_mma<kCoarse>(st, x, hv, sc, a.gshift, lane, t);
                const int tok = lane_token<NT>(tokens, q, n);
                if (((tokens >> tok) & 1u) && (n == 0 || ((tokens >> q) & 1u))) {  // else: none, or pass 0 had it
                    if (NT == 1 || tok < 4) {
                        acc[0][0] += t[0];
                        acc[0][1] += t[1];
                    } else {
                        acc[NT - 1][0] += t[0];
                        acc[NT - 1][1] += t[1];
                    }
                }
                if (NT == 1 || ++n == passes) break;
                load_h(d, tokens, n, x, hv);
            }
            __syncwarp();
            issue();
        }
        float* part = red + parity * kRed;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float* o = part + (warp * 4 * NT + 4 * n + q) * 16;
            o[g] = acc[n][0];
            o[g + 8] = acc[n][1];
        }
        __syncthreads();
        if (tid < 16 * T) {
            const int r = tid & 15, t = tid >> 4;
            const size_t o = (size_t)t * a.H + i * 16 + r;
            float v = a.flags & kFlagResidual ? bf16lo(__ldcg(reinterpret_cast<const unsigned short*>(a.x) + o)) : 0.f;
            float y = 0.f;
#pragma unroll
            for (int w = 0; w < kDownWarps; ++w) y += part[(w * 4 * NT + t) * 16 + r];
            v += y;
            if (a.flags & kFlagOutF32) static_cast<float*>(a.out)[o] = v;
            else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
        }
    }
    cp_async_wait<0>();
}

namespace {

// SMs of the current device, and the CTAs of the gate/up kernel that run at
// once in clusters of kFewCluster.
struct FewDevice {
    std::atomic<int> sms, clustered;  // clustered = 0: not asked yet; written last
};

cudaError_t few_launch_cluster(void (*k)(FewArgs), int grid, int cluster, size_t smem, cudaStream_t stream, const FewArgs& a,
                               int* max_clusters) {
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(kFewThreads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    if (max_clusters) {
        c.attrs = at + 1;
        c.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(max_clusters, k, &c);
    }
    return cudaLaunchKernelEx(&c, k, a);
}

template <int NT, bool kCoarse>
cudaError_t few_launch(const FewArgs& a, cudaStream_t stream) {
    auto* up = few_gate_up_kernel<NT, kCoarse>;
    auto* down = few_down_kernel<NT, kCoarse>;
    static FewDevice devs[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    FewDevice& d = devs[dev];
    if (d.clustered == 0) {
        int n = 0, sms = 0;
        e = cudaFuncSetAttribute(up, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewDynMax);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewDynMax);
        if (e == cudaSuccess) e = few_launch_cluster(up, kFewCluster, kFewCluster, kFewDynMax, nullptr, a, &n);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        d.sms = sms;
        d.clustered = n * kFewCluster;
    }
    const size_t smem = few_smem(NT, a.T, a.H, x_stride<kCoarse>((a.H + kChunkK - 1) / kChunkK), a.lslices > 0);
    const int sms = d.sms, clustered = d.clustered;
    const int cluster = a.lslices > 0 ? 1 : kFewCluster, most = a.lslices > 0 ? sms : clustered;
    const int tiles = few_tiles(a);
    int grid = (tiles + cluster - 1) / cluster * cluster;
    if (grid > most) grid = most;
    e = few_launch_cluster(up, grid, cluster, smem, stream, a, nullptr);
    const int out_tiles = a.H / 16;
    const size_t units = (a.Is + kChunkK - 1) / kChunkK + (size_t)few_touched(a) * ((a.I + kChunkK - 1) / kChunkK);
    const size_t smem_down = (size_t)kDownWarps * kDownDepth * kStageBytes + 2 * (size_t)kDownWarps * 4 * NT * 16 * 4 +
                             units * sizeof(Unit);
    if (e == cudaSuccess)
        e = launch_pdl(down, dim3(out_tiles < sms ? out_tiles : sms), dim3(kDownThreads),
                       smem_down, stream, a);
    return e;
}

}  // namespace

int few_pass_tokens(const FewArgs& a) {
    const int fit = kFewXMax / (2 * x_stride<true>((a.H + kChunkK - 1) / kChunkK));
    return fit < kFewTok ? fit : kFewTok;
}

int few_pass_launches(const FewArgs& a) { return few_split_router(a) ? 3 : 2; }

size_t few_workspace(FewArgs& a, void* ws) {
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? static_cast<char*>(ws) + o : nullptr;
        o = (o + bytes + 255) & ~size_t(255);
        return p;
    };
    const size_t TK = (size_t)a.T * a.K, n = TK * a.I + (size_t)a.T * a.Is;
    a.picks = reinterpret_cast<FewPicks*>(take(sizeof(FewPicks)));
    a.hq = reinterpret_cast<int8_t*>(take(2 * n));
    a.hs = reinterpret_cast<float*>(take(n / 32 * 4));
    a.lslices = few_split_router(a) ? few_logit_slices(a.H) : 0;
    a.lpart = reinterpret_cast<float*>(take((size_t)a.lslices * a.T * a.E * 4));
    return o;
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t stream) {
    if (a.lslices > 0) {
        Params p = {};
        p.T = a.T;
        p.H = a.H;
        p.E = a.E;
        p.x = a.x;
        p.rw = a.rw;
        p.lpart = a.lpart;
        p.lslices = a.lslices;
        const cudaError_t e = launch_router_logits(p, stream);
        if (e != cudaSuccess) return e;
    }
    const bool coarse = a.gshift >= 7;
    if (a.T <= 4) return coarse ? few_launch<1, true>(a, stream) : few_launch<1, false>(a, stream);
    return coarse ? few_launch<2, true>(a, stream) : few_launch<2, false>(a, stream);
}

}  // namespace moe
