// Dense projection with int4 weights and group scales:
//   out[t][n] = sum_k x[t][k] c[n][k] s[n][k / group]  (+ add[t][n]).
#include "group_stream.cuh"

namespace moe {

// Weight streaming for up to eight tokens.  A CTA takes tiles of 16 * wr rows;
// its warps are wr teams of wk, warp (team, j) multiplying the chunks j, j +
// wk, ... of its team's 16 rows (chunk_mma) and the team's partial sums
// meeting in shared memory.  Each warp runs its own ring of kDepth staged
// chunks on cp.async (no barrier with another warp), across tile borders, and
// fills it before waiting on the previous kernel: weights and scales are
// constants, x and add are not.
//
// What bounds it: the weights' bytes where there are many (one token x 49152 x
// 6144: 27.3 us, 88 % of the copy rate), a fixed 4 us of launch, rounding of x,
// ring fill and drain where there are few (6144 x 6144: 6.5 us, 3.0 at the copy
// rate; 1024 x 1024: 2.0), and from three tokens on the instructions of the
// integer products and their scaling (four tokens x 12288 x 6144: 13.8 us, 7.3
// at the copy rate).  A ring of two or four stages is no faster than three.
constexpr int kDepth = 3;
// Dynamic shared memory of one CTA at most, and of the activations alone
// (eight tokens of 7168 columns).
constexpr int kSmemMax = 227 * 1024;
constexpr int kXMax = 113 * 1024;

struct StreamPlan {
    int wk_log, wr_log;  // warps along the columns, teams: 1 << each
    int chunks, tiles;   // 256-column chunks of a row; CTA tiles of 16 rows a team
};

template <int NW>
__host__ __device__ constexpr int red_floats(int ntok) {
    return NW * 16 * ntok;
}

template <int NW, int NT, bool kCoarse>
__global__ void __launch_bounds__(32 * NW, NW == 8 ? (NT == 1 ? 3 : 2) : 1) linear_stream_kernel(LinearArgs a, StreamPlan p) {
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wk = 1 << p.wk_log, team = warp >> p.wk_log, j = warp & (wk - 1);
    const int g = lane >> 2, q = lane & 3;
    const int xs_bytes = x_stride<kCoarse>(p.chunks);
    float* red = reinterpret_cast<float*>(smem + NW * kDepth * kStageBytes);  // [2][NW][4 NT][16]
    float* xs = red + 2 * red_floats<NW>(4 * NT);                            // [chunks][4 NT]
    int8_t* xq = reinterpret_cast<int8_t*>(xs + p.chunks * 4 * NT);          // [token][part][xs_bytes]
    const uint32_t ring = smem_addr(smem + warp * (kDepth * kStageBytes));

    // this warp's chunks, tile after tile
    const int per = j < p.chunks ? ((p.chunks - j - 1) >> p.wk_log) + 1 : 0;
    const int tiles = p.tiles > (int)blockIdx.x ? (p.tiles - blockIdx.x - 1) / gridDim.x + 1 : 0;
    const int rows_cta = 16 << p.wr_log, last = a.N - 1, half = a.K / 2;
    int left = per * tiles;  // copies to issue
    int ir = blockIdx.x * rows_cta + team * 16, ic = j;  // row and chunk of the next copy
    uint32_t dst = ring + stage_at(lane);
    const uint32_t dst_end = dst + kDepth * kStageBytes;
    const uint8_t* ip[4];
    auto open_tile = [&]() {  // rows past the last repeat it: their sums are not stored
#pragma unroll
        for (int i = 0; i < 4; ++i) ip[i] = a.w + (size_t)min(ir + (lane >> 3) + 4 * i, last) * half + (lane & 7) * 16;
    };
    auto issue = [&]() {
        if (left > 0) {
            --left;
            issue_chunk(dst, ip, ic, ic * kChunkK + (lane & 7) * 32 < a.K);
            dst += kStageBytes;
            if (dst == dst_end) dst -= kDepth * kStageBytes;
            ic += wk;
            if (ic >= p.chunks) {
                ic = j;
                ir += rows_cta * gridDim.x;
                open_tile();
            }
        }
        cp_async_commit();
    };
    float nxt[4];
    ScaleRows sr;
    auto open_scales = [&](int row) { sr.open(a.scales, min(row + g, last), min(row + g + 8, last), a.G, a.stype); };
    auto scales = [&](int c) { load_chunk_scales<kCoarse>(nxt, sr, c, a.gshift, a.G, a.stype, q); };
    int row = ir;
    open_tile();
    for (int i = 0; i < kDepth; ++i) issue();
    open_scales(row);
    if (per > 0 && tiles > 0) scales(j);
    pdl_wait();
    pdl_release();

    quantize_tokens<kCoarse, true>(a.x, a.ldx, a.K, p.chunks, a.T, xq, xs_bytes, xs, 4 * NT, warp, NW, lane);
    __syncthreads();

    uint32_t xrow[NT];  // a column past the last token repeats it: its sums are not stored
    const float* xsc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = min(4 * n + (g >> 1), a.T - 1);
        xrow[n] = smem_addr(xq + (2 * t + (g & 1)) * xs_bytes);
        xsc[n] = xs + min(4 * n + q, a.T - 1);
    }
    int slot = 0;
    // Output o of a tile: its row o mod rows_cta, token o / rows_cta.
    const int outs = a.T * rows_cta;
    auto place = [&](int o, int& t, int& n) {
        t = o >> (4 + p.wr_log);
        n = row - team * 16 + (o & (rows_cta - 1));
        return n < a.N;
    };
    // from L2, as x: the kernel before this one may have written it
    auto addend = [&](int t, int n) { return bf16lo(__ldcg(reinterpret_cast<const unsigned short*>(a.add) + t * a.lda + n)); };
    for (int i = 0; i < tiles; ++i, row += rows_cta * gridDim.x) {
        float plus = 0.f;  // what the thread's first output is added to: on its way during the products
        if (a.add && tid < outs) {
            int t, n;
            if (place(tid, t, n)) plus = addend(t, n);
        }
        float acc[NT][2] = {};
        for (int c = j; c < p.chunks; c += wk) {
            float sc[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) sc[u] = nxt[u];
            scale_values(sc, a.stype);
            if (c + wk < p.chunks) {
                scales(c + wk);
            } else if (i + 1 < tiles) {
                open_scales(row + rows_cta * gridDim.x);
                scales(j);
            }
            cp_async_wait<kDepth - 1>();
            __syncwarp();
            uint32_t xb[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xb[n] = xrow[n] + c * kChunkK;
            float t[NT][2];
            chunk_mma<NT, kCoarse>(ring + slot * kStageBytes, xb, sc, a.gshift, lane, t);
            slot = slot == kDepth - 1 ? 0 : slot + 1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float s = xsc[n][c * 4 * NT];
                acc[n][0] = fmaf(t[n][0], s, acc[n][0]);
                acc[n][1] = fmaf(t[n][1], s, acc[n][1]);
            }
            __syncwarp();
            issue();
        }
        float* part = red + (i & 1) * red_floats<NW>(4 * NT);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float* o = part + (warp * 4 * NT + 4 * n + q) * 16;
            o[g] = acc[n][0];
            o[g + 8] = acc[n][1];
        }
        __syncthreads();
        for (int o = tid; o < outs; o += 32 * NW) {
            int t, n;
            if (!place(o, t, n)) continue;
            const int tm = (o & (rows_cta - 1)) >> 4;
            float v = 0.f;
            for (int u = 0; u < wk; ++u) v += part[(((tm << p.wk_log) + u) * 4 * NT + t) * 16 + (o & 15)];
            if (a.add) v += o == tid ? plus : addend(t, n);
            if (a.out_f32) static_cast<float*>(a.out)[t * a.ldo + n] = v;
            else static_cast<__nv_bfloat16*>(a.out)[t * a.ldo + n] = __float2bfloat16_rn(v);
        }
    }
    cp_async_wait<0>();
}

namespace {

int sms() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    if (cache[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
        cache[dev] = n;
    }
    return cache[dev];
}

template <int NW, int NT>
size_t stream_smem(const LinearArgs& a) {
    const int chunks = (a.K + kChunkK - 1) / kChunkK;
    return (size_t)NW * kDepth * kStageBytes + 2 * red_floats<NW>(4 * NT) * 4 + (size_t)chunks * 4 * NT * 4 +
           (size_t)a.T * 2 * (a.gshift >= 7 ? x_stride<true>(chunks) : x_stride<false>(chunks));
}

template <int NW, int NT, bool kCoarse>
cudaError_t launch_stream(const LinearArgs& a, StreamPlan p, cudaStream_t stream) {
    const size_t smem = stream_smem<NW, NT>(a);
    auto* k = linear_stream_kernel<NW, NT, kCoarse>;
    static std::atomic<int> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 && !set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e != cudaSuccess) return e;
        set[dev] = 1;
    }
    p.tiles = (a.N + (16 << p.wr_log) - 1) >> (4 + p.wr_log);
    const int grid = p.tiles < sms() ? p.tiles : sms();
    return launch_pdl(k, dim3(grid), dim3(32 * NW), smem, stream, a, p);
}

template <int NW, int NT>
cudaError_t launch_stream(const LinearArgs& a, const StreamPlan& p, cudaStream_t stream) {
    return a.gshift >= 7 ? launch_stream<NW, NT, true>(a, p, stream) : launch_stream<NW, NT, false>(a, p, stream);
}

// Up to eight tokens stream where their activations fit; the rest goes to the
// tensor memory GEMM.  Here and there, us: eight tokens x 6144 x 6144 11.1, 12.3;
// x 12288 x 6144 13.9, 19.7; x 1024 x 1024 2.5, 3.6; nine x 2048 x 2048 4.4, 4.0;
// 12 x 12288 x 2048 9.1, 8.4.  A GEMM as accurate for eight tokens (see
// linear_gemm.cu) is no faster but for a few hundred rows: eight x 512 x 6144
// 7.4, 6.4; x 1024 x 6144 7.4, 8.0; x 2048 x 6144 7.8, 9.6; five x 512 x 6144 6.1, 6.5.
bool streams(const LinearArgs& a) {
    return a.T <= kStreamTok && a.T * 2 * x_stride<true>((a.K + kChunkK - 1) / kChunkK) <= kXMax;
}

}  // namespace

int linear_launches(const LinearArgs&) { return 1; }

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
    if (!streams(a)) return launch_linear_gemm(a, stream);
    StreamPlan p = {};
    p.chunks = (a.K + kChunkK - 1) / kChunkK;
    while (p.wk_log < 3 && (1 << p.wk_log) < p.chunks) ++p.wk_log;
    auto teams = [&](int warps) {
        p.wr_log = (warps == 8 ? 3 : 4) - p.wk_log;
        return p;
    };
    // 16 rows an SM: eight warps a CTA, the finest tiles, and room for the next
    // launch to start beside it (1024 x 1024, one token 2.0 us against 2.2 with 16
    // warps, four 2.2 and 2.5, eight 2.5 and 3.1; one x 512 x 6144 3.2 and 3.7).
    // Otherwise 16 warps share the rounding of x (4096 x 6144: 5.1 us against 5.8;
    // two tokens x 6144 x 6144 6.8 and 8.5; four tokens x 12288 x 6144 13.8, and
    // 14.3 with 24 warps, which leave 80 registers a thread).
    const bool few_rows = a.N <= 16 * sms();
    if (a.T <= 4) {
        if (few_rows && 3 * stream_smem<8, 1>(a) <= kSmemMax - 3 * 1024) return launch_stream<8, 1>(a, teams(8), stream);
        return launch_stream<16, 1>(a, teams(16), stream);
    }
    if (few_rows && 2 * stream_smem<8, 2>(a) <= kSmemMax - 2 * 1024) return launch_stream<8, 2>(a, teams(8), stream);
    return launch_stream<16, 2>(a, teams(16), stream);
}

}  // namespace moe
