// A whole MoE layer for a few tokens, with group-scaled int4 weights.
#include "group_int4.h"

namespace moe {

__device__ __forceinline__ float few_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Routing of one token (one CTA): logits, scores, the K largest keys.
__global__ void __launch_bounds__(256) few_route_kernel(FewArgs a) {
    __shared__ float s_score[kMaxE], s_key[kMaxE];
    const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_release();
    for (int e = warp; e < a.E; e += 8) {
        float acc = 0.f;
        for (int h = lane; h < a.H; h += 32)
            acc = fmaf(__bfloat162float(a.x[(size_t)t * a.H + h]), __ldg(a.rw + (size_t)e * a.H + h), acc);
        acc = few_sum(acc);
        if (lane == 0) {
            const float s = 1.0f / (1.0f + expf(-acc)), k = s + a.rb[e];
            s_score[e] = s;
            s_key[e] = isnan(k) ? -INFINITY : k;
        }
    }
    __syncthreads();
    if (warp != 0) return;
    unsigned taken = 0;
    int my_e = -1;
    float my_s = 0.f, ssum = 0.f;
    for (int k = 0; k < a.K; ++k) {
        float bk = -INFINITY;
        int be = 0x7fffffff;
        for (int j = 0; j < kMaxE / 32; ++j) {
            const int e = lane + 32 * j;
            if (e < a.E && !((taken >> j) & 1u) && (s_key[e] > bk || (s_key[e] == bk && e < be))) { bk = s_key[e]; be = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const float ok = __shfl_xor_sync(0xffffffffu, bk, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (ok > bk || (ok == bk && oe < be)) { bk = ok; be = oe; }
        }
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        if (lane == k) { my_e = be; my_s = s_score[be]; }
        ssum += s_score[be];
    }
    int oe;
    float ow;
    topp_picks(a.K, a.topp, a.scale, lane, my_e, my_s, ssum, oe, ow);
    if (lane < a.K) {
        const size_t o = (size_t)t * a.K + lane;
        a.idx[o] = oe;
        a.wts[o] = ow;
        if (a.topk_idx_out) a.topk_idx_out[o] = oe;
        if (a.topk_w_out) a.topk_w_out[o] = ow;
    }
}

// sum_k v[k] c[k] s[k / group] over one weight row (one warp): lane l takes
// the words (eight codes) l, l + 32, ...
template <typename V>
__device__ __forceinline__ float few_row(const uint8_t* w, const void* s, size_t s0, int gshift, int stype, int n, V v) {
    const int lane = threadIdx.x & 31;
    float acc = 0.f;
    for (int i = lane; i < n / 8; i += 32) {
        const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(w) + i);
        float p = 0.f;
        for (int j = 0; j < 8; ++j) p = fmaf((float)((int)(c << (28 - 4 * j)) >> 28), v(8 * i + j), p);
        acc = fmaf(load_scale(s, s0 + ((8 * i) >> gshift), stype), p, acc);
    }
    return few_sum(acc);
}

// h of one pick (or of the shared expert, blockIdx.y = K) of token blockIdx.z: a warp per element.
__global__ void __launch_bounds__(256) few_gate_up_kernel(FewArgs a) {
    const int t = blockIdx.z, k = blockIdx.y, lane = threadIdx.x & 31;
    const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_release();
    const bool sh = k == a.K;
    const int I = sh ? a.Is : a.I, e = sh ? 0 : a.idx[(size_t)t * a.K + k];
    if (i >= I || e < 0) return;
    const uint8_t* w = sh ? a.sh_w13 : a.w13 + (size_t)e * 2 * I * (a.H / 2);
    const void* s = sh ? a.sh_s13 : a.s13;
    const size_t r0 = sh ? 0 : (size_t)e * 2 * I;
    const __nv_bfloat16* x = a.x + (size_t)t * a.H;
    auto v = [&](int h) { return __bfloat162float(x[h]); };
    const float g = few_row(w + (size_t)i * (a.H / 2), s, (r0 + i) * a.G13, a.gshift, a.stype, a.H, v);
    const float u = few_row(w + (size_t)(I + i) * (a.H / 2), s, (r0 + I + i) * a.G13, a.gshift, a.stype, a.H, v);
    if (lane == 0) {
        float* h = sh ? a.h + (size_t)a.T * a.K * a.I + (size_t)t * I : a.h + ((size_t)t * a.K + k) * I;
        h[i] = silu_mul(g, u);
    }
}

// One output element: a warp.
__global__ void __launch_bounds__(256) few_down_kernel(FewArgs a) {
    const int t = blockIdx.y, lane = threadIdx.x & 31;
    const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_release();
    if (j >= a.H) return;
    float y = 0.f;
    for (int k = 0; k < a.K; ++k) {
        const int e = a.idx[(size_t)t * a.K + k];
        if (e < 0) continue;
        const float* h = a.h + ((size_t)t * a.K + k) * a.I;
        const size_t r = (size_t)e * a.H + j;
        y = fmaf(a.wts[(size_t)t * a.K + k],
                 few_row(a.w2 + r * (a.I / 2), a.s2, r * a.G2, a.gshift, a.stype, a.I, [&](int i) { return h[i]; }), y);
    }
    if (a.Is > 0) {
        const float* h = a.h + (size_t)a.T * a.K * a.I + (size_t)t * a.Is;
        y += few_row(a.sh_w2 + (size_t)j * (a.Is / 2), a.sh_s2, (size_t)j * a.Gs2, a.gshift, a.stype, a.Is,
                     [&](int i) { return h[i]; });
    }
    if (lane) return;
    const size_t o = (size_t)t * a.H + j;
    if (a.flags & kFlagResidual) y += __bfloat162float(a.x[o]);
    if (a.flags & kFlagOutF32) static_cast<float*>(a.out)[o] = y;
    else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
}

int few_pass_tokens(const FewArgs&) { return 8; }
int few_pass_launches(const FewArgs&) { return 3; }

size_t few_workspace(FewArgs& a, void* ws) {
    size_t o = 0;
    auto take = [&](size_t bytes) {
        char* p = ws ? static_cast<char*>(ws) + o : nullptr;
        o = (o + bytes + 255) & ~size_t(255);
        return p;
    };
    const size_t TK = (size_t)a.T * a.K;
    a.idx = reinterpret_cast<int32_t*>(take(TK * 4));
    a.wts = reinterpret_cast<float*>(take(TK * 4));
    a.h = reinterpret_cast<float*>(take((TK * a.I + (size_t)a.T * a.Is) * 4));
    return o;
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t stream) {
    cudaError_t e = launch_pdl(few_route_kernel, dim3(a.T), dim3(256), 0, stream, a);
    const int im = a.Is > a.I ? a.Is : a.I;
    if (e == cudaSuccess)
        e = launch_pdl(few_gate_up_kernel, dim3((im + 7) / 8, a.K + (a.Is > 0), a.T), dim3(256), 0, stream, a);
    if (e == cudaSuccess) e = launch_pdl(few_down_kernel, dim3((a.H + 7) / 8, a.T), dim3(256), 0, stream, a);
    return e;
}

}  // namespace moe
