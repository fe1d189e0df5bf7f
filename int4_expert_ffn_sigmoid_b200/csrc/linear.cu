// Dense projection with int4 weights and group scales:
//   out[t][n] = sum_k x[t][k] c[n][k] s[n][k / group]  (+ add[t][n]).
#include "group_int4.h"

namespace moe {

// Elements of word w of codes, in order.
__device__ __forceinline__ float code_of(uint32_t w, int j) { return (float)((int)(w << (28 - 4 * j)) >> 28); }

// A warp per output row, eight tokens at a time, f32 multiply-adds: lane l
// takes the words (eight codes) l, l + 32, ... of the row.
constexpr int kRowWarps = 8, kRowTok = 8;

__global__ void __launch_bounds__(32 * kRowWarps) linear_row_kernel(LinearArgs a) {
    const int lane = threadIdx.x & 31;
    const long long n = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_release();
    if (n >= a.N) return;
    const uint32_t* wr = reinterpret_cast<const uint32_t*>(a.w + (size_t)n * (a.K / 2));
    for (long long t0 = (long long)blockIdx.y * kRowTok; t0 < a.T; t0 += (long long)gridDim.y * kRowTok) {
        float acc[kRowTok] = {};
        for (int i = lane; i < a.K / 8; i += 32) {
            const uint32_t w = __ldg(wr + i);
            const float s = load_scale(a.scales, (size_t)n * a.G + ((8 * i) >> a.gshift), a.stype);
#pragma unroll
            for (int u = 0; u < kRowTok; ++u) {
                if (t0 + u >= a.T) break;
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(a.x + (t0 + u) * a.ldx) + i);
                const uint32_t xs[4] = {v.x, v.y, v.z, v.w};
                float p = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p = fmaf(code_of(w, 2 * j), bf16lo(xs[j]), p);
                    p = fmaf(code_of(w, 2 * j + 1), bf16hi(xs[j]), p);
                }
                acc[u] = fmaf(s, p, acc[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kRowTok; ++u) {
            if (t0 + u >= a.T) break;
            float v = acc[u];
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) {
                if (a.add) v += __bfloat162float(a.add[(t0 + u) * a.lda + n]);
                if (a.out_f32) static_cast<float*>(a.out)[(t0 + u) * a.ldo + n] = v;
                else static_cast<__nv_bfloat16*>(a.out)[(t0 + u) * a.ldo + n] = __float2bfloat16_rn(v);
            }
        }
    }
}

int linear_launches(const LinearArgs&) { return 1; }

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream) {
    const int gy = (a.T + kRowTok - 1) / kRowTok;
    return launch_pdl(linear_row_kernel, dim3((a.N + kRowWarps - 1) / kRowWarps, gy < 65535 ? gy : 65535),
                      dim3(32 * kRowWarps), 0, stream, a);
}

}  // namespace moe
