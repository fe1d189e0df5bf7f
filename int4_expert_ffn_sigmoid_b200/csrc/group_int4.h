// Operators on int4 weights with group scales (internal): the arguments of
// their kernels and the host-side launch entry points.
#pragma once

#include <cuda_runtime.h>

#include "moe_common.cuh"

namespace moe {

// Scale types (the MOE_SCALE_* values of the C ABI).
constexpr int kScaleF32 = 0, kScaleBf16 = 1, kScaleF16 = 2;

// Tokens of a projection that weight streaming takes at most.
constexpr int kStreamTok = 8;

// log2 of the columns per scale; kRowGroup: one scale a row (k >> kRowGroup
// is 0 for every column).
constexpr int kRowGroup = 31;

struct LinearArgs {
    const __nv_bfloat16* x;
    const uint8_t* w;
    const void* scales;
    const __nv_bfloat16* add;  // or null
    void* out;
    int T, N, K;
    int gshift, G;  // columns per scale: 1 << gshift; scales per row
    int stype, out_f32;
    int full;   // MOE_FULL_WEIGHTS
    int stall;  // MOE_TEST_STALL
    long long ldx, ldo, lda;
};

// What the picks of a pass of the few-token layer come to.
constexpr int kFewTok = 8;  // tokens of a pass at most
constexpr int kFewMaxU = kFewTok * kMaxK;
struct FewPicks {
    int U;                           // touched experts
    int expert[kFewMaxU];            // ascending
    unsigned tokens[kFewMaxU];       // bit t: token t picked it
    int8_t slot[kFewMaxU][kFewTok];  // t * K + k of token t's pick of the expert (0 where it has none)
};

struct FewArgs {
    const __nv_bfloat16* x;
    const float* rw;
    const float* rb;
    const uint8_t *w13, *w2, *sh_w13, *sh_w2;
    const void *s13, *s2, *sh_s13, *sh_s2;
    void* out;
    int32_t* topk_idx_out;
    float* topk_w_out;
    int T, H, E, K, I, Is;
    float scale, topp;
    unsigned flags;
    int gshift, stype;
    int G13, G2, Gs2;  // scales per row of w13 (and sh_w13), w2, sh_w2
    // workspace
    FewPicks* picks;
    int8_t* hq;    // [T*K][2][I] then [T][2][Is]: both int8 parts of h
    float* hs;     // [T*K][I/32] then [T][Is/32]: their scales
    float* lpart;  // [lslices][T][E] partial router logits (lslices = 0: none)
    int lslices;
};

int linear_launches(const LinearArgs& a);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t stream);

// The tcgen05 GEMM of more tokens (linear_gemm.cu).
cudaError_t launch_linear_gemm(const LinearArgs& a, cudaStream_t stream);

int few_pass_tokens(const FewArgs& a);
int few_pass_launches(const FewArgs& a);
// Points a's workspace fields into ws (null: only measures); returns the bytes.
size_t few_workspace(FewArgs& a, void* ws);
cudaError_t launch_few(const FewArgs& a, cudaStream_t stream);

}  // namespace moe
