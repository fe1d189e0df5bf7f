// C ABI of the operators on int4 weights with group scales: argument
// validation and the passes of a call.  See include/moe_int4.h.
#include <math.h>
#include <string.h>

#include "group_int4.h"
#include "moe_int4.h"

namespace {

using namespace moe;

static_assert(kScaleF32 == MOE_SCALE_F32 && kScaleBf16 == MOE_SCALE_BF16 && kScaleF16 == MOE_SCALE_F16,
              "scale types match the C ABI");

constexpr int32_t kMaxTokens = 1 << 20;

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

// group -> log2 of the columns per scale; false: not a group of the format.
bool group_shift(int32_t group, int* shift) {
    if (group == 0) {
        *shift = kRowGroup;
        return true;
    }
    if (group < 32 || group > 32768 || (group & (group - 1))) return false;
    int s = 0;
    while ((1 << s) < group) ++s;
    *shift = s;
    return true;
}

int groups_of(int cols, int shift) { return shift == kRowGroup ? 1 : (int)(((long long)cols + (1 << shift) - 1) >> shift); }

size_t scale_bytes(int stype) { return stype == kScaleF32 ? 4 : 2; }

struct Range {
    uintptr_t lo, hi;
    bool meets(const Range& o) const { return lo < o.hi && o.lo < hi && lo < hi && o.lo < o.hi; }
};
Range range(const void* p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }

int linear_args(const moe_linear_cfg_t* c, int32_t T, LinearArgs* a) {
    if (!c || c->struct_size != sizeof(moe_linear_cfg_t)) return MOE_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxTokens || c->N <= 0 || c->K <= 0) return MOE_ERR_INVALID_ARG;
    if (c->flags & ~(MOE_OUT_F32 | MOE_FULL_WEIGHTS | MOE_TEST_STALL)) return MOE_ERR_INVALID_ARG;
    if (c->scale_type < kScaleF32 || c->scale_type > kScaleF16) return MOE_ERR_INVALID_ARG;
    memset(a, 0, sizeof *a);
    a->T = T;
    a->N = c->N;
    a->K = c->K;
    a->stype = c->scale_type;
    a->out_f32 = (c->flags & MOE_OUT_F32) != 0;
    a->full = (c->flags & MOE_FULL_WEIGHTS) != 0;
    a->stall = (c->flags & MOE_TEST_STALL) != 0;
    a->ldx = c->ldx ? c->ldx : c->K;
    a->ldo = c->ldo ? c->ldo : c->N;
    a->lda = c->lda ? c->lda : c->N;
    // strides up to 2^40 elements keep every byte offset below 2^63
    const int64_t most = (int64_t)1 << 40;
    if (a->ldx < c->K || a->ldo < c->N || a->lda < c->N || a->ldx > most || a->ldo > most || a->lda > most)
        return MOE_ERR_INVALID_ARG;
    if (!group_shift(c->group, &a->gshift)) return MOE_ERR_UNSUPPORTED;
    if (c->K % 32 || c->K > 32768 || c->N > (1 << 20) || a->ldx % 8) return MOE_ERR_UNSUPPORTED;
    a->G = groups_of(c->K, a->gshift);
    return MOE_OK;
}

int few_args(const moe_few_cfg_t* c, int32_t T, FewArgs* a) {
    if (!c || c->struct_size != sizeof(moe_few_cfg_t)) return MOE_ERR_INVALID_ARG;
    if (T < 0 || T > kMaxTokens) return MOE_ERR_INVALID_ARG;
    if (c->H <= 0 || c->E <= 0 || c->K <= 0 || c->I <= 0 || c->Is < 0 || c->K > c->E) return MOE_ERR_INVALID_ARG;
    if (!(c->routed_scaling > 0.0f) || !isfinite(c->routed_scaling)) return MOE_ERR_INVALID_ARG;
    if (!(c->topp >= 0.0f) || !isfinite(c->topp)) return MOE_ERR_INVALID_ARG;
    if (c->flags & ~(MOE_ADD_RESIDUAL | MOE_OUT_F32 | MOE_DEBUG_POISON)) return MOE_ERR_INVALID_ARG;
    if (c->scale_type < kScaleF32 || c->scale_type > kScaleF16) return MOE_ERR_INVALID_ARG;
    memset(a, 0, sizeof *a);
    if (!group_shift(c->group, &a->gshift)) return MOE_ERR_UNSUPPORTED;
    if (c->H % 128 || c->H > 16384 || c->E > kMaxE || c->K > kMaxK) return MOE_ERR_UNSUPPORTED;
    if (c->I % 128 || c->I > 8192 || c->Is % 128 || c->Is > 8192) return MOE_ERR_UNSUPPORTED;
    a->H = c->H;
    a->E = c->E;
    a->K = c->K;
    a->I = c->I;
    a->Is = c->Is;
    a->scale = c->routed_scaling;
    a->topp = c->topp;
    a->flags = c->flags;
    a->stype = c->scale_type;
    a->G13 = groups_of(c->H, a->gshift);
    a->G2 = groups_of(c->I, a->gshift);
    a->Gs2 = c->Is ? groups_of(c->Is, a->gshift) : 0;
    const int pass = few_pass_tokens(*a);
    a->T = T < pass ? T : pass;
    return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_linear_kernel_launches(const moe_linear_cfg_t* cfg, int32_t T) {
    LinearArgs a;
    if (linear_args(cfg, T, &a) != MOE_OK || T == 0) return 0;
    return linear_launches(a);
}

int moe_linear_forward(const void* x, const uint8_t* w, const void* scales, const void* add, void* out, int32_t T,
                       const moe_linear_cfg_t* cfg, void* stream) {
    LinearArgs a;
    const int st = linear_args(cfg, T, &a);
    if (st != MOE_OK) return st;
    if (!x || !w || !scales || !out) return MOE_ERR_INVALID_ARG;
    const size_t osz = a.out_f32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(scales, 16) || !aligned(out, osz) || !aligned(add, 2))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const Range ro = range(out, ((size_t)(T - 1) * a.ldo + a.N) * osz);
    if (ro.meets(range(x, ((size_t)(T - 1) * a.ldx + a.K) * 2)) || ro.meets(range(w, (size_t)a.N * (a.K / 2))) ||
        ro.meets(range(scales, (size_t)a.N * a.G * scale_bytes(a.stype))))
        return MOE_ERR_INVALID_ARG;
    const bool in_place = add == out && !a.out_f32 && (a.lda == a.ldo || T == 1);
    if (add && !in_place && ro.meets(range(add, ((size_t)(T - 1) * a.lda + a.N) * 2))) return MOE_ERR_INVALID_ARG;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.w = w;
    a.scales = scales;
    a.add = static_cast<const __nv_bfloat16*>(add);
    a.out = out;
    return launch_linear(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_few_workspace_bytes(const moe_few_cfg_t* cfg, int32_t T) {
    FewArgs a;
    if (few_args(cfg, T, &a) != MOE_OK) return 0;
    if (a.T == 0) a.T = 1;  // a size of 0 means a rejected cfg
    return few_workspace(a, nullptr);
}

int32_t moe_few_pass_tokens(const moe_few_cfg_t* cfg) {
    FewArgs a;
    return few_args(cfg, 0, &a) == MOE_OK ? few_pass_tokens(a) : 0;
}

int32_t moe_few_kernel_launches(const moe_few_cfg_t* cfg, int32_t T) {
    FewArgs a;
    if (few_args(cfg, T, &a) != MOE_OK || T == 0) return 0;
    const int pass = few_pass_tokens(a);
    int n = T / pass * few_pass_launches(a);  // a.T: the tokens of a full pass
    a.T = T % pass;
    if (a.T > 0) n += few_pass_launches(a);
    return n;
}

int moe_few_forward(const void* x, const moe_few_weights_t* w, void* out, int32_t T, const moe_few_cfg_t* cfg,
                    void* stream) {
    FewArgs a;
    const int st = few_args(cfg, T, &a);
    if (st != MOE_OK) return st;
    if (!x || !w || !out) return MOE_ERR_INVALID_ARG;
    const void* need[] = {x, out, w->router_w, w->router_bias, w->w13, w->s13, w->w2, w->s2};
    for (const void* p : need)
        if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    const void* shared[] = {w->sh_w13, w->sh_s13, w->sh_w2, w->sh_s2};
    for (const void* p : shared)
        if (a.Is > 0 && (!p || !aligned(p, 16))) return MOE_ERR_INVALID_ARG;
    if (!aligned(cfg->topk_idx_out, 16) || !aligned(cfg->topk_w_out, 16)) return MOE_ERR_INVALID_ARG;
    const size_t osz = (a.flags & MOE_OUT_F32) ? 4 : 2, n = (size_t)T * a.H;
    const size_t need_ws = moe_few_workspace_bytes(cfg, T);
    if (!cfg->workspace || cfg->workspace_bytes < need_ws) return MOE_ERR_WORKSPACE;
    if (!aligned(cfg->workspace, 256)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    // What a call writes meets nothing else that it reads or writes.
    const size_t tk = (size_t)T * a.K, sb = scale_bytes(a.stype), E = a.E, H = a.H, I = a.I, Is = a.Is;
    const Range writes[] = {range(out, n * osz), range(cfg->workspace, need_ws),
                            range(cfg->topk_idx_out, cfg->topk_idx_out ? tk * 4 : 0),
                            range(cfg->topk_w_out, cfg->topk_w_out ? tk * 4 : 0)};
    const Range reads[] = {range(x, n * 2), range(w->router_w, E * H * 4), range(w->router_bias, E * 4),
                           range(w->w13, E * I * H), range(w->s13, E * 2 * I * a.G13 * sb),
                           range(w->w2, E * H * I / 2), range(w->s2, E * H * a.G2 * sb),
                           range(w->sh_w13, Is * H), range(w->sh_s13, 2 * Is * a.G13 * sb),
                           range(w->sh_w2, H * Is / 2), range(w->sh_s2, H * a.Gs2 * sb)};
    for (const Range& o : writes) {
        for (const Range& r : reads)
            if (o.meets(r)) return MOE_ERR_INVALID_ARG;
        for (const Range& r : writes)
            if (&o != &r && o.meets(r)) return MOE_ERR_INVALID_ARG;
    }
    a.rw = w->router_w;
    a.rb = w->router_bias;
    a.w13 = w->w13;
    a.s13 = w->s13;
    a.w2 = w->w2;
    a.s2 = w->s2;
    a.sh_w13 = w->sh_w13;
    a.sh_s13 = w->sh_s13;
    a.sh_w2 = w->sh_w2;
    a.sh_s2 = w->sh_s2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int pass = few_pass_tokens(a);
    for (int32_t t0 = 0; t0 < T; t0 += pass) {
        a.T = T - t0 < pass ? T - t0 : pass;
        a.x = static_cast<const __nv_bfloat16*>(x) + (size_t)t0 * a.H;
        a.out = static_cast<char*>(out) + (size_t)t0 * a.H * osz;
        a.topk_idx_out = cfg->topk_idx_out ? cfg->topk_idx_out + (size_t)t0 * a.K : nullptr;
        a.topk_w_out = cfg->topk_w_out ? cfg->topk_w_out + (size_t)t0 * a.K : nullptr;
        few_workspace(a, cfg->workspace);
        // every byte a kernel reads must have been written first
        if ((a.flags & MOE_DEBUG_POISON) && cudaMemsetAsync(cfg->workspace, 0xFF, need_ws, s) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (launch_few(a, s) != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

}  // extern "C"
