// Weight streaming of the group-scaled int4 operators (internal): one warp
// multiplies 16 weight rows x 256 columns (a chunk: 2 KB of codes) with up to
// eight tokens on mma.sync m16n8k32 s8.
//
// Activations.  A token's 256 columns of a chunk are written as s * (q0 + q1 /
// 256) with int8 q0, q1 and a power of two s from their largest magnitude
// (qscale): 16 bits, off by at most 2^-15 of that magnitude.  Columns 2j and
// 2j + 1 of an mma's n-tile are the two parts of token j, so a tile serves
// four tokens.  int8 instead of bf16 operands because a weight word then
// reaches the mma in three logic operations per eight codes (lo8 / hi8;
// eleven to bf16) and an mma covers twice the columns: at the copy rate of HBM
// an SM has ~46 codes a cycle to convert.  The products sum exactly in int32
// within a group: |256 sum(q0 c) + sum(q1 c)| < 2^31 for up to 256 columns.
//
// A chunk is staged in shared memory, 128 bytes a row, its 16-byte segments
// permuted by the row (seg_perm), so that both fragment reads are free of
// bank conflicts:
//  - fine groups (32, 64 columns): lane (g, q) of an mma reads word q of a
//    32-column block of rows g and g + 8 (all four lanes of a row in one group);
//  - coarse groups (128 columns and more): it reads the 16 bytes of columns
//    32 q of a 128-column half, whose four words go to four mmas; the
//    activations are stored in that order (x_pos).
#pragma once

#include "group_int4.h"
#include "stream_ops.cuh"

namespace moe {

constexpr int kChunkK = 256;
constexpr int kStageBytes = 16 * kChunkK / 2;

__device__ __forceinline__ int seg_perm(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }

// Bytes of one part of one token's activations, `chunks` chunks long: the
// padding puts the rows of a fragment read on different banks.
template <bool kCoarse>
__host__ __device__ constexpr int x_stride(int chunks) {
    return chunks * kChunkK + (kCoarse ? 64 : 32);
}

// Byte offset, within its chunk, of the eight columns 8 i .. 8 i + 7.
template <bool kCoarse>
__device__ __forceinline__ int x_pos(int i) {
    if (!kCoarse) return 8 * i;
    return (i >> 4) * 128 + ((i & 3) >> 1) * 64 + ((i >> 2) & 3) * 16 + (i & 1) * 8;
}

// Scale of 256 values whose largest magnitude has the bf16 bits m (sign
// cleared): *s = 2^e with |v| / 2^e <= 127, *inv = 256 / s.  Below 2^-113 e stays
// at -119 (256 / s is finite then) and a step is 2^-127, whatever the largest
// magnitude; NaN for NaN and infinity.
__device__ __forceinline__ void block_scale(uint32_t m, float* s, float* inv) {
    // |v| / 2^e in [64, 127]: the largest significand, 127.5 / 64, takes the next e
    const int e = max((int)(m >> 7) - 133 + ((m & 127) == 127), -119);
    *s = m >= 0x7f80 ? __int_as_float(0x7fc00000) : __int_as_float((e + 127) << 23);
    *inv = __int_as_float((135 - e) << 23);
}

// v * inv (inv = 256 / s, |v| <= 127 s) rounded to the nearest integer q: the
// addition of 1.5 * 2^23 leaves q in the low bits.  Byte 0 is q1 (signed);
// byte 1 of the sum with 128 is q0, q = 256 q0 + q1.
__device__ __forceinline__ uint32_t fixed16(float v, float inv) { return __float_as_uint(fmaf(v, inv, 12582912.f)); }

// Eight fixed16 values to the bytes of both parts, in the order of lo8 / hi8
// (0, 2, 4, 6, 1, 3, 5, 7).
__device__ __forceinline__ void pack_parts(const uint32_t (&f)[8], uint2& p0, uint2& p1) {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = f[i] + 128;
    auto low = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    };
    auto high = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
        return __byte_perm(__byte_perm(a, b, 0x0051), __byte_perm(c, d, 0x0051), 0x5410);
    };
    p0 = make_uint2(high(h[0], h[2], h[4], h[6]), high(h[1], h[3], h[5], h[7]));
    p1 = make_uint2(low(f[0], f[2], f[4], f[6]), low(f[1], f[3], f[5], f[7]));
}

// One chunk of one token (a warp; lane l holds columns 8 l .. 8 l + 7 as
// bf16, zero past the row's end): both int8 parts to q0 / q1 (the chunk's
// bytes of each part's row), the scale of the integer sums to *xs (2^-12 of
// the block's: the weights enter as 16 c, part 0 as 256 q0); NaN for a chunk
// that holds NaN or an infinity.
template <bool kCoarse>
__device__ __forceinline__ void quantize_chunk(uint4 v, int8_t* q0, int8_t* q1, float* xs, int lane) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                 __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    float s, inv;
    block_scale(m, &s, &inv);
    uint32_t f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = fixed16(bf16lo(w[i]), inv);
        f[2 * i + 1] = fixed16(bf16hi(w[i]), inv);
    }
    uint2 a, b;
    pack_parts(f, a, b);
    *reinterpret_cast<uint2*>(q0 + x_pos<kCoarse>(lane)) = a;
    *reinterpret_cast<uint2*>(q1 + x_pos<kCoarse>(lane)) = b;
    if (lane == 0) *xs = s * 0x1p-12f;
}

// All chunks of nt tokens (x: the first token's row, ldx elements apart, K
// columns) over the CTA's nw warps, four loads in flight a warp; token t's
// scale of chunk c goes to xs[c * xs_tok + t].  kGlobal: x is in global
// memory (read from L2: what the previous kernel wrote), else in shared memory.
template <bool kCoarse, bool kGlobal>
__device__ __forceinline__ void quantize_tokens(const __nv_bfloat16* x, long long ldx, int K, int chunks, int nt,
                                                int8_t* xq, int xs_bytes, float* xs, int xs_tok, int warp, int nw,
                                                int lane) {
    constexpr int kAhead = 4;
    for (int i0 = warp; i0 < nt * chunks; i0 += kAhead * nw) {
        uint4 v[kAhead];
        int t[kAhead], c[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + u * nw;
            t[u] = i / chunks;
            c[u] = i - t[u] * chunks;
            const int k = c[u] * kChunkK + 8 * lane;
            const uint4* p = reinterpret_cast<const uint4*>(x + t[u] * ldx + k);
            v[u] = t[u] >= nt || k >= K ? make_uint4(0, 0, 0, 0) : kGlobal ? __ldcg(p) : *p;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t[u] >= nt) break;
            int8_t* r = xq + 2 * t[u] * xs_bytes + c[u] * kChunkK;
            quantize_chunk<kCoarse>(v[u], r, r + xs_bytes, xs + c[u] * xs_tok + t[u], lane);
        }
    }
}

// Where lane l's copies of a chunk go: it copies segment l % 8 of rows l / 8 +
// 4 i, i < 4, to stage_at(l) ^ (i odd ? 32 : 0) + 512 i.
__device__ __forceinline__ uint32_t stage_at(int lane) {
    const int r = lane >> 3;
    return r * 128 + (((lane & 7) ^ seg_perm(r)) << 4);
}

// Issues the copies of a chunk of 16 rows (one warp).  dst: the stage's
// shared address + stage_at(lane); p[i]: this lane's segment of the row's
// first chunk; `in`: the segment is inside the row.  Segments past a row's end
// are left as they are: their activations are zero, and the sums are of
// integers.
__device__ __forceinline__ void issue_chunk(uint32_t dst, const uint8_t* const (&p)[4], int c, bool in) {
    if (in) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"((dst ^ ((i & 1) << 5)) + 512 * i),
                         "l"(p[i] + c * (kChunkK / 2))
                         : "memory");
    }
}

// The scales of the rows g and g + 8 of a lane's quad.
struct ScaleRows {
    const char *p0, *p8;
    __device__ __forceinline__ void open(const void* s, size_t row0, size_t row8, int G, int stype) {
        const int sh = stype == kScaleF32 ? 2 : 1;
        p0 = static_cast<const char*>(s) + ((row0 * G) << sh);
        p8 = static_cast<const char*>(s) + ((row8 * G) << sh);
    }
};

// Scales of chunk c's groups: lane q of a quad holds groups q and q + 4 (fine
// groups), or group q & 1 (coarse ones) of row g in sc[0], sc[1] and of row g +
// 8 in sc[2], sc[3]; 0 past the row's end.
template <bool kCoarse>
__device__ __forceinline__ void load_chunk_scales(float (&sc)[4], const ScaleRows& r, int c, int gshift, int G, int stype,
                                                  int q) {
    const int i = kCoarse ? min((c * kChunkK + (q & 1) * 128) >> gshift, G - 1) : ((c * kChunkK) >> gshift) + q;
    const bool in0 = kCoarse || i < G, in1 = !kCoarse && gshift == 5 && i + 4 < G;
    if (stype == kScaleF32) {
        const float *a = reinterpret_cast<const float*>(r.p0) + i, *b = reinterpret_cast<const float*>(r.p8) + i;
        sc[0] = in0 ? __ldg(a) : 0.f;
        sc[2] = in0 ? __ldg(b) : 0.f;
        sc[1] = in1 ? __ldg(a + 4) : 0.f;
        sc[3] = in1 ? __ldg(b + 4) : 0.f;
    } else {
        const unsigned short *a = reinterpret_cast<const unsigned short*>(r.p0) + i,
                             *b = reinterpret_cast<const unsigned short*>(r.p8) + i;
        // kept as raw bits until they are used (see scale_value)
        sc[0] = __uint_as_float(in0 ? __ldg(a) : 0);
        sc[2] = __uint_as_float(in0 ? __ldg(b) : 0);
        sc[1] = __uint_as_float(in1 ? __ldg(a + 4) : 0);
        sc[3] = __uint_as_float(in1 ? __ldg(b + 4) : 0);
    }
}

// What load_chunk_scales left, as f32: converting there would wait for the load.
__device__ __forceinline__ void scale_values(float (&sc)[4], int stype) {
    if (stype == kScaleBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = __uint_as_float(__float_as_uint(sc[i]) << 16);
    } else if (stype == kScaleF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[i] = __half2float(__ushort_as_half((unsigned short)__float_as_uint(sc[i])));
    }
}

__device__ __forceinline__ void mma_s8_first(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// t[n][0 / 1] += scale of row g / g + 8 times the joined integer sums.
template <int NT>
__device__ __forceinline__ void scale_group(float (&t)[NT][2], const int (&d)[NT][4], float s0, float s8) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        t[n][0] = fmaf((float)(d[n][0] * 256 + d[n][1]), s0, t[n][0]);
        t[n][1] = fmaf((float)(d[n][2] * 256 + d[n][3]), s8, t[n][1]);
    }
}

// One staged chunk times the tokens' chunk: t[n][0 / 1], for token 4 n + q
// and rows g / g + 8, in units of the token's xs.  stage: shared address;
// xb[n]: shared address of this lane's B row (token 4 n + g / 2, part g % 2)
// at the chunk's start.
template <int NT, bool kCoarse>
__device__ __forceinline__ void chunk_mma(uint32_t stage, const uint32_t (&xb)[NT], const float (&sc)[4], int gshift,
                                          int lane, float (&t)[NT][2]) {
    const int g = lane >> 2, q = lane & 3, quad = lane & 28;
    const uint32_t row = stage + g * 128 + (seg_perm(g) << 4) + (kCoarse ? 0 : q * 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) t[n][0] = t[n][1] = 0.f;
    int d[NT][4];
    if (kCoarse) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = row ^ ((4 * h + q) << 4);
            const uint4 wa = lds128(at), wb = lds128(at + 1024);
            const uint32_t u[4] = {wa.x, wa.y, wa.z, wa.w}, v[4] = {wb.x, wb.y, wb.z, wb.w};
            uint4 b[NT];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a[4] = {lo8(u[j]), lo8(v[j]), hi8(u[j]), hi8(v[j])};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if ((j & 1) == 0) b[n] = lds128(xb[n] + h * 128 + (j >> 1) * 64 + q * 16);
                    const uint32_t b0 = (j & 1) ? b[n].z : b[n].x, b1 = (j & 1) ? b[n].w : b[n].y;
                    if (j == 0 && (h == 0 || gshift == 7)) mma_s8_first(d[n], a, b0, b1);
                    else mma_s8(d[n], a, b0, b1);
                }
            }
            if (h == 1 || gshift == 7)
                scale_group<NT>(t, d, __shfl_sync(0xffffffffu, sc[0], quad | h), __shfl_sync(0xffffffffu, sc[2], quad | h));
        }
    } else {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const uint32_t at = row ^ (b << 4);
            const uint32_t wa = lds32(at), wb = lds32(at + 1024);
            const uint32_t a[4] = {lo8(wa), lo8(wb), hi8(wa), hi8(wb)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 x = lds64(xb[n] + 32 * b + 8 * q);
                if ((b & 1) == 0 || gshift == 5) mma_s8_first(d[n], a, x.x, x.y);
                else mma_s8(d[n], a, x.x, x.y);
            }
            if (gshift == 5)
                scale_group<NT>(t, d, __shfl_sync(0xffffffffu, sc[b >> 2], quad | (b & 3)),
                                __shfl_sync(0xffffffffu, sc[2 + (b >> 2)], quad | (b & 3)));
            else if (b & 1)
                scale_group<NT>(t, d, __shfl_sync(0xffffffffu, sc[0], quad | (b >> 1)),
                                __shfl_sync(0xffffffffu, sc[2], quad | (b >> 1)));
        }
    }
}

}  // namespace moe
