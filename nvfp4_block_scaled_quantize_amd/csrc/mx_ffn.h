// mx_ffn.h -- what the kernels of the gated feed-forward block share: the 8-bit checkpoint's format,
// the activations, and what becomes of a 32 x 32 block of accumulators.
#pragma once
#include "mxffn.h"
#include "mx_common.h"

namespace nvfp4 {

// ---------------------------------------------------------------- E4M3 with E8M0 scales
// E8M0 code of a block from the binary32 bits of its largest magnitude: with 448 = 1.75 * 2^8 the
// smallest power of two s with amax <= 448 s has the exponent field e less 8, or one more where the
// fraction of amax exceeds 0.75.
__device__ __forceinline__ uint32_t mx8_scale_code(uint32_t amax_bits) {
    uint32_t e = amax_bits >> 23;
    if (e == 255u) return 255u;
    e += (amax_bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u;
    return (e > 8u ? e : 8u) - 8u;
}

// Four codes.  inv: 1 / scale, a power of two from mx8_inverse; the products are exact but for
// those below 2^-126, whose code is a zero either way, and none exceeds 448.
__device__ __forceinline__ float mx8_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d, float inv) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

// The scale of a code as a factor; NaN for 255.
__device__ __forceinline__ float mx8_factor(uint32_t code) {
    return code == 255u ? __builtin_nanf("") : mx_scale_value(code);
}
// Four values times s.
struct Quad {
    float v[4];
};
__device__ __forceinline__ Quad mx8_values(uint32_t w, float s) {
    const float2v a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return {{a[0] * s, a[1] * s, b[0] * s, b[1] * s}};
}

// ---------------------------------------------------------------- activations
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluA = 0.7978845608028654f, kGeluB = 0.7978845608028654f * 0.044715f;   // z = A x + B x^3

// x S with S = 1 / (1 + 2^-y): y = x log2 e, or 2 z log2 e.  2^-y may be infinite (S = 0).
template <int ACT>
__device__ __forceinline__ float act_arg(float x) {
    if constexpr (ACT == MXFP4_SILU) return -kLog2e * x;
    else return x * __builtin_fmaf(-2.0f * kLog2e * kGeluB, x * x, -2.0f * kLog2e * kGeluA);
}
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(act_arg<ACT>(x)));
}
// a(x) and a'(x) = S + x S (1 - S) y', y' = 1 or 2 z'.  1 - S as it stands where S is small (2^-y may
// be infinite there), as 2^-y S where the difference would cancel.
struct Act {
    float a, slope;
};
template <int ACT>
__device__ __forceinline__ Act act_both(float x) {
    const float e = __builtin_amdgcn_exp2f(act_arg<ACT>(x)), s = __builtin_amdgcn_rcpf(1.0f + e);
    const float t = s < 0.5f ? 1.0f - s : e * s, a = x * s;
    if constexpr (ACT == MXFP4_SILU) return {a, __builtin_fmaf(a, t, s)};
    else return {a, __builtin_fmaf(a * t, __builtin_fmaf(6.0f * kGeluB, x * x, 2.0f * kGeluA), s)};
}

// ---------------------------------------------------------------- blocks of accumulators
// A product of the block.  g: the product itself (g.N columns of H); g.c, g.ldc: H, or [dG dU].
struct MxFfnArgs {
    MxGArgs g;
    uint32_t above;             // scale rule of H's copy
    uint8_t *qc, *qs;           // H's copy, or null
    uint8_t *kc, *ks;           // the checkpoint (forward: or null)
    int64_t np;                 // K extent of the rows of both: N padded
    void* h;                    // backward: H, or null
    int64_t ldh;
};

typedef uint32_t uint2v __attribute__((ext_vector_type(2)));
typedef int int2_by2 __attribute__((ext_vector_type(2), aligned(2)));
typedef int int4_by4f __attribute__((ext_vector_type(4), aligned(4)));
// Four consecutive elements of a row, of which `left` exist.
__device__ __forceinline__ void store_c4(uint16_t* p, float a, float b, float c, float d, int left) {
    alignas(8) uint16_t e[4];
    put_c4(e, a, b, c, d);
    if (left >= 4) {
        int2_by2 v;
        __builtin_memcpy(&v, e, 8);
        *(int2_by2*)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = e[i];
    }
}
__device__ __forceinline__ void store_c4(float* p, float a, float b, float c, float d, int left) {
    const float e[4] = {a, b, c, d};
    if (left >= 4) {
        int4_by4f v;
        __builtin_memcpy(&v, e, 16);
        *(int4_by4f*)p = v;
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = e[i];
    }
}

// The upper half of a's lanes and the lower half of b's change places.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
}

// The largest magnitude (its bits) of a row's 32 elements: 16 in this lane, 16 in lane ^ 32.
__device__ __forceinline__ uint32_t block_max(const float16v& x) {
    uint32_t m = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) m = max(m, __float_as_uint(x[r]) & 0x7FFFFFFFu);
    uint32_t o = m;
    swap_halves(m, o);
    return max(m, o);
}

// A 32 x 32 block as the matrix instructions leave it: lane l holds row l mod 32, and in register r
// column 8 (r / 4) + 4 (l / 32) + r mod 4.
//
// Its MXFP4 copy: codes at `codes` (16 bytes of the row), the scale at `scale`.  A lane makes a half of
// each of the row's four dwords; the halves of the wave exchange them so that each lane has two.
__device__ __forceinline__ void put_copy_block(const float16v& x, uint32_t above, uint8_t* codes, uint8_t* scale,
                                               int h, bool in) {
    const uint32_t code = mx_scale_code(block_max(x), above);
    const float cs = mx_scale_value(code);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = cvt_fp4x2<0>(0u, x[8 * i], x[8 * i + 1], cs);
        w[i] = cvt_fp4x2<1>(w[i], x[8 * i + 2], x[8 * i + 3], cs);
        w[i] = cvt_fp4x2<2>(w[i], x[8 * i + 4], x[8 * i + 5], cs);
        w[i] = cvt_fp4x2<3>(w[i], x[8 * i + 6], x[8 * i + 7], cs);
        if (code == 255u) w[i] = 0;
    }
    swap_halves(w[0], w[1]);
    if (!in) return;
    *(uint2*)(codes + 8 * h) = make_uint2(__builtin_amdgcn_perm(w[1], w[0], 0x05040100u),
                                          __builtin_amdgcn_perm(w[1], w[0], 0x07060302u));
    if (h == 0) *scale = (uint8_t)code;
}

// Its checkpoint: 32 bytes of the row at `codes`, 16 of them a lane's.
__device__ __forceinline__ void put_checkpoint_block(const float16v& x, uint8_t* codes, uint8_t* scale, int h, bool in) {
    const uint32_t code = mx8_scale_code(block_max(x));
    const float inv = mx8_inverse(code);
    uint32_t d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        d[q] = mx8_codes(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3], inv);
        if (code == 255u) d[q] = 0;
    }
    swap_halves(d[0], d[2]);
    swap_halves(d[1], d[3]);
    if (!in) return;
    *(uint4*)(codes + 16 * h) = make_uint4(d[0], d[2], d[1], d[3]);
    if (h == 0) *scale = (uint8_t)code;
}
// And back: the lane's 16 bytes, as they lie there, to the dwords of its four columns each.
__device__ __forceinline__ void spread_checkpoint(uint4 v, uint32_t (&d)[4]) {
    d[0] = v.x, d[2] = v.y, d[1] = v.z, d[3] = v.w;
    swap_halves(d[0], d[2]);
    swap_halves(d[1], d[3]);
}

// The forward's results from a block of G and of U: row m of the lane (stored if `in`), columns from
// c0, of which `left` are below N (the rest are zeros in the copies).
template <typename T, int ACT>
__device__ __forceinline__ void put_forward(const MxFfnArgs& f, float16v& g, float16v& u, int64_t m, bool in, int64_t c0,
                                            int left, int h) {
    float16v x;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        if (left < 32 && 8 * (r / 4) + 4 * h + r % 4 >= left) g[r] = u[r] = 0.0f;
        x[r] = act_value<ACT>(g[r]) * u[r];
    }
    if (f.g.c && in) {
        T* p = (T*)f.g.c + m * f.g.ldc + c0 + 4 * h;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            store_c4(p + 8 * q, x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3], left - 8 * q - 4 * h);
    }
    const int64_t at = m * f.np + c0;
    if (f.qc) put_copy_block(x, f.above, f.qc + at / 2, f.qs + at / 32, h, in);
    if (f.kc) {
        const int64_t second = f.g.M * f.np;
        put_checkpoint_block(g, f.kc + at, f.ks + at / 32, h, in);
        put_checkpoint_block(u, f.kc + second + at, f.ks + (second + at) / 32, h, in);
    }
}

// The backward's results from a block d of dH and the checkpoint.  `left` of its columns are below N.
template <typename T, int ACT>
__device__ __forceinline__ void put_backward(const MxFfnArgs& f, const float16v& d, int64_t m, bool in, int64_t c0, int left,
                                             int h, bool zero) {
    if (!in || left <= 0) return;       // (the same for both lanes of a row)
    const int64_t at = m * f.np + c0, second = f.g.M * f.np;
    uint32_t gw[4], uw[4];
    spread_checkpoint(*(const uint4*)(f.kc + at + 16 * h), gw);
    spread_checkpoint(*(const uint4*)(f.kc + second + at + 16 * h), uw);
    const float gs = mx8_factor(f.ks[at / 32]), us = mx8_factor(f.ks[(second + at) / 32]);
    T* const pg = (T*)f.g.c + m * f.g.ldc + c0 + 4 * h;
    T* const ph = (T*)f.h + m * f.ldh + c0 + 4 * h;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const Quad g = mx8_values(gw[q], gs), u = mx8_values(uw[q], us);
        Quad dg, du, x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Act a = act_both<ACT>(g.v[i]);
            du.v[i] = zero ? 0.0f : d[4 * q + i] * a.a;
            dg.v[i] = zero ? 0.0f : d[4 * q + i] * u.v[i] * a.slope;
            x.v[i] = zero ? 0.0f : a.a * u.v[i];
        }
        const int n = left - 8 * q - 4 * h;
        store_c4(pg + 8 * q, dg.v[0], dg.v[1], dg.v[2], dg.v[3], n);
        store_c4(pg + f.g.N + 8 * q, du.v[0], du.v[1], du.v[2], du.v[3], n);
        if (f.h) store_c4(ph + 8 * q, x.v[0], x.v[1], x.v[2], x.v[3], n);
    }
}

// ---------------------------------------------------------------- host
inline int mx8_check_tensor(const mxfp8_tensor* t, bool used) {
    return mx_check_tensor((const mxfp4_tensor*)t, used);
}
inline bool mx_activation(int32_t a) { return a == MXFP4_SILU || a == MXFP4_GELU; }

}  // namespace nvfp4
