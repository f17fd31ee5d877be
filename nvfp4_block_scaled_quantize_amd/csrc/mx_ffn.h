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

// Four codes.  The conversion takes the scale, mx_scale_value(code), as an operand and divides by it
// exactly; nothing exceeds 448.
typedef short short2v __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t mx8_codes(float a, float b, float c, float d, float scale) {
    short2v w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, scale, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, scale, true);
    return __builtin_bit_cast(uint32_t, w);
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

// The same by the conversion's own scale operand, for scale codes up to 254.
__device__ __forceinline__ Quad mx8_scaled(uint32_t w, uint32_t code) {
    const float s = mx_scale_value(code);
    const float2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true);
    return {{a[0], a[1], b[0], b[1]}};
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
// a(x) and a'(x) = S + x S T y', T = 1 - S = 2^-y S, y' = 1 or 2 z'.  (The difference 1 - S would leave T off by a
// step of 1, which against a' near 1 is |x y'| of them.)  2^-y is kept finite, for the product with S = 0, where a(x)
// is 0 and T does not matter; x^2 for the one with T = 0.
struct Act {
    float a, slope;
};
template <int ACT>
__device__ __forceinline__ Act act_both(float x) {
    const float e = fminf(__builtin_amdgcn_exp2f(act_arg<ACT>(x)), 3.402823466e38f), s = __builtin_amdgcn_rcpf(1.0f + e);
    const float t = e * s, a = x * s;
    if constexpr (ACT == MXFP4_SILU) return {a, __builtin_fmaf(a, t, s)};
    else return {a, __builtin_fmaf(a * t, __builtin_fmaf(6.0f * kGeluB, fminf(x * x, 1e30f), 2.0f * kGeluA), s)};
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
// The upper half of a's lanes and the lower half of b's change places.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0], b = r[1];
}

// The largest magnitude (its bits) of a row's 32 elements: 16 in this lane, 16 in lane ^ 32.  As signed
// numbers the bits of the positive ones order as their values do, as unsigned ones those of the negative ones
// do and lie above the others.
__device__ __forceinline__ uint32_t block_max(const float16v& x) {
    int p = __float_as_int(x[0]);
    uint32_t n = __float_as_uint(x[0]);
#pragma unroll
    for (int r = 1; r < 16; ++r) p = max(p, __float_as_int(x[r])), n = max(n, __float_as_uint(x[r]));
    // (without a negative one n is p; without a positive one p has the sign set)
    uint32_t m = max((uint32_t)max(p, 0), n & 0x7FFFFFFFu), o = m;
    swap_halves(m, o);
    return max(m, o);
}

// A 32 x 32 block as the matrix instructions leave it: lane l holds row l mod 32, and in register r
// column 8 (r / 4) + 4 (l / 32) + r mod 4.
//
// Its E2M1 codes, and the scale's: w[i] holds the lane's halves of dwords 2 i and 2 i + 1 of the row's four.
// `past`: no column of it exists.  (Those of a block that some of exist in are zeros, or of a row that is NaN.)
__device__ __forceinline__ uint32_t copy_codes(const float16v& x, uint32_t above, bool past, uint32_t (&w)[2]) {
    const uint32_t code = past ? 0u : mx_scale_code(block_max(x), above);
    const float cs = mx_scale_value(code);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = cvt_fp4x2<0>(0u, x[8 * i], x[8 * i + 1], cs);
        w[i] = cvt_fp4x2<1>(w[i], x[8 * i + 2], x[8 * i + 3], cs);
        w[i] = cvt_fp4x2<2>(w[i], x[8 * i + 4], x[8 * i + 5], cs);
        w[i] = cvt_fp4x2<3>(w[i], x[8 * i + 6], x[8 * i + 7], cs);
        if (code == 255u || past) w[i] = 0;
    }
    return code;
}
// Two dwords from this lane's halves (`a` of the wave's lower lanes, `b` of its upper ones) of both.
__device__ __forceinline__ void join_halves(uint32_t a, uint32_t b, uint32_t& first, uint32_t& second) {
    first = __builtin_amdgcn_perm(b, a, 0x05040100u), second = __builtin_amdgcn_perm(b, a, 0x07060302u);
}
// The MXFP4 copy of J blocks side by side: 16 J bytes of codes of the row at `codes`, the scales at `scale`.  The
// wave's halves exchange what they hold of each other's dwords: of one block each has two then, of two blocks all
// four of one of them.
template <int J>
__device__ __forceinline__ void put_copy(const float16v (&x)[J], uint32_t above, uint8_t* codes, uint8_t* scale, int left, int h,
                                         bool in) {
    static_assert(J == 1 || J == 2);
    uint32_t w[2][2], code[2], d[4];
#pragma unroll
    for (int j = 0; j < J; ++j) code[j] = copy_codes(x[j], above, left <= 32 * j, w[j]);
    if constexpr (J == 1) {
        swap_halves(w[0][0], w[0][1]);
        join_halves(w[0][0], w[0][1], d[0], d[1]);
        if (!in) return;
        *(uint2*)(codes + 8 * h) = make_uint2(d[0], d[1]);
        if (h == 0) *scale = (uint8_t)code[0];
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            swap_halves(w[0][i], w[1][i]);
            join_halves(w[0][i], w[1][i], d[2 * i], d[2 * i + 1]);
        }
        if (!in) return;
        *(uint4*)(codes + 16 * h) = make_uint4(d[0], d[1], d[2], d[3]);
        if (h == 0) *(uint16_t*)scale = (uint16_t)(code[0] | code[1] << 8);
    }
}

// A block's E4M3 codes, and the scale's: d[q] of columns 8 q + 4 h .. + 3.
__device__ __forceinline__ uint32_t checkpoint_codes(const float16v& x, bool past, uint32_t (&d)[4]) {
    const uint32_t code = past ? 0u : mx8_scale_code(block_max(x));
    const float scale = mx_scale_value(code);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        d[q] = mx8_codes(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3], scale);
        if (code == 255u || past) d[q] = 0;
    }
    return code;
}
// The checkpoint of 32 rows: J blocks side by side of G, and of U `second` elements on; `at`: of row 0.  A
// block's 32 bytes of a row are exchanged between the wave's halves, two blocks' 64 go through LDS.  The lower half
// of the wave stores the scales of G, the upper one those of U.
template <int J>
__device__ __forceinline__ void put_checkpoint(const float16v (&g)[J], const float16v (&u)[J], uint8_t* piece, uint8_t* kc,
                                               uint8_t* ks, int64_t at, int64_t np, int64_t second, int rows, int left, int lane) {
    static_assert(J == 1 || J == 2);
    const int h = lane >> 5, li = lane & 31;
    uint32_t gs = 0, us = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t d[4];
            const uint32_t code = checkpoint_codes(t ? u[j] : g[j], left <= 32 * j, d);
            (t ? us : gs) |= code << (8 * j);
            if constexpr (J == 1) {
                swap_halves(d[0], d[2]);
                swap_halves(d[1], d[3]);
                if (li < rows) *(uint4*)(kc + t * second + at + li * np + 16 * h) = make_uint4(d[0], d[2], d[1], d[3]);
            } else {
                // 64 bytes a row; its chunks of 16 in an order that changes every four rows, which the banks repeat in
                uint8_t* p = piece + t * 2048 + li * 64 + 4 * h;
#pragma unroll
                for (int q = 0; q < 4; ++q) *(uint32_t*)(p + (((2 * j + q / 2) ^ ((li >> 2) & 3)) << 4) + 8 * (q & 1)) = d[q];
            }
        }
    if constexpr (J == 2) {
        const int row = lane >> 2, c = lane & 3;
        const uint8_t* p = piece + row * 64 + ((c ^ ((row >> 2) & 3)) << 4);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint4 v = *(const uint4*)(p + t * 2048 + k * 1024);
                if (row + 16 * k < rows) *(uint4*)(kc + t * second + at + (row + 16 * k) * np + 16 * c) = v;
            }
    }
    if (li < rows) {
        const int64_t s = ((h ? second : 0) + at + li * np) / 32;
        if constexpr (J == 1) ks[s] = (uint8_t)(h ? us : gs);
        else *(uint16_t*)(ks + s) = (uint16_t)(h ? us : gs);
    }
}
// And back: the lane's 16 bytes of a block, as they lie in the row, to the dwords of its four columns each.
__device__ __forceinline__ void spread_checkpoint(uint4 v, uint32_t (&d)[4]) {
    d[0] = v.x, d[2] = v.y, d[1] = v.z, d[3] = v.w;
    swap_halves(d[0], d[2]);
    swap_halves(d[1], d[3]);
}

// What a tiled kernel's product is for: C itself, the block's forward, or its backward.
// (Constants and a trait with a name each: what is unnamed would be part of the kernels' names.)
constexpr int kProduct = 0, kForward = 1, kBackward = 2;
template <int KIND> struct MxKind { using Args = MxFfnArgs; };
template <> struct MxKind<kProduct> { using Args = MxGArgs; };
template <int KIND> using MxKindArgs = typename MxKind<KIND>::Args;
__host__ __device__ inline const MxGArgs& mx_product(const MxGArgs& a) { return a; }
__host__ __device__ inline const MxGArgs& mx_product(const MxFfnArgs& a) { return a.g; }
// Rows of a matrix of B for each column of the result.
template <int KIND> constexpr int kMxWeights = KIND == kForward ? 2 : 1;

// 32 rows x 32 J columns of a result, as blocks of accumulators, to p by way of LDS: `piece`, this wave's 4
// KiB, takes up to 128 bytes a row, its 16-byte chunks in an order by which eight consecutive rows (or four
// pairs of them) touch every bank once, and a wave stores whole pieces of rows from there, 16 bytes a lane, past
// the caches.  `whole`: all rows and columns exist, else `rows` and `left` of them.
template <typename T, int J>
struct Rows {
    static constexpr int kBytes = 32 * J * (int)sizeof(T) < 128 ? 32 * J * (int)sizeof(T) : 128;    // of a row at a time
    static constexpr int kN = kBytes / (int)sizeof(T), kPasses = 32 * J / kN, kChunks = kBytes / 16, kAtOnce = 64 / kChunks;
    using Vec = typename Oct<T>::Vec;
    int h, lr, rr, q;
    __device__ explicit Rows(int lane) : h(lane >> 5), lr(lane & 31), rr(lane / kChunks), q(lane % kChunks) {
#ifdef __HIP_DEVICE_COMPILE__
        asm volatile("" : "+v"(h), "+v"(lr), "+v"(rr), "+v"(q));    // opaque: addresses are made where they are used
#endif
    }
    __device__ static int swizzle(int r) { return kChunks == 8 ? r & 7 : (r >> 1) & 3; }
    // Blocks into the piece.
    __device__ __forceinline__ void put(uint8_t* piece, const float16v (&x)[J], int pass) const {
#pragma unroll
        for (int j = 0; j < kN / 32; ++j)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int byte = (j * 32 + 2 * r + 4 * h) * (int)sizeof(T);
                const float16v& v = x[pass * (kN / 32) + j];
                put_c4((T*)(piece + lr * kBytes + (((byte >> 4) ^ swizzle(lr)) << 4) + (byte & 15)), v[r], v[r + 1], v[r + 2],
                       v[r + 3]);
            }
    }
    // The piece to p.
    __device__ __forceinline__ void store(const uint8_t* piece, T* p, int64_t ld, int pass, int rows, int left, bool whole) const {
        const uint8_t* from = piece + rr * kBytes + ((q ^ swizzle(rr)) << 4);
        const int col = pass * kN + q * (16 / (int)sizeof(T));
        T* to = p + rr * ld + col;
        if (whole) {
#pragma unroll
            for (int k = 0; k < 32 / kAtOnce; ++k) {
                __builtin_nontemporal_store((Vec)*(const int4v*)(from + k * 1024), (Vec*)to);
                to += kAtOnce * ld;
            }
        } else {
#pragma unroll 1
            for (int k = 0; k < 32 / kAtOnce; ++k) {
                const int4v v = *(const int4v*)(from + k * 1024);
                if (rr + k * kAtOnce < rows) store_c16<true>(to, v, left - col);
                to += kAtOnce * ld;
            }
        }
    }
};
template <typename T, int J>
__device__ __forceinline__ void put_rows(uint8_t* piece, const float16v (&x)[J], T* p, int64_t ld, int rows, int left,
                                         bool whole, int lane) {
    const Rows<T, J> r(lane);
#pragma unroll
    for (int pass = 0; pass < r.kPasses; ++pass) {
        r.put(piece, x, pass);
        r.store(piece, p, ld, pass, rows, left, whole);
    }
}

// The forward's results from J blocks of G and as many of U: rows from m0, of which `rows` exist, columns from
// c0, of which `left` are below N: the rest are zeros, products of B's rows past the end, which the copies'
// rows, up to np, hold.
template <typename T, int ACT, int J>
__device__ __forceinline__ void forward_rows(const MxFfnArgs& f, const float16v (&g)[J], const float16v (&u)[J], uint8_t* piece, int64_t m0,
                                             int rows, int64_t c0, int left, bool whole, int lane) {
    const int h = lane >> 5, li = lane & 31;
    float16v x[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) x[j][r] = act_value<ACT>(g[j][r]) * u[j][r];
    if (f.g.c) put_rows<T, J>(piece, x, (T*)f.g.c + m0 * f.g.ldc + c0, f.g.ldc, rows, left, whole, lane);
    if (!f.qc && !f.kc) return;
    const int have = c0 < f.np ? rows : 0;
    const int64_t at = m0 * f.np + c0, b = at + li * f.np;
    if (f.qc) put_copy<J>(x, f.above, f.qc + b / 2, f.qs + b / 32, left, h, li < have);
    if (f.kc) put_checkpoint<J>(g, u, piece, f.kc, f.ks, at, f.np, f.g.M * f.np, have, left, lane);
}
// The stores at least that a wave issues for `groups` times 32 whole rows of J blocks: 128 bytes x 8 rows of a
// tensor each, one a pair of blocks of the copy's codes, and two a block of the checkpoint's.
template <typename T>
__device__ __forceinline__ int forward_stores(const MxFfnArgs& f, int groups, int blocks) {
    return groups * (blocks * ((f.g.c ? (int)sizeof(T) : 0) + (f.kc ? 2 : 0)) + (f.qc ? 1 : 0));
}

// Two blocks of the checkpoint in a row: the 32 code bytes of G and of U that this lane decodes, and the scales.
struct Kept {
    uint4 g[2], u[2];
    uint32_t gs, us;
};
// Of row m (or the last there is), columns from c0, a multiple of 64.  No branch: a join would wait for the loads.
__device__ __forceinline__ Kept load_kept(const MxFfnArgs& f, int64_t m, int64_t c0, int h) {
    c0 = c0 < f.np ? c0 : 0;        // (nothing of it will be stored)
    const int64_t at = (m < f.g.M ? m : f.g.M - 1) * f.np + c0, second = f.g.M * f.np;
    Kept k;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        k.g[j] = *(const uint4*)(f.kc + at + 32 * j + 16 * h);
        k.u[j] = *(const uint4*)(f.kc + second + at + 32 * j + 16 * h);
    }
    k.gs = *(const uint16_t*)(f.ks + at / 32);
    k.us = *(const uint16_t*)(f.ks + (second + at) / 32);
    return k;
}

// The backward's results from two blocks d of dH and the checkpoint's; `piece`: 12 KiB.
template <typename T, int ACT>
__device__ __forceinline__ void backward_rows(const MxFfnArgs& f, const float16v (&d)[2], const Kept& kept, uint8_t* piece,
                                              int64_t m0, int rows, int64_t c0, int left, bool whole, int lane) {
    float16v dg[2], du[2], x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t gw[4], uw[4];
        spread_checkpoint(kept.g[j], gw);
        spread_checkpoint(kept.u[j], uw);
        const uint32_t gs = (kept.gs >> (8 * j)) & 0xFFu, us = (kept.us >> (8 * j)) & 0xFFu;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const Quad g = mx8_scaled(gw[q], gs), u = mx8_scaled(uw[q], us);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Act a = act_both<ACT>(g.v[i]);
                const float v = d[j][4 * q + i];
                du[j][4 * q + i] = v * a.a;
                dg[j][4 * q + i] = v * u.v[i] * a.slope;
                x[j][4 * q + i] = a.a * u.v[i];
            }
        }
        if (__builtin_amdgcn_ballot_w64(gs == 255u || us == 255u)) {     // blocks of NaN are rare
            const float both = gs == 255u || us == 255u ? __builtin_nanf("") : 0.0f, gate = gs == 255u ? __builtin_nanf("") : 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) dg[j][r] += both, x[j][r] += both, du[j][r] += gate;
        }
    }
    T* const p = (T*)f.g.c + m0 * f.g.ldc + c0;
    T* const ph = (T*)f.h + m0 * f.ldh + c0;
    const Rows<T, 2> r(lane);
#pragma unroll
    for (int pass = 0; pass < r.kPasses; ++pass) {
        r.put(piece, dg, pass);
        r.put(piece + 4096, du, pass);
        if (f.h) r.put(piece + 8192, x, pass);
        r.store(piece, p, f.g.ldc, pass, rows, left, whole);
        r.store(piece + 4096, p + f.g.N, f.g.ldc, pass, rows, left, whole);
        if (f.h) r.store(piece + 8192, ph, f.ldh, pass, rows, left, whole);
    }
}

// The results of `rows` rows in no group, `width` columns from n0, by a workgroup of 256.
template <typename T>
__device__ __forceinline__ void zero_forward(const MxFfnArgs& f, int64_t m0, int rows, int64_t n0, int width, int t) {
    const int wid = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
    const int64_t second = f.g.M * f.np;
    for (int r = wid; r < rows; r += 4) {
        const int64_t m = m0 + r, at = m * f.np + n0;
        if (f.g.c)
            for (int k = lane; k < width && n0 + k < f.g.N; k += 64) store_c((T*)f.g.c + m * f.g.ldc + n0 + k, 0.0f);
        if (n0 >= f.np) continue;
        if (f.qc && lane < width / 32) *(uint4*)(f.qc + at / 2 + 16 * lane) = uint4{}, f.qs[at / 32 + lane] = 0;
        if (f.kc && lane < width / 16) {
            *(uint4*)(f.kc + at + 16 * lane) = *(uint4*)(f.kc + second + at + 16 * lane) = uint4{};
            if (lane < width / 32) f.ks[at / 32 + lane] = f.ks[(second + at) / 32 + lane] = 0;
        }
    }
}
template <typename T>
__device__ __forceinline__ void zero_backward(const MxFfnArgs& f, int64_t m0, int rows, int64_t n0, int cols, int t) {
    for (int r = __builtin_amdgcn_readfirstlane(t >> 6); r < rows; r += 4)
        for (int k = t & 63; k < cols; k += 64) {
            T* const p = (T*)f.g.c + (m0 + r) * f.g.ldc + n0 + k;
            store_c(p, 0.0f);
            store_c(p + f.g.N, 0.0f);
            if (f.h) store_c((T*)f.h + (m0 + r) * f.ldh + n0 + k, 0.0f);
        }
}

// ---------------------------------------------------------------- host
inline int mx8_check_tensor(const mxfp8_tensor* t, bool used) {
    return mx_check_tensor((const mxfp4_tensor*)t, used);
}
// The tiled kernels (mx_ffn_forward256.hip and so on; that one for bfloat16 alone); mode: MxDense or MxRows.
int mx_forward256(const MxFfnArgs& f, int mode, int act, hipStream_t st);
int mx_forward128(const MxFfnArgs& f, int mode, int dtype, int act, hipStream_t st);
int mx_backward128(const MxFfnArgs& f, int mode, int dtype, int act, hipStream_t st);
// H alone for few rows or few tiles (mx_ffn_few.hip): A packed (f.x null) or quantized from x.  Whether a dense
// product belongs there, and the elements of x that a workgroup quantizes, times the workgroups a compute unit.
int mx_ffn_few(const MxFArgs& f, int x_dtype, int dtype, int act, hipStream_t st);
int mx_ffn_few_backward(const MxFfnArgs& f, int64_t K, int dtype, int act, hipStream_t st);
bool mx_ffn_few_dense(int64_t M, int64_t N, int64_t kp);
int64_t mx_ffn_few_quantized(int64_t M, int64_t N, int64_t kp);
inline bool mx_activation(int32_t a) { return a == MXFP4_SILU || a == MXFP4_GELU; }

}  // namespace nvfp4
