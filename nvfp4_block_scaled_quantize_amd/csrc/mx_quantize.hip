// mx_quantize.hip -- MXFP4 quantization and its inverse.
//
// x_hat = E2M1(x / s) s with s = 2^(code - 127) from the block's largest magnitude (32
// elements).  Division by s is exact, so the only rounding is E2M1's.  The conversion
// instructions take s as an operand (its exponent) and bfloat16 pairs as they are.
//
// Bound by memory: an element costs 2 or 4 bytes read and 17/32 written per copy.  There is no
// pass for a tensor maximum, so every element is read once.
//
// From a checkpoint it is 33/32 bytes read, and as many instructions as the vector units do meanwhile: 8192 x 4096
// both copies 22 us (the same of bfloat16 29), the row copy 10, the column copy 12, against floors of 10, 7 and 7;
// 8192 x 9216 49, 22 and 30.  Stochastic, eight checkpoints and their copies in turn: 8192 x 9216 both copies 75 against
// 49 to nearest there, 36 against 23 and 45 against 31; 8192 x 4096 38 against 25; 8191 x 1536 in 15 groups 22 against 11.
//
// Stochastic rounding of bfloat16 is bound by the vector units instead (busy in 0.84 of the
// cycles, in 0.42 to nearest): ten Philox rounds per eight elements and copy, and a conversion
// each.  8192 x 9216 both copies 78 us against 47 to nearest, the row copy alone 44 against 35;
// 8192 x 4608 float32 both 52 against 45; 8191 x 1536 bfloat16 in 15 groups 25 against 15.
#include "mx_ffn.h"
#include "mx_pieces.h"

namespace nvfp4 {

struct MxQArgs {
    const void* x;
    const uint8_t* xs;              // x is a checkpoint's codes: their scales
    int64_t batch, rows, cols, ld, stride;
    const int32_t* offsets;
    int n_groups;
    uint8_t *rc, *rs, *cc, *cs;     // rc / cc null: no such copy
    int64_t row_kp, col_kp;         // K extents of the two copies
    uint32_t above;                 // the scale rule, see mx_scale_code
    int sr_row, sr_col;             // stochastic rounding
    int stream;                     // read x past the caches
    uint32_t k0, k1;                // Philox key
};

// Stochastic: x / s in binary32 (exact but for results below 2^-126, which round to 0 with
// every draw that f 2^16 < 1 allows), then the conversion at unit scale.  e: the first
// element's index in the copy (a multiple of 8).
template <typename T>
__device__ __forceinline__ uint32_t codes_sr(const Oct<T>& o, uint32_t code, int64_t e, uint32_t copy,
                                             uint32_t k0, uint32_t k1) {
    const U4 c = {(uint32_t)(e >> 3), (uint32_t)(e >> 35), copy, kTagMxSR};
    const U4 r = philox10(c, k0, k1);
    const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
    const float inv = __uint_as_float((254u - code) << 23);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t bits = (i & 1) ? rw[i >> 1] & 0xFFFF0000u : rw[i >> 1] << 16;
        w |= (cvt_fp4_sr(value(o, i) * inv, bits) & 0xFu) << (4 * i);
    }
    return w;
}

// SR: the kernel may round stochastically (then `sr` decides).
template <bool SR, typename T>
__device__ __forceinline__ uint32_t codes_of(const Oct<T>& o, uint32_t code, bool sr, int64_t e, uint32_t copy,
                                             const MxQArgs& g) {
    uint32_t w;
    if (SR && sr) w = codes_sr(o, code, e, copy, g.k0, g.k1);
    else w = codes_rne(o, mx_scale_value(code));
    return code == 255u ? 0u : w;
}

// Rowwise copy alone: a lane per eight elements, a quad per block, so that loads and stores
// are contiguous over the wave.  A workgroup takes kRowSteps times 256 consecutive octs of the
// copy (rows padded to row_kp), all loaded before the first is used.  From memory (inputs of 600 MB
// in turn) 8192 x 9216 bfloat16 35 to 37 us, 5.5 to 5.2 TB/s read and written; 16 x 4096 2.7 us, an
// empty kernel's time.
constexpr int kRowSteps = 4;
template <typename T, bool SR>
__global__ __launch_bounds__(256) void k_mx_rows(MxQArgs g) {
    const uint32_t per = (uint32_t)(g.row_kp / 8);      // octs of a row
    const int64_t first = (int64_t)blockIdx.x * (256 * kRowSteps), total = g.batch * g.rows * per;
    const int64_t row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    Oct<T> o[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const uint32_t at = rem + threadIdx.x + 256 * i, dr = at / per;
        const int64_t r = row0 + dr, k = (int64_t)(at - dr * per) * 8;
        const int64_t b = g.batch == 1 ? 0 : r / g.rows;
        const bool in = first + threadIdx.x + 256 * i < total;
        o[i] = load_oct((const T*)g.x + b * g.stride + (r - b * g.rows) * g.ld + k, in ? g.cols - k : 0);
    }
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const int64_t at = first + threadIdx.x + 256 * i;   // oct of the copy
        const uint32_t code = mx_scale_code(quad_max(max_bits(o[i])), g.above);
        const uint32_t w = codes_of<SR>(o[i], code, g.sr_row, at * 8, 0, g);
        if (at < total) {
            ((uint32_t*)g.rc)[at] = w;
            if ((threadIdx.x & 3) == 0) g.rs[at >> 2] = (uint8_t)code;
        }
    }
}

// Both copies, or the columnwise one: a workgroup takes a 128-row unit times 256 bytes of
// columns (128 bfloat16, 64 float32).  Rows are loaded a lane per oct, quantized rowwise from
// registers, and put into LDS as dwords [row][64]; then a thread takes one dword column (two
// bfloat16 columns or one float32 one) of 32 rows.  Dword c of row r lies at c ^ 16 (r / 32), so
// that the four row blocks of 16 dword columns, which a wave reads at once (a quad of lanes
// per column, for 64 contiguous bytes of its codes), are in different banks.  From memory 8192 x 9216
// bfloat16 47 to 49 us, 4.9 to 4.7 TB/s; 8192 x 4608 float32 45 to 47 us, 4.2 to 4.0 TB/s.
template <typename T, bool SR>
__global__ __launch_bounds__(256) void k_mx_tile(MxQArgs g, unsigned units, unsigned col_tiles) {
    constexpr int kTileCols = 256 / sizeof(T), kPerRow = kTileCols / 8;   // octs of a tile row
    constexpr int kRowsAtOnce = 256 / kPerRow, kSteps = kMxPad / kRowsAtOnce;
    __shared__ __attribute__((aligned(16))) uint32_t tile[kMxPad * 64];
    const int t = threadIdx.x;
    unsigned u, ct;
    int64_t b = 0, row0, rows, kp0;
    bool has_col = g.cc != nullptr;
    if (g.n_groups) {
        MxUnit m;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.rows, kMxPad, blockIdx.x, col_tiles, u, ct, m)) return;
        row0 = m.row0, rows = m.rows, kp0 = (int64_t)u * kMxPad;
        if (m.group == g.n_groups) has_col = false;
    } else {
        mx_tile_of(blockIdx.x, units * (unsigned)g.batch, col_tiles, u, ct);
        b = u / units, u = u % units;
        row0 = kp0 = (int64_t)u * kMxPad;
        rows = g.rows - row0 < kMxPad ? g.rows - row0 : kMxPad;
    }
    const int64_t c0 = (int64_t)ct * kTileCols;
    const int tr = t / kPerRow, tc = t % kPerRow;        // this lane's row and oct of a step
    const int64_t left = g.cols - c0 - tc * 8;
    const T* p = (const T*)g.x + b * g.stride + (row0 + tr) * g.ld + c0 + tc * 8;
    Oct<T> o[kSteps];
    const auto load = [&](auto stream) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
            o[i] = load_oct<T, decltype(stream)::value>(p + (int64_t)i * kRowsAtOnce * g.ld,
                                                        tr + i * kRowsAtOnce < rows ? left : 0);
    };
    if (g.stream) load(std::true_type{});
    else load(std::false_type{});
    if (has_col) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = tr + i * kRowsAtOnce;
            uint32_t* d = tile + r * 64 + ((tc * (int)sizeof(T) * 2) ^ (16 * (r >> 5)));
            const uint4* src = (const uint4*)&o[i];
#pragma unroll
            for (int q = 0; q < (int)sizeof(T) / 2; ++q) ((uint4*)d)[q] = src[q];
        }
    }
    if (g.rc) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = tr + i * kRowsAtOnce;
            const uint32_t code = mx_scale_code(quad_max(max_bits(o[i])), g.above);
            const int64_t e = (b * g.rows + row0 + r) * g.row_kp + c0 + tc * 8;
            const uint32_t w = codes_of<SR>(o[i], code, g.sr_row, e, 0, g);
            // the scale bytes of the four blocks in 16 lanes: of one bfloat16 row, or of two
            // float32 rows, in one store a row
            uint32_t sc = code << (8 * ((t >> 2) & 3));
            sc |= (uint32_t)dpp<kRor4>(0, (int)sc);
            sc |= (uint32_t)dpp<kRor8>(0, (int)sc);
            if (r < rows) {
                *(uint32_t*)(g.rc + e / 2) = w;
                if (tc == 0) {
                    if constexpr (sizeof(T) == 2) *(uint32_t*)(g.rs + e / 32) = sc;
                    else *(uint16_t*)(g.rs + e / 32) = (uint16_t)(sc >> (8 * ((t >> 2) & 2)));
                }
            }
        }
    }
    if (!has_col) return;
    __syncthreads();
    // dword column dc, rows 32 rb .. 32 rb + 31
    const int rb = t & 3, dc = t >> 2;
    const uint32_t* s = tile + rb * 32 * 64 + (dc ^ (16 * rb));
    uint32_t d[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) d[j] = s[j * 64];
    constexpr int kCols = 4 / sizeof(T);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if constexpr (sizeof(T) == 2) m = max_bf16x2(m, d[j] & 0x7FFF7FFFu);
        else m = max(m, d[j] & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int q = 0; q < kCols; ++q) {
        const uint32_t bits = sizeof(T) == 4 ? m : q ? m & 0xFFFF0000u : m << 16;
        const uint32_t code = mx_scale_code(bits, g.above);
        const int64_t c = c0 + dc * kCols + q;
        const int64_t e = (b * g.cols + c) * g.col_kp + kp0 + rb * 32;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            Oct<T> v;
            if constexpr (sizeof(T) == 2) {
                // the two halves of rows j and j + 1 that belong to column q
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v.w[j] = __builtin_amdgcn_perm(d[8 * k + 2 * j + 1], d[8 * k + 2 * j],
                                                   q ? 0x07060302u : 0x05040100u);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v.v[j] = __uint_as_float(d[8 * k + j]);
            }
            w[k] = codes_of<SR>(v, code, g.sr_col, e + 8 * k, 1, g);
        }
        uint32_t sc = code << (8 * rb);
        sc |= (uint32_t)dpp<kXor1>(0, (int)sc);
        sc |= (uint32_t)dpp<kXor2>(0, (int)sc);
        if (c < g.cols) {
            *(uint4*)(g.cc + e / 2) = make_uint4(w[0], w[1], w[2], w[3]);
            if (rb == 0) *(uint32_t*)(g.cs + e / 32) = sc;
        }
    }
}

// ---------------------------------------------------------------- from a checkpoint
// A lane takes 16 elements, half a block: their codes in one load.  A checkpoint's rows are as wide as the
// rowwise copy's, so element for element the two lie at the same index.  The conversion takes the block's scale
// and gives bfloat16, rounded only below 2^-126; with scale code 255 every code gives NaN.  (Row copy of 8192 x 4096
// 10 us against 15 with eight elements a lane, conversions by way of binary32 and the rows' divisions.)
struct Kept16 {
    int4v w;
    uint32_t code;
};
template <bool STREAM>
__device__ __forceinline__ Kept16 load_kept16(const MxQArgs& g, int64_t at) {
    const int4v* p = (const int4v*)((const uint8_t*)g.x + at);
    return {STREAM ? __builtin_nontemporal_load(p) : *p, g.xs[at / kMxBlock]};
}
// Zeros in place of all but the first `left` elements.
__device__ __forceinline__ void keep16(Kept16& x, int64_t left) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (left < 4 * i + 4) x.w[i] = left <= 4 * i ? 0 : x.w[i] & ((1 << (8 * (left - 4 * i))) - 1);
    if (left <= 0) x.code = 0;
}
struct Oct16 {
    Oct<uint16_t> o[2];
};
__device__ __forceinline__ uint32_t kept_pair(uint32_t w, float s, bool upper) {
    return upper ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))
                 : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
}
__device__ __forceinline__ Oct16 values_of(const Kept16& x) {
    const float s = mx8_factor(x.code);
    Oct16 v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v.o[i / 2].w[i % 2 * 2] = kept_pair(x.w[i], s, false), v.o[i / 2].w[i % 2 * 2 + 1] = kept_pair(x.w[i], s, true);
    return v;
}
__device__ __forceinline__ uint32_t pair_scale(const Oct16& v, uint32_t above) {
    const uint32_t m = max(max_bits(v.o[0]), max_bits(v.o[1]));
    return mx_scale_code(max(m, (uint32_t)dpp<kXor1>(0, (int)m)), above);
}
// The bits of four lane pairs' values, of eight lanes.
__device__ __forceinline__ uint32_t join8(uint32_t v) {
    v |= (uint32_t)dpp<kXor2>(0, (int)v);
    return v | (uint32_t)dpp<kHalfMirror>(0, (int)v);
}

template <bool SR>
__global__ __launch_bounds__(256) void k_mx8_rows(MxQArgs g) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, total = g.batch * g.rows * (g.row_kp / 16);
    const int64_t from = (at < total ? at : total - 1) * 16;
    Kept16 x = g.stream ? load_kept16<true>(g, from) : load_kept16<false>(g, from);
    if (g.cols < g.row_kp) {
        const uint32_t per = (uint32_t)(g.row_kp / 16), rem = (uint32_t)((int64_t)blockIdx.x * 256 % per);
        keep16(x, g.cols - (int64_t)((rem + threadIdx.x) % per) * 16);
    }
    const Oct16 v = values_of(x);
    const uint32_t code = pair_scale(v, g.above);
    const uint32_t w0 = codes_of<SR>(v.o[0], code, g.sr_row, at * 16, 0, g);
    const uint32_t w1 = codes_of<SR>(v.o[1], code, g.sr_row, at * 16 + 8, 0, g);
    if (at < total) {
        ((uint2*)g.rc)[at] = make_uint2(w0, w1);
        if ((threadIdx.x & 1) == 0) g.rs[at >> 1] = (uint8_t)code;
    }
}

// Both copies, or the columnwise one: a workgroup takes 128 rows x 128 columns.  LDS holds the codes as they came, and
// the blocks' scales as factors; a thread takes four columns of 16 rows, eight lanes a column's 128.  Byte c of row r
// lies at c ^ 32 (r / 32), so that the four row blocks are in different banks.  18 KB, so that eight workgroups run
// at once on a compute unit: 8192 x 4096 22 us against 25 with the values in LDS, 32 KB, and eight elements a lane.  Without
// the columns' stores 16; those past the caches it takes 17, but decodes of both copies after it 5 more than they save.
constexpr int kKeptStride = kMxPad + 4;
template <bool SR>
__global__ __launch_bounds__(256, 8) void k_mx8_tile(MxQArgs g, unsigned units, unsigned col_tiles) {
    constexpr int kSteps = 4;
    __shared__ __attribute__((aligned(16))) uint8_t tile[kMxPad * 128];
    __shared__ __attribute__((aligned(16))) float factors[4 * kKeptStride];
    const int t = threadIdx.x;
    unsigned u, ct;
    int64_t b = 0, row0, rows, kp0;
    bool has_col = true;
    if (g.n_groups) {
        MxUnit m;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.rows, kMxPad, blockIdx.x, col_tiles, u, ct, m)) return;
        row0 = m.row0, rows = m.rows, kp0 = (int64_t)u * kMxPad;
        has_col = m.group != g.n_groups;
    } else {
        mx_tile_of(blockIdx.x, units * (unsigned)g.batch, col_tiles, u, ct);
        b = u / units, u = u % units;
        row0 = kp0 = (int64_t)u * kMxPad;
        rows = g.rows - row0 < kMxPad ? g.rows - row0 : kMxPad;
    }
    const int64_t c0 = (int64_t)ct * 128;
    const int tr = t >> 3, tc = t & 7;      // this lane's row and 16 columns of a step
    const int64_t first = (b * g.rows + row0) * g.row_kp + c0 + tc * 16;
    Kept16 x[kSteps];
    const auto load = [&](auto stream) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = tr + 32 * i;
            x[i] = load_kept16<decltype(stream)::value>(g, first + (r < rows ? r : 0) * g.row_kp);
        }
    };
    if (g.stream) load(std::true_type{});
    else load(std::false_type{});
    if (rows < kMxPad || c0 + 128 > g.cols) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) keep16(x[i], tr + 32 * i < rows ? g.cols - c0 - tc * 16 : 0);
    }
    if (has_col) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = tr + 32 * i;
            *(int4v*)(tile + r * 128 + ((tc * 16) ^ (32 * i))) = x[i].w;
            if ((tc & 1) == 0) factors[(tc >> 1) * kKeptStride + r] = mx8_factor(x[i].code);
        }
    }
    if (g.rc) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = tr + 32 * i;
            const Oct16 v = values_of(x[i]);
            const uint32_t code = pair_scale(v, g.above);
            const int64_t e = first + r * g.row_kp;
            const uint32_t w0 = codes_of<SR>(v.o[0], code, g.sr_row, e, 0, g);
            const uint32_t w1 = codes_of<SR>(v.o[1], code, g.sr_row, e + 8, 0, g);
            const uint32_t sc = join8(code << (8 * (tc >> 1)));
            if (r < rows) {
                *(uint2*)(g.rc + e / 2) = make_uint2(w0, w1);
                if (tc == 0) *(uint32_t*)(g.rs + e / 32) = sc;
            }
        }
    }
    if (!has_col) return;
    __syncthreads();
    // columns 4 dc .. 4 dc + 3, rows 16 h .. 16 h + 15
    const int h = t & 7, dc = t >> 3, rb = h >> 1;
    const uint8_t* s = tile + h * 16 * 128 + ((dc * 4) ^ (32 * rb));
    const float* f = factors + (dc >> 3) * kKeptStride + h * 16;
    uint32_t d[2][16], m[2] = {};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t w = *(const uint32_t*)(s + j * 128);
        d[0][j] = kept_pair(w, f[j], false), d[1][j] = kept_pair(w, f[j], true);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int j = 0; j < 16; ++j) m[p] = max_bf16x2(m[p], d[p][j] & 0x7FFF7FFFu);
        m[p] = max_bf16x2(m[p], (uint32_t)dpp<kXor1>(0, (int)m[p]));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t* v = d[q >> 1];
        const uint32_t code = mx_scale_code(q & 1 ? m[q >> 1] & 0xFFFF0000u : m[q >> 1] << 16, g.above);
        const int64_t c = c0 + dc * 4 + q, e = (b * g.cols + c) * g.col_kp + kp0 + h * 16;
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            Oct<uint16_t> o;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o.w[j] = __builtin_amdgcn_perm(v[8 * k + 2 * j + 1], v[8 * k + 2 * j], q & 1 ? 0x07060302u : 0x05040100u);
            w[k] = codes_of<SR>(o, code, g.sr_col, e + 8 * k, 1, g);
        }
        const uint32_t sc = join8(code << (8 * rb));
        if (c < g.cols) {
            *(uint2*)(g.cc + e / 2) = make_uint2(w[0], w[1]);
            if (h == 0) *(uint32_t*)(g.cs + e / 32) = sc;
        }
    }
}

struct MxDArgs {
    const uint8_t *codes, *scales;
    int64_t n, k, kp;
    const int32_t* offsets;
    int n_groups;
    void* out;
    int64_t ld;
};

// A lane's decoded elements as four dwords.  bfloat16: exact for copies of bfloat16 values,
// nearest even otherwise.
template <typename T>
__device__ __forceinline__ int4v decode_piece(uint32_t w, uint32_t code) {
    constexpr int n = Piece<T>::n;
    const float s = code == 255u ? __builtin_nanf("") : mx_scale_value(code);
    const float2v v[4] = {fp4x2_to_f32<0>(w), fp4x2_to_f32<1>(w), fp4x2_to_f32<2>(w), fp4x2_to_f32<3>(w)};
    T e[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const float f = v[i >> 1][i & 1] * s;
        if constexpr (sizeof(T) == 2) e[i] = __builtin_bit_cast(uint16_t, (__bf16)f);
        else e[i] = f;
    }
    int4v d;
    __builtin_memcpy(&d, e, sizeof(d));
    return d;
}

// Plain copy: consecutive pieces of the padded copy, as k_mx_rows.
template <typename T>
__global__ __launch_bounds__(256) void k_mx_decode(MxDArgs g) {
    constexpr int n = Piece<T>::n;
    const uint32_t per = (uint32_t)(g.kp / n);
    const int64_t first = (int64_t)blockIdx.x * (256 * kRowSteps), total = g.n * per;
    const int64_t row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    uint32_t w[kRowSteps], code[kRowSteps];
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const int64_t at = first + threadIdx.x + 256 * i;
        w[i] = at < total ? ((const typename Piece<T>::Codes*)g.codes)[at] : 0u;
        code[i] = at < total ? g.scales[at / (32 / n)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kRowSteps; ++i) {
        const uint32_t at = rem + threadIdx.x + 256 * i, dr = at / per;
        const int64_t r = row0 + dr, k = (int64_t)(at - dr * per) * n;
        const bool in = first + threadIdx.x + 256 * i < total;
        store_piece(decode_piece<T>(w[i], code[i]), (T*)g.out + r * g.ld + k, in ? g.k - k : 0,
                    k == 0 || (threadIdx.x & 63) == 0);
    }
}

// Grouped columnwise copy: a wave takes the positions of kDecodeUnits 128-row units in one row of the
// copy at a time, and a workgroup's four waves four such stretches, in all 4 KiB of output that is one
// run but for where groups end.  8192 x 4096 bfloat16 in 15 groups 22 us (27 with a workgroup on 64
// rows of one unit; plain 14), 12001 x 2048 in 64 groups 25 us (27; plain 10): what is left goes with
// the number of group ends in a row.
constexpr int kDecodeSteps = 4;
template <typename T> constexpr int kDecodeUnits = 64 * Piece<T>::n / kMxPad;
template <typename T>
__global__ __launch_bounds__(256) void k_mx_decode_grouped(MxDArgs g, unsigned unit_tiles, unsigned row_tiles) {
    constexpr int n = Piece<T>::n, kLanes = kMxPad / n, kUnits = kDecodeUnits<T>;
    unsigned ut, rt;
    mx_tile_of(blockIdx.x, unit_tiles, row_tiles, ut, rt);
    const int rows = (int)g.k, lane = threadIdx.x & 63, j = lane % kLanes * n;
    const int u0 = ((int)ut * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kUnits, u = u0 + lane / kLanes;
    // the stretch's units, from one pass over the offsets
    bool in = false;
    int at = 0, left = 0, found = 0, end = 0, units = 0;
    for (int base = 0; base < g.n_groups && found < kUnits; base += 64) {
        const MxSpan x = mx_span(g.offsets, g.n_groups, rows, kMxPad, base, end);
        for (; found < kUnits; ++found) {
            const uint64_t hit = __builtin_amdgcn_ballot_w64(units + x.p > u0 + found);
            if (!hit) break;
            const int of = __builtin_ctzll(hit);
            const int row = lane_value(x.s, of) + (u0 + found - units - lane_value(x.p - x.n, of)) * kMxPad;
            if (found == lane / kLanes) in = true, at = row + j, left = min(lane_value(x.e, of) - row, kMxPad) - j;
        }
        end = lane_value(x.e, 63);
        units += lane_value(x.p, 63);
    }
    // the rows in no group follow
    if (!in) at = end + (u - units) * kMxPad + j, left = min(rows - at, kMxPad - j);
    const int64_t row0 = (int64_t)rt * kDecodeSteps;
    uint32_t w[kDecodeSteps], code[kDecodeSteps];
#pragma unroll
    for (int i = 0; i < kDecodeSteps; ++i) {
        const int64_t r = row0 + i, e = r * g.kp + (int64_t)u * kMxPad + j;
        const bool ok = in && r < g.n;
        w[i] = ok ? *(const typename Piece<T>::Codes*)(g.codes + e / 2) : 0u;
        code[i] = ok ? g.scales[e / 32] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kDecodeSteps; ++i) {
        const int64_t r = row0 + i;
        store_piece(decode_piece<T>(w[i], code[i]), (T*)g.out + r * g.ld + at, r < g.n ? left : 0, j == 0);
    }
}

template <typename T>
static int launch_decode(const MxDArgs& g, hipStream_t st) {
    if (g.n_groups) {
        // one unit more than the copy holds: the rows in no group
        const int64_t row_tiles = (g.n + kDecodeSteps - 1) / kDecodeSteps;
        const int64_t unit_tiles = (g.kp / kMxPad + 4 * kDecodeUnits<T>) / (4 * kDecodeUnits<T>);
        const __int128 grid = (__int128)unit_tiles * row_tiles;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx_decode_grouped<T><<<dim3((unsigned)grid), 256, 0, st>>>(g, (unsigned)unit_tiles, (unsigned)row_tiles);
    } else {
        const int per = 256 * kRowSteps;
        const __int128 grid = ((__int128)g.n * (g.kp / Piece<T>::n) + per - 1) / per;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx_decode<T><<<dim3((unsigned)grid), 256, 0, st>>>(g);
    }
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename T, bool SR>
static int launch_quantize(const MxQArgs& g, hipStream_t st) {
    if (!g.cc) {
        const int per = 256 * kRowSteps;
        const __int128 grid = ((__int128)g.batch * g.rows * (g.row_kp / 8) + per - 1) / per;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx_rows<T, SR><<<dim3((unsigned)grid), 256, 0, st>>>(g);
    } else {
        // units cover the rows in no group too (one more partial unit at most); tiles cover the
        // rowwise copy's padding
        const int64_t units = g.col_kp / kMxPad, col_tiles = g.row_kp * (int64_t)sizeof(T) / 256;
        const __int128 grid = (g.n_groups ? units + 1 : (__int128)units * g.batch) * col_tiles;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx_tile<T, SR><<<dim3((unsigned)grid), 256, 0, st>>>(g, (unsigned)units, (unsigned)col_tiles);
    }
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <bool SR>
static int launch_kept(const MxQArgs& g, hipStream_t st) {
    if (!g.cc) {
        const __int128 grid = ((__int128)g.batch * g.rows * (g.row_kp / 16) + 255) / 256;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx8_rows<SR><<<dim3((unsigned)grid), 256, 0, st>>>(g);
    } else {
        const int64_t units = g.col_kp / kMxPad, col_tiles = g.row_kp / 128;
        const __int128 grid = (g.n_groups ? units + 1 : (__int128)units * g.batch) * col_tiles;
        if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
        k_mx8_tile<SR><<<dim3((unsigned)grid), 256, 0, st>>>(g, (unsigned)units, (unsigned)col_tiles);
    }
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// The arguments that mxfp4_quantize and mxfp8_to_mxfp4 share.  *used: there is anything to do.
static int check_copies(MxQArgs& g, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets, int64_t n_groups,
                        const mxfp4_quant_params* p, const mxfp4_tensor* row_out, const mxfp4_tensor* col_out,
                        bool* used) {
    const auto flag = [](int32_t v) { return v == 0 || v == 1; };
    if (!flag(p->rowwise) || !flag(p->colwise) || !(p->rowwise || p->colwise) || !flag(p->scale_rule) ||
        !flag(p->round_row) || !flag(p->round_col))
        return NVFP4_ERR_MODE;
    if (int rc = mx_check_groups(offsets, n_groups, rows)) return rc;
    if (n_groups && batch != 1) return NVFP4_ERR_MODE;
    *used = batch && rows && cols;
    if (p->rowwise)
        if (int rc = mx_check_tensor(row_out, *used)) return rc;
    if (p->colwise)
        if (int rc = mx_check_tensor(col_out, *used)) return rc;
    g.row_kp = mx_pad(cols);
    g.col_kp = n_groups ? mxfp4_grouped_k(rows, n_groups) : mx_pad(rows);
    g.batch = batch, g.rows = rows, g.cols = cols;
    g.offsets = offsets, g.n_groups = (int)n_groups;
    if (p->rowwise) g.rc = row_out->codes, g.rs = row_out->scales;
    if (p->colwise) g.cc = col_out->codes, g.cs = col_out->scales;
    g.k0 = (uint32_t)p->seed, g.k1 = (uint32_t)(p->seed >> 32);
    g.above = mx_above(p->scale_rule);
    g.sr_row = p->round_row == NVFP4_SR, g.sr_col = p->round_col == NVFP4_SR;
    return NVFP4_OK;
}
static bool stochastic(const MxQArgs& g) { return (g.rc && g.sr_row) || (g.cc && g.sr_col); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int mxfp4_abi_version(void) { return MXFP4_ABI_VERSION; }

extern "C" int64_t mxfp4_padded_k(int64_t k) { return k > 0 ? mx_pad(k) : 0; }

extern "C" int64_t mxfp4_grouped_k(int64_t rows, int64_t n_groups) {
    if (rows <= 0 || n_groups <= 0) return 0;
    const int64_t busy = n_groups < rows ? n_groups : rows;
    return (rows + busy * (kMxPad - 1)) / kMxPad * kMxPad;
}

extern "C" int mxfp4_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols,
                              int64_t ld_x, int64_t batch_stride, const int32_t* offsets,
                              int64_t n_groups, const mxfp4_quant_params* p,
                              const mxfp4_tensor* row_out, const mxfp4_tensor* col_out, void* stream) {
    if (!p) return NVFP4_ERR_NULL;
    if (!mx_extent(batch) || !mx_extent(rows) || !mx_extent(cols) || ld_x < cols) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    MxQArgs g = {};
    bool used;
    if (int rc = check_copies(g, batch, rows, cols, offsets, n_groups, p, row_out, col_out, &used)) return rc;
    if (!used) return NVFP4_OK;
    if (!x) return NVFP4_ERR_NULL;
    if ((uintptr_t)x % size) return NVFP4_ERR_ALIGN;
    g.x = x, g.ld = ld_x, g.stride = batch_stride;
    const hipStream_t st = (hipStream_t)stream;
    // An input of half the last-level cache (256 MB) or more is not still there from its
    // producer, whose own operands went through as well: past the caches 8192 x 9216 bfloat16
    // takes 50 us against 58 when it comes from memory, but 47 against 39 when it is cached.
    g.stream = (__int128)batch * rows * cols * size >= ((int64_t)128 << 20);
    const bool sr = stochastic(g);
    if (dtype == NVFP4_BF16) return sr ? launch_quantize<uint16_t, true>(g, st) : launch_quantize<uint16_t, false>(g, st);
    return sr ? launch_quantize<float, true>(g, st) : launch_quantize<float, false>(g, st);
}

extern "C" int mxfp8_to_mxfp4(const mxfp8_tensor* q, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets,
                              int64_t n_groups, const mxfp4_quant_params* p, const mxfp4_tensor* row_out,
                              const mxfp4_tensor* col_out, void* stream) {
    if (!p) return NVFP4_ERR_NULL;
    if (!mx_extent(batch) || !mx_extent(rows) || !mx_extent(cols)) return NVFP4_ERR_SHAPE;
    MxQArgs g = {};
    bool used;
    if (int rc = check_copies(g, batch, rows, cols, offsets, n_groups, p, row_out, col_out, &used)) return rc;
    if (int rc = mx8_check_tensor(q, used)) return rc;
    if (!used) return NVFP4_OK;
    g.x = q->codes, g.xs = q->scales;
    g.stream = (__int128)batch * rows * g.row_kp >= ((int64_t)128 << 20);   // as in mxfp4_quantize
    return stochastic(g) ? launch_kept<true>(g, (hipStream_t)stream) : launch_kept<false>(g, (hipStream_t)stream);
}

extern "C" int mxfp4_dequantize(const mxfp4_tensor* q, int64_t n, int64_t k, const int32_t* offsets,
                                int64_t n_groups, int out_dtype, void* out, int64_t ld_out,
                                void* stream) {
    if (!mx_extent(n) || !mx_extent(k) || ld_out < k) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(out_dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    if (int rc = mx_check_groups(offsets, n_groups, k)) return rc;
    if (int rc = mx_check_tensor(q, n && k)) return rc;
    if (n == 0 || k == 0) return NVFP4_OK;
    if (!out) return NVFP4_ERR_NULL;
    if ((uintptr_t)out % size) return NVFP4_ERR_ALIGN;
    MxDArgs g = {q->codes, q->scales, n, k, n_groups ? mxfp4_grouped_k(k, n_groups) : mx_pad(k),
                 offsets, (int)n_groups, out, ld_out};
    const hipStream_t st = (hipStream_t)stream;
    return out_dtype == NVFP4_BF16 ? launch_decode<uint16_t>(g, st) : launch_decode<float>(g, st);
}
