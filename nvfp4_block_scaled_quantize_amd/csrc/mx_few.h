// mx_few.h -- MXFP4 products with few rows of A or few tiles in all: the forward for single
// tokens and batches of them, dense or grouped by expert, with A packed or quantized on the way.
//
// C[m][n] = Q(x_m) . w_n is bound by reading W (17/32 byte per element) and by latency.  A
// workgroup takes 16 BLOCKS rows and NT columns of C; each of its waves takes 16 of the columns and
// a part of K.  W's fragments come straight from memory into registers, a batch of K steps ahead (a
// load covers 16 rows x 64 contiguous bytes); the rows of A are put into LDS once per workgroup,
// quantized there from x while the first of W is on its way; the waves' partial sums meet in LDS at
// the end, in wave order.  v_mfma_scale_f32_16x16x128: lane l holds row l mod 16 and the 32
// elements of K at 32 (l / 16), with their scale byte.
//
// Measured (GPU time per call in a replayed graph, three sets of operands in turn): 1 x 6144 x
// 4096, x in bfloat16, 5.3 us (W alone at the rate of plain reads: 1.9 us, an empty kernel: about
// 2.4 us) against 8.2 as quantize and packed product; 16 rows, packed, 6.1 us against 10.7 by tiles; 24
// rows over 17 groups (4096 x 2048, 71 MB of W) 15.0 us.  With branches around the loads, whose
// joins wait for them, the packed 16 rows took 10.2 us.
//
// The gated feed-forward block's forward (KIND): columns of H instead of C, a wave's 16 of them from 16 rows of the
// gate's weights and 16 of the up projection's; or (NT = 8) eight of them from eight rows of each, as one fragment.
// 1 x 9216 x 4096 9.2 us (W, 40 MB, at the rate of plain reads 5.6, an empty kernel 2.4), 1 x 4096 x 2048 4.3,
// 24 rows over 17 of 32 groups, 1536 x 2048 (57 MB of W), 12.8.  Its backward: a product whose last step reads
// the checkpoint, a byte a column.
#pragma once
#include "mx_ffn.h"

#include <atomic>
#include <type_traits>

namespace nvfp4 {
namespace few {

// Activation and type of the results, which only a workgroup's last step looks at, are arguments; `b`: what the
// backward reads and writes besides.
struct FfnArgs {
    MxFArgs f;
    int act, bf16;
    struct Backward {
        const uint8_t *kc, *ks;
        int64_t np;
        void* h;
        int64_t ldh;
    } b;
};
template <int KIND> struct FewKind { using Args = FfnArgs; };
template <> struct FewKind<kProduct> { using Args = MxFArgs; };
__host__ __device__ inline const MxFArgs& few_args(const MxFArgs& a) { return a; }
__host__ __device__ inline const MxFArgs& few_args(const FfnArgs& a) { return a.f; }

constexpr int kFewRows = 16;
constexpr int kFewBatch = 4;                 // K steps of 128 in one batch of loads (of scales: 16 bytes)
// LDS row strides of A: 64 and 4 bytes past the row, so that 16 rows' reads spread over the banks
__host__ __device__ constexpr int few_code_stride(int kp) { return kp / 2 + 64; }
__host__ __device__ constexpr int few_scale_stride(int kp) { return kp / 32 + 4; }
inline int64_t few_lds(int64_t kp, int64_t M, int waves, int blocks, int weights = 1) {
    const int64_t rows = M < kFewRows * blocks ? M : kFewRows * blocks;
    const int64_t a = rows * (kp / 2 + 64 + kp / 32 + 4), sums = waves * blocks * weights * 16 * 17 * 4;
    return a > sums ? a : sums;
}
inline bool few_fits(int64_t kp, int64_t M, int blocks) { return few_lds(kp, M, 8, blocks) <= kMxMaxLds; }
// Whether a launch can count that many workgroups, of four waves each: the eight of others are for few of them.
inline bool few_launches(int64_t workgroups) { return mx_grid_fits(workgroups, 256); }

// The tile of a grouped product: four waves on 16 rows and 32 columns, two of them sharing K (80 packed
// rows over 17 groups, 4096 x 2048: 14.2 us against 16.4 with 16 columns and 15.4 with 64, which need no
// split), or on 16 columns where 32 would leave compute units without work (4 rows over 4 groups, 1024 x
// 2048: 3.3 us against 3.8), or on 32 rows and 64 columns, without a split, where the groups have
// more than about 12 rows (400 packed rows over 17 groups 17.8 us against 23.6; 200 rows 16.4
// either way) and there are workgroups for all compute units (1000 rows of x, 4096 x 128 over 16
// groups 12.8 against 23.5, 200 packed rows, 2048 x 256 over 8 groups, 480 of them, 4.6 against
// 4.9; but 100 of 1024 x 2048 over 8 groups, 192 of them, 6.7 against 5.8, 400 of x, 512 x 384 over
// 30, 344, 5.8 against 5.1). The rule is the same for A packed and x, so that both add their sums
// in the same order.
struct RowsTile {
    int blocks, cols;
    int64_t units, workgroups;
};
inline RowsTile rows_tile(int64_t M, int64_t N, int64_t kp, int64_t n_groups) {
    // every group, and the rows in none, may end in a partial unit
    const int64_t busy = n_groups < M ? n_groups : M, units = M / 16 + busy + 1, pairs = M / 32 + busy + 1;
    const auto tile = [&](int blocks, int cols, int64_t n) -> RowsTile { return {blocks, cols, n, n * ((N + cols - 1) / cols)}; };
    if (M > 12 * busy && pairs * ((N + 63) / 64) >= 448 && few_fits(kp, M, 2)) return tile(2, 64, pairs);
    if (units * ((N + 31) / 32) < 256) return tile(1, 16, units);
    return tile(1, 32, units);
}

// At most 16 rows of an operand; an offset past them, kFewNone for one, reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_buffer(const uint8_t* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ int4v few_load16(__amdgpu_buffer_rsrc_t b, int at) {
    return __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0));
}
constexpr int kFewNone = 0x7FFFFFF0;

// XT: uint8_t (A packed), uint16_t or float (x).
template <typename T, typename XT, int MODE, int NT, int WAVES, int BLOCKS, int KIND = kProduct>
__global__ __launch_bounds__(64 * WAVES) void k_mx_few(typename FewKind<KIND>::Args args, unsigned tiles_n) {
    constexpr bool kHalves = NT == 8;       // a fragment of W is half the gate's, half the up projection's
    constexpr int kThreads = 64 * WAVES, kW = kHalves ? 1 : kMxWeights<KIND>;
    const MxFArgs& f = few_args(args);
    constexpr int kSubs = kHalves ? 1 : NT / 16, kSplit = WAVES / kSubs;      // the waves' columns and K parts
    constexpr int kRows = kFewRows * BLOCKS;
    const MxGArgs& g = f.g;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int li = lane & 15, q = lane >> 4, sub = wid % kSubs, part = wid / kSubs;
    unsigned tn, tu;
    int64_t m0 = 0;
    [[maybe_unused]] bool none = false;     // the rows are in no group
    int rows = (int)g.M, steps = (int)(g.kp / 128);
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    const uint8_t *bc = g.bc, *bs = g.bs;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, kRows, blockIdx.x, tiles_n, tu, tn, u)) return;
        m0 = u.row0, rows = (int)u.rows;
        none = u.group == g.n_groups;
        if (none) steps = 0;
        else bc += u.group * kMxWeights<KIND> * g.N * pitch, bs += u.group * kMxWeights<KIND> * g.N * spitch;
    } else {
        mx_tile_of(blockIdx.x, (unsigned)((g.M + kRows - 1) / kRows), tiles_n, tu, tn);
        m0 = (int64_t)tu * kRows;
        rows = (int)(g.M - m0 < kRows ? g.M - m0 : kRows);
    }
    // Loads are checked against their operand's rows by the hardware, which returns zeros beyond
    // them: with no branch around a load none is waited for before its use.
    const int64_t n0 = (int64_t)tn * NT + sub * 16;
    constexpr int kCols = kHalves ? 8 : 16;
    const int cols = (int)(g.N - n0 < 0 ? 0 : g.N - n0 < kCols ? g.N - n0 : kCols);
    __amdgpu_buffer_rsrc_t wc[kW], ws[kW];
    int wc_at = (int)(li * pitch) + q * 16, ws_at = (int)(li * spitch);
    if constexpr (kHalves) {
        // from the gate's first row here to the matrix's end, below 2^31 bytes; lanes without a column read none
        wc[0] = few_buffer(bc + n0 * pitch, (2 * g.N - n0) * pitch), ws[0] = few_buffer(bs + n0 * spitch, (2 * g.N - n0) * spitch);
        const int64_t row = (li & 7) + (li < 8 ? 0 : g.N);
        wc_at = (li & 7) < cols ? (int)(row * pitch) + q * 16 : kFewNone - (int)pitch;
        ws_at = (li & 7) < cols ? (int)(row * spitch) : kFewNone - (int)pitch;
    } else {
#pragma unroll
        for (int j = 0; j < kW; ++j) {
            wc[j] = few_buffer(bc + (j * g.N + n0) * pitch, cols * pitch);
            ws[j] = few_buffer(bs + (j * g.N + n0) * spitch, cols * spitch);
        }
    }
    const int s0 = steps * part / kSplit, s1 = steps * (part + 1) / kSplit;

    // A load of 16 rows costs the address unit as much for 4 bytes a row as for 64, so a batch's
    // scales come in one (past a row's end they are not used).
    struct Batch {
        int4v w[kW][kFewBatch], s[kW];
    };
    const auto load = [&](Batch& b, int s) {
#pragma unroll
        for (int j = 0; j < kW; ++j) {
#pragma unroll
            for (int i = 0; i < kFewBatch; ++i)
                b.w[j][i] = few_load16(wc[j], s + i < s1 ? wc_at + (s + i) * 64 : kFewNone);
            b.s[j] = few_load16(ws[j], s < s1 ? ws_at + s * 4 : kFewNone);
        }
    };
    // The first of x is asked for before W: loads return in order, and x has to be quantized
    // while W is on its way.  A lane takes eight elements, a quad a block.
    const int per = (int)(g.kp / 8), octs = steps ? rows * per : 0;
    const unsigned per_inverse = 0xFFFFFFFFu / (unsigned)per + 1;     // i / per, exact below 2^32 / per
    const auto load_x = [&](int i) -> Oct<XT> {
        const int r = (int)__umulhi((unsigned)i, per_inverse), k = (i - r * per) * 8;
        if constexpr (sizeof(XT) > 1) return load_oct((const XT*)f.x + (m0 + r) * f.ldx + k, i < octs ? f.K - k : 0);
        else return {};
    };
    constexpr int kAhead = 4;
    [[maybe_unused]] Oct<XT> o[kAhead];
    const auto load_ahead = [&](int b) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (b + j * kThreads < octs) o[j] = load_x(t + b + j * kThreads);
    };
    if constexpr (sizeof(XT) > 1) load_ahead(0);
    // Packed rows of A are one stretch of memory: a thread takes every kThreads-th 16 bytes of codes
    // and 4 of scales.  (Division of less than 2^16 by less than 2^16.)
    constexpr int kEach = 2 * BLOCKS, kEachScales = (kEach + 3) / 4;
    struct Piece {
        int4v c[kEach];
        int s[kEachScales];
    };
    const unsigned pieces = (unsigned)(g.kp / 32), inverse = 0xFFFFFFFFu / pieces + 1;
    const unsigned spieces = pieces / 4;
    const unsigned end = steps ? rows * pieces : 0, send = steps ? rows * spieces : 0;
    const auto ar = few_buffer(g.ac + m0 * pitch, rows * pitch), sr = few_buffer(g.as + m0 * spitch, rows * spitch);
    const auto load_a = [&](Piece& p, unsigned i, unsigned k) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) p.c[j] = few_load16(ar, (int)(i + j * kThreads) * 16);
#pragma unroll
        for (int j = 0; j < kEachScales; ++j)
            p.s[j] = __builtin_amdgcn_raw_buffer_load_b32(sr, (int)(k + j * kThreads) * 4, 0, 0);
    };
    [[maybe_unused]] Piece piece;
    if constexpr (sizeof(XT) == 1) load_a(piece, t, t);
    Batch cur;
    load(cur, s0);

    // A's rows into LDS
    uint8_t* ac = lds;
    const int cstride = few_code_stride((int)g.kp), sstride = few_scale_stride((int)g.kp);
    uint8_t* as = lds + rows * cstride;
    if constexpr (sizeof(XT) == 1) {
        for (unsigned i = t, k = t;;) {
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                const unsigned at = i + j * kThreads, r = __umulhi(at, inverse);
                if (at < end) *(int4v*)(ac + r * cstride + (at - r * pieces) * 16) = piece.c[j];
            }
#pragma unroll
            for (int j = 0; j < kEachScales; ++j) {
                const unsigned at = k + j * kThreads, r = __umulhi(at * 4, inverse);
                if (at < send) *(int*)(as + r * sstride + (at - r * spieces) * 4) = piece.s[j];
            }
            i += kEach * kThreads, k += kEachScales * kThreads;
            if (i - t >= end && k - t >= send) break;
            load_a(piece, i, k);
        }
    } else {
        const auto put_x = [&](int i, const Oct<XT>& x) {
            const int r = (int)__umulhi((unsigned)i, per_inverse), k = (i - r * per) * 8;
            const uint32_t code = mx_scale_code(quad_max(max_bits(x)), f.above);
            const uint32_t w = codes_rne(x, mx_scale_value(code));
            if (i >= octs) return;
            *(uint32_t*)(ac + r * cstride + k / 2) = code == 255u ? 0u : w;
            if ((t & 3) == 0) as[r * sstride + k / 32] = (uint8_t)code;
        };
        const auto put_ahead = [&](int b) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (b + j * kThreads < octs) put_x(t + b + j * kThreads, o[j]);
        };
        put_ahead(0);
        for (int b = kAhead * kThreads; b < octs; b += kAhead * kThreads) load_ahead(b), put_ahead(b);
    }
    __syncthreads();

    // rows past the last repeat it (their sums are not stored)
    float4v acc[kW][BLOCKS] = {};
    const uint8_t *pa[BLOCKS], *ps[BLOCKS];
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j) {
        const int r = li + j * 16 < rows ? li + j * 16 : rows - 1;
        pa[j] = ac + r * cstride + q * 16, ps[j] = as + r * sstride + q;
    }
    const auto multiply = [&](const Batch& b, int s, auto last) {
#pragma unroll
        for (int i = 0; i < kFewBatch; ++i) {
            // past the part's end W is zero, and its scale must not be NaN
            const bool in = !last || s + i < s1;
            const int at = in ? s + i : s1 - 1;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                const int sw = in ? b.s[k][i] >> (8 * q) : 0;
#pragma unroll
                for (int j = 0; j < BLOCKS; ++j)
                    acc[k][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        mx_frag(b.w[k][i]), mx_frag(*(const int4v*)(pa[j] + at * 64)), acc[k][j], kE2M1, kE2M1, 0, sw, 0,
                        ps[j][at * 4]);
            }
        }
    };
    Batch next;
    for (int s = s0; s < s1; s += 2 * kFewBatch) {
        if (s + kFewBatch >= s1) {
            multiply(cur, s, std::true_type{});
            break;
        }
        load(next, s + kFewBatch);
        multiply(cur, s, std::false_type{});
        if (s + 2 * kFewBatch >= s1) {
            multiply(next, s + kFewBatch, std::true_type{});
            break;
        }
        load(cur, s + 2 * kFewBatch);
        multiply(next, s + kFewBatch, std::false_type{});
    }
    __syncthreads();        // A's rows are done with: their LDS takes the partial sums

    // register i of lane l: column 4 (l / 16) + i, row l mod 16
    float* sums = (float*)lds;
    constexpr int kWave = kW * kRows * 17;      // a wave's sums
#pragma unroll
    for (int k = 0; k < kW; ++k)
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[wid * kWave + ((k * BLOCKS + j) * 16 + li) * 17 + 4 * q + i] = acc[k][j][i];
    __syncthreads();
    for (int i = t; i < kRows * NT; i += kThreads) {
        const int row = i / NT, col = i % NT;
        const float* p = sums + (col >> 4) * kWave + row * 17 + (col & 15);
        constexpr int kOther = kHalves ? 8 : kRows * 17;        // from the gate's sum to the up projection's
        float v[kMxWeights<KIND>];
#pragma unroll
        for (int k = 0; k < kMxWeights<KIND>; ++k) {
            v[k] = p[k * kOther];
#pragma unroll
            for (int w = 1; w < kSplit; ++w) v[k] += p[w * kSubs * kWave + k * kOther];
        }
        const int64_t c = (int64_t)tn * NT + col;
        if (row >= rows || c >= g.N) continue;
        if constexpr (KIND == kProduct) store_c((T*)g.c + (m0 + row) * g.ldc + c, v[0]);
        else if constexpr (KIND == kBackward) {
            const FfnArgs::Backward& b = args.b;
            const int64_t m = m0 + row, at = m * b.np + c, second = g.M * b.np;
            const float gate = mx8_values(b.kc[at], mx8_factor(b.ks[at / 32])).v[0];
            const float up = mx8_values(b.kc[second + at], mx8_factor(b.ks[(second + at) / 32])).v[0];
            const Act a = args.act == MXFP4_SILU ? act_both<MXFP4_SILU>(gate) : act_both<MXFP4_GELU>(gate);
            const float dg = none ? 0.0f : v[0] * up * a.slope, du = none ? 0.0f : v[0] * a.a, x = none ? 0.0f : a.a * up;
            const auto put = [&](auto* p, auto* h) {
                store_c(p + m * g.ldc + c, dg);
                store_c(p + m * g.ldc + g.N + c, du);
                if (h) store_c(h + m * b.ldh + c, x);
            };
            if (args.bf16) put((uint16_t*)g.c, (uint16_t*)b.h);
            else put((float*)g.c, (float*)b.h);
        } else {
            const float a = args.act == MXFP4_SILU ? act_value<MXFP4_SILU>(v[0]) : act_value<MXFP4_GELU>(v[0]);
            const int64_t at = (m0 + row) * g.ldc + c;
            if (args.bf16) store_c((uint16_t*)g.c + at, a * v[1]);
            else store_c((float*)g.c + at, a * v[1]);
        }
    }
}

template <typename T, typename XT, int MODE, int NT, int WAVES, int BLOCKS = 1, int KIND = kProduct>
inline int launch(const typename FewKind<KIND>::Args& args, int64_t units, hipStream_t st) {
    const MxFArgs& f = few_args(args);
    const int64_t tn = (f.g.N + NT - 1) / NT;
    if (!mx_grid_fits(units * tn, 64 * WAVES)) return NVFP4_ERR_SHAPE;
    const int lds = (int)few_lds(f.g.kp, f.g.M, WAVES, BLOCKS, kMxWeights<KIND>);
    const auto kernel = k_mx_few<T, XT, MODE, NT, WAVES, BLOCKS, KIND>;
    static std::atomic<uint64_t> ready{0};
    if (lds > 64 * 1024)
        if (int rc = mx_allow_lds((const void*)kernel, kMxMaxLds, ready)) return rc;
    kernel<<<dim3((unsigned)(units * tn)), 64 * WAVES, lds, st>>>(args, (unsigned)tn);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace few
}  // namespace nvfp4
