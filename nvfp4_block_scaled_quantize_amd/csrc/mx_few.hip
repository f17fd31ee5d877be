// mx_few.hip -- MXFP4 products with few rows of A or few tiles in all: the forward for single
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
#include "mx_common.h"

#include <atomic>
#include <type_traits>

namespace nvfp4 {

constexpr int kFewRows = 16;
constexpr int kFewBatch = 4;                 // K steps of 128 in one batch of loads (of scales: 16 bytes)
// LDS row strides of A: 64 and 4 bytes past the row, so that 16 rows' reads spread over the banks
__host__ __device__ constexpr int few_code_stride(int kp) { return kp / 2 + 64; }
__host__ __device__ constexpr int few_scale_stride(int kp) { return kp / 32 + 4; }
inline int64_t few_lds(int64_t kp, int64_t M, int waves, int blocks) {
    const int64_t rows = M < kFewRows * blocks ? M : kFewRows * blocks;
    const int64_t a = rows * (kp / 2 + 64 + kp / 32 + 4), sums = waves * blocks * 16 * 17 * 4;
    return a > sums ? a : sums;
}
inline bool few_fits(int64_t kp, int64_t M, int blocks) { return few_lds(kp, M, 8, blocks) <= kMxMaxLds; }

// At most 16 rows of an operand; an offset past them, kFewNone for one, reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_buffer(const uint8_t* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ int4v few_load16(__amdgpu_buffer_rsrc_t b, int at) {
    return __builtin_bit_cast(int4v, __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0));
}
constexpr int kFewNone = 0x7FFFFFF0;

// XT: uint8_t (A packed), uint16_t or float (x).
template <typename T, typename XT, int MODE, int NT, int WAVES, int BLOCKS>
__global__ __launch_bounds__(64 * WAVES) void k_mx_few(MxFArgs f, unsigned tiles_n) {
    constexpr int kThreads = 64 * WAVES;
    constexpr int kSubs = NT / 16, kSplit = WAVES / kSubs;      // the waves' columns and K parts
    constexpr int kRows = kFewRows * BLOCKS;
    const MxGArgs& g = f.g;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int li = lane & 15, q = lane >> 4, sub = wid % kSubs, part = wid / kSubs;
    unsigned tn, tu;
    int64_t m0 = 0;
    int rows = (int)g.M, steps = (int)(g.kp / 128);
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    const uint8_t *bc = g.bc, *bs = g.bs;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, kRows, blockIdx.x, tiles_n, tu, tn, u)) return;
        m0 = u.row0, rows = (int)u.rows;
        if (u.group == g.n_groups) steps = 0;
        else bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
    } else {
        mx_tile_of(blockIdx.x, (unsigned)((g.M + kRows - 1) / kRows), tiles_n, tu, tn);
        m0 = (int64_t)tu * kRows;
        rows = (int)(g.M - m0 < kRows ? g.M - m0 : kRows);
    }
    // Loads are checked against their operand's rows by the hardware, which returns zeros beyond
    // them: with no branch around a load none is waited for before its use.
    const int64_t n0 = (int64_t)tn * NT + sub * 16;
    const int cols = (int)(g.N - n0 < 0 ? 0 : g.N - n0 < 16 ? g.N - n0 : 16);
    const auto wc = few_buffer(bc + n0 * pitch, cols * pitch), ws = few_buffer(bs + n0 * spitch, cols * spitch);
    const int wc_at = (int)(li * pitch) + q * 16, ws_at = (int)(li * spitch);
    const int s0 = steps * part / kSplit, s1 = steps * (part + 1) / kSplit;

    // A load of 16 rows costs the address unit as much for 4 bytes a row as for 64, so a batch's
    // scales come in one (past a row's end they are not used).
    struct Batch {
        int4v w[kFewBatch], s;
    };
    const auto load = [&](Batch& b, int s) {
#pragma unroll
        for (int i = 0; i < kFewBatch; ++i)
            b.w[i] = few_load16(wc, s + i < s1 ? wc_at + (s + i) * 64 : kFewNone);
        b.s = few_load16(ws, s < s1 ? ws_at + s * 4 : kFewNone);
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
    float4v acc[BLOCKS] = {};
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
            const int at = in ? s + i : s1 - 1, sw = in ? b.s[i] >> (8 * q) : 0;
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j)
                acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    mx_frag(b.w[i]), mx_frag(*(const int4v*)(pa[j] + at * 64)), acc[j], kE2M1, kE2M1, 0, sw, 0,
                    ps[j][at * 4]);
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
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[((wid * BLOCKS + j) * 16 + li) * 17 + 4 * q + i] = acc[j][i];
    __syncthreads();
    for (int i = t; i < kRows * NT; i += kThreads) {
        const int row = i / NT, col = i % NT;
        const float* p = sums + ((col >> 4) * kRows + row) * 17 + (col & 15);
        float v = p[0];
#pragma unroll
        for (int w = 1; w < kSplit; ++w) v += p[w * kSubs * kRows * 17];
        const int64_t c = (int64_t)tn * NT + col;
        if (row < rows && c < g.N) store_c((T*)g.c + (m0 + row) * g.ldc + c, v);
    }
}

template <typename T, typename XT, int MODE, int NT, int WAVES, int BLOCKS = 1>
static int launch(const MxFArgs& f, int64_t units, hipStream_t st) {
    const int64_t tn = (f.g.N + NT - 1) / NT;
    if (!mx_grid_fits(units * tn, 64 * WAVES)) return NVFP4_ERR_SHAPE;
    const int lds = (int)few_lds(f.g.kp, f.g.M, WAVES, BLOCKS);
    const auto kernel = k_mx_few<T, XT, MODE, NT, WAVES, BLOCKS>;
    static std::atomic<uint64_t> ready{0};
    if (lds > 64 * 1024)
        if (int rc = mx_allow_lds((const void*)kernel, kMxMaxLds, ready)) return rc;
    kernel<<<dim3((unsigned)(units * tn)), 64 * WAVES, lds, st>>>(f, (unsigned)tn);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// The tile of a dense product (counts of workgroups: for an MI355X's 256 compute units).  Up to 16
// rows: 16 columns a workgroup.  Eight waves halve a wave's K (1 x 1024 x 8192 4.6 against 5.0 us,
// 16 x 6144 x 4096 6.1 against 6.3), but with more than about 448 workgroups four are enough and
// start sooner (1 x 16384 x 2048 5.3 against 6.5 us, 4 x 9216 x 2048 4.9 against 5.2).  More rows:
// the smallest tile that leaves no compute unit two workgroups, or else 32 x 32.  Packed, 32 x 1024
// x 4096: 16 x 16 4.0 us, 32 x 16 4.5; 128 x 1024 x 4096: 5.5, 4.7, 32 x 32 5.7; 64 x 6144 x 4096:
// 13.0, 9.4, 9.1.
struct FewTile {
    int blocks, cols;
    int64_t units, workgroups;
};
static FewTile few_tile(int64_t M, int64_t N) {
    const int64_t units = (M + 15) / 16, pairs = (M + 31) / 32, tn = (N + 15) / 16;
    if (units == 1 || units * tn <= 256) return {1, 16, units, units * tn};
    if (pairs * tn <= 256) return {2, 16, pairs, pairs * tn};
    return {2, 32, pairs, pairs * ((N + 31) / 32)};
}
template <typename T, typename XT>
static int launch_dense(const MxFArgs& f, hipStream_t st) {
    const FewTile t = few_tile(f.g.M, f.g.N);
    if (t.cols == 32) return launch<T, XT, MxDense, 32, 8, 2>(f, t.units, st);
    if (t.blocks == 2) return launch<T, XT, MxDense, 16, 8, 2>(f, t.units, st);
    if (t.workgroups > 448) return launch<T, XT, MxDense, 16, 4>(f, t.units, st);
    return launch<T, XT, MxDense, 16, 8>(f, t.units, st);
}

// Grouped: four waves on 16 rows and 32 columns, two of them sharing K (80 packed rows over 17
// groups, 4096 x 2048: 14.2 us against 16.4 with 16 columns and 15.4 with 64, which need no split),
// or on 16 columns where 32 would leave compute units without work (4 rows over 4 groups, 1024 x
// 2048: 3.3 us against 3.8), or on 32 rows and 64 columns, without a split, where the groups have
// more than about 12 rows (400 packed rows over 17 groups 17.8 us against 23.6; 200 rows 16.4
// either way) and there are workgroups for all compute units (1000 rows of x, 4096 x 128 over 16
// groups 12.8 against 23.5, 200 packed rows, 2048 x 256 over 8 groups, 480 of them, 4.6 against
// 4.9; but 100 of 1024 x 2048 over 8 groups, 192 of them, 6.7 against 5.8, 400 of x, 512 x 384 over
// 30, 344, 5.8 against 5.1). The rule is the same for A packed and x, so that both add their sums
// in the same order.
template <typename T, typename XT>
static int launch_rows(const MxFArgs& f, hipStream_t st) {
    // every group, and the rows in none, may end in a partial unit
    const int64_t busy = f.g.n_groups < f.g.M ? f.g.n_groups : f.g.M, units = f.g.M / 16 + busy + 1;
    const int64_t pairs = f.g.M / 32 + busy + 1;
    if (f.g.M > 12 * busy && pairs * ((f.g.N + 63) / 64) >= 448 && few_fits(f.g.kp, f.g.M, 2))
        return launch<T, XT, MxRows, 64, 4, 2>(f, pairs, st);
    if (units * ((f.g.N + 31) / 32) < 256) return launch<T, XT, MxRows, 16, 4>(f, units, st);
    return launch<T, XT, MxRows, 32, 4>(f, units, st);
}

bool mx_few_fits(int64_t M, int64_t kp) { return few_fits(kp, M, 1); }

bool mx_few_dense(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile(M, N);
    return (M <= 16 || t.workgroups <= 512) && few_fits(kp, M, t.blocks);
}

int64_t mx_few_quantized(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile(M, N);
    const int64_t rows = M < kFewRows * t.blocks ? M : kFewRows * t.blocks;
    return rows * kp * (t.workgroups > 256 ? t.workgroups : 256) / 256;
}

template <typename XT>
static int launch_x(const MxFArgs& f, int c_dtype, hipStream_t st) {
    if (f.g.n_groups) return c_dtype == NVFP4_BF16 ? launch_rows<uint16_t, XT>(f, st) : launch_rows<float, XT>(f, st);
    return c_dtype == NVFP4_BF16 ? launch_dense<uint16_t, XT>(f, st) : launch_dense<float, XT>(f, st);
}

int mx_few_packed(const MxFArgs& f, int c_dtype, hipStream_t st) { return launch_x<uint8_t>(f, c_dtype, st); }

int mx_few_linear(const MxFArgs& f, int x_dtype, int c_dtype, hipStream_t st) {
    return x_dtype == NVFP4_BF16 ? launch_x<uint16_t>(f, c_dtype, st) : launch_x<float>(f, c_dtype, st);
}

}  // namespace nvfp4
