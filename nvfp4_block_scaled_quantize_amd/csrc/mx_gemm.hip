// mx_gemm.hip -- products of MXFP4 operands on gfx950's block-scaled matrix instructions.
//
// C[m][n] = sum over blocks of 2^(ea + eb - 254) sum_k a_k b_k.  v_mfma_scale_f32_32x32x64
// with both operands E2M1 multiplies 32 x 64 by 64 x 32 elements, scales each lane's 32
// elements of K by the E8M0 byte that the lane supplies, and accumulates in FP32.
//
// K ordering.  Lane l of an operand holds row l mod 32; lanes 0-31 supply the first 32 of an
// instruction's 64 k-slots and lanes 32-63 the others.
#include "mx_common.h"

namespace nvfp4 {

// ---------------------------------------------------------------- small tiles
//
// Products with too few 256 x 256 tiles for the card take 128 x 128 ones here, two workgroups a
// compute unit.  A workgroup of four waves computes a tile, wave (wm, wn) a quarter of it as
// 2 x 2 accumulators of 32 x 32.  K advances in stages of 128 elements (64 code bytes a row, the
// padding unit of the copies, so there is no partial stage).  Four stages of codes are in flight
// in LDS; a row's scale bytes come 32 at a time, for eight stages, into two buffers.  All of it
// is written by direct global -> LDS loads: row r's four 16-byte chunks lie at slots
// q ^ (r / 4 mod 4), which lets 16 consecutive rows' reads of one chunk touch every bank once, and
// the loads realise that order by which chunk each lane fetches.  Rows past the operand read as
// zeros (the loads' range check).
//
// A stage is two half-stages of 2 x 2 matrix instructions: half j multiplies chunk 2h + j of
// every row (h: the lane's half of the wave), whose scale is byte j of the 16 bits that the
// lane holds.  While a half-stage multiplies, the next one's fragments are read from LDS into
// a second set of registers; the one barrier of a stage stands between its halves, and the
// loads for three stages ahead are issued right after it.
//
// Measured: 2048 x 2048 x 4096 (256 tiles) 12 us, 2.9 PFLOP/s; 1024 x 1024 x 8192 (64 tiles) 20 us,
// bound by the time of one workgroup's stage (0.22 us: LDS reads and the barrier of a lone wave a
// SIMD); deeper prefetch (eight stages) and whole-stage read-ahead changed neither.
constexpr int kMxStage = 128, kMxStages = 4;

struct MxTile {
    static constexpr int kSide = 128;
    static constexpr int kCodes = kSide * 64;                    // code bytes of a stage, one operand
    static constexpr int kLoads = 4;                             // per wave and stage, two of each operand
    static constexpr int kScales = kMxStages * 2 * kCodes;       // LDS offset of the scales
    static constexpr int kScaleBuf = kSide * 32;                 // one operand, eight stages
    static constexpr int kLds = kScales + 4 * kScaleBuf;
};

template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename T, int MODE, bool STREAM>
__global__ __launch_bounds__(256, 1) void k_mx_tiles(MxGArgs g, unsigned tiles_n, unsigned tiles_m) {
    using Tile = MxTile;
    constexpr int TM = 2, TN = 2;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wid >> 1, wn = wid & 1, li = lane & 31, h = lane >> 5;
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;

    // the tile: rows [m0, m1) of A and C, rows [n0, N) of B, K from k0 (in elements)
    unsigned tm, tn;
    int64_t m0, m1 = g.M, k0 = 0;
    int nst = (int)(g.kp / kMxStage);
    const uint8_t *bc = g.bc, *bs = g.bs;
    T* c = (T*)g.c;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, Tile::kSide, blockIdx.x, tiles_n, tm, tn, u)) return;
        m0 = u.row0, m1 = u.row0 + u.rows;
        if (u.group == g.n_groups) nst = 0;
        else bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
    } else if constexpr (MODE == MxK) {
        mx_tile_of(blockIdx.x, tiles_m * g.n_groups, tiles_n, tm, tn);
        MxUnit u;
        mx_group(g.offsets, g.n_groups, (int)g.k_rows, kMxPad, (int)(tm / tiles_m), u);
        k0 = u.first * kMxPad, nst = (int)(mx_blocks(u.rows) / (kMxPad / kMxBlock));
        c += (int64_t)u.group * g.M * g.ldc;
        m0 = (int64_t)(tm % tiles_m) * Tile::kSide;
    } else {
        mx_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
        m0 = (int64_t)tm * Tile::kSide;
    }
    const int64_t n0 = (int64_t)tn * Tile::kSide;

    float16v acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    if (nst > 0) {
        const int ra = (int)(m1 - m0 < Tile::kSide ? m1 - m0 : Tile::kSide);
        const int rb = (int)(g.N - n0 < Tile::kSide ? g.N - n0 : Tile::kSide);
        const int4v rac = make_rsrc(g.ac + m0 * pitch + k0 / 2, (uint32_t)(ra * pitch - k0 / 2));
        const int4v ras = make_rsrc(g.as + m0 * spitch + k0 / 32, (uint32_t)(ra * spitch - k0 / 32));
        const int4v rbc = make_rsrc(bc + n0 * pitch + k0 / 2, (uint32_t)(rb * pitch - k0 / 2));
        const int4v rbs = make_rsrc(bs + n0 * spitch + k0 / 32, (uint32_t)(rb * spitch - k0 / 32));
        const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
        // this lane's global offsets within a stage (codes) and within four stages (scales)
        uint32_t off[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int q = (wid * 2 + i) * 64 + lane, row = q >> 2;
            off[i] = (uint32_t)(row * pitch) + (((q & 3) ^ ((row >> 2) & 3)) << 4);
        }
        // scales: a load covers 32 rows x 32 bytes, two waves load A's and two B's; row r's 16-byte halves
        // are exchanged where r / 8 is odd, so that 16 consecutive rows' reads of one half touch
        // every bank once
        const uint32_t srow0 = (uint32_t)(wid & 1) * 32;
        const int srow = (int)srow0 + (lane >> 1);
        const uint32_t os = (uint32_t)(srow * spitch) + (((lane ^ (srow >> 3)) & 1) << 4);

        // load number i of stage s (an offset past the operand where there is no such stage: the
        // count of loads in flight stays fixed)
        const auto load_codes = [&](int s, auto ic) {
            constexpr int i = decltype(ic)::value;
            const uint32_t buf = lds0 + (uint32_t)(s & 3) * (2 * Tile::kCodes);
            const uint32_t k = s < nst ? (uint32_t)s * 64 : kOutOfRange;
            dma16(i < 2 ? rac : rbc, buf + (i < 2 ? 0 : Tile::kCodes) + (uint32_t)(wid * 2 + (i & 1)) * 1024, off[i & 1] + k);
        };
        // part 0 or 1 (half the rows) of the scales of eight stages
        const auto load_scales = [&](int grp, int part) {
            const uint32_t buf = lds0 + Tile::kScales + (uint32_t)(grp & 1) * (2 * Tile::kScaleBuf);
            const uint32_t row = (uint32_t)part * (Tile::kSide / 2), at = (row + srow0) * 32;
            const uint32_t k = grp * 8 < nst ? os + row * (uint32_t)spitch + (uint32_t)grp * 32 : kOutOfRange;
            if (wid < 2) dma16(ras, buf + at, k);
            else dma16(rbs, buf + Tile::kScaleBuf + at, k);
        };
        const auto frag = [&](int s, bool b, int tile, int j) -> int4v {
            const int row = (b ? wn * (Tile::kSide / 2) : wm * (Tile::kSide / 2)) + tile * 32 + li;
            const uint8_t* p = lds + (s & 3) * (2 * Tile::kCodes) + (b ? Tile::kCodes : 0) + row * 64 +
                               (((2 * h + j) ^ ((row >> 2) & 3)) << 4);
            return *(const int4v*)p;
        };
        const auto scale = [&](int s, bool b, int tile) -> int {
            const int row = (b ? wn * (Tile::kSide / 2) : wm * (Tile::kSide / 2)) + tile * 32 + li;
            const uint8_t* p = lds + Tile::kScales + ((s >> 3) & 1) * (2 * Tile::kScaleBuf) +
                               (b ? Tile::kScaleBuf : 0) + row * 32 + ((((s >> 2) ^ (row >> 3)) & 1) << 4) +
                               (s & 3) * 4 + 2 * h;
            return *(const uint16_t*)p;
        };

        load_scales(0, 0);
        load_scales(0, 1);
        static_for<0, Tile::kLoads>([&](auto i) { load_codes(0, i); });
        static_for<0, Tile::kLoads>([&](auto i) { load_codes(1, i); });
        static_for<0, Tile::kLoads>([&](auto i) { load_codes(2, i); });
        wait_loads_and_barrier<2 * Tile::kLoads>();

        int4v a0[TM], b0[TN], a1[TM], b1[TN];
        int sa[TM], sb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) a0[i] = frag(0, false, i, 0), sa[i] = scale(0, false, i);
#pragma unroll
        for (int j = 0; j < TN; ++j) b0[j] = frag(0, true, j, 0), sb[j] = scale(0, true, j);

        // Q: stage mod 4, which decides the loads in flight
        const auto stage = [&](int s, auto qc) {
            constexpr int Q = decltype(qc)::value;
            int na[TM], nb[TN];
            // first half: multiply chunk 0, read chunk 1
            static_for<0, TM * TN>([&](auto mc) {
                constexpr int m = decltype(mc)::value, i = m / TN, j = m % TN;
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    mx_frag(b0[j]), mx_frag(a0[i]), acc[i][j], kE2M1, kE2M1, 0, sb[j], 0, sa[i]);
                if constexpr (m < TN) b1[m] = frag(s, true, m, 1);
                else if constexpr (m < TM + TN) a1[m - TN] = frag(s, false, m - TN, 1);
                __builtin_amdgcn_sched_barrier(0);
            });
            // stage s + 1 has landed; in flight: stage s + 2, and the scales issued a stage (Q 1)
            // or two stages (Q 2) ago
            wait_loads_and_barrier<Tile::kLoads + (Q == 1 || Q == 2 ? 1 : 0)>();
            // second half: multiply chunk 1; issue the loads of stage s + 3 and read chunk 0 of s + 1
            static_for<0, TM * TN>([&](auto mc) {
                constexpr int m = decltype(mc)::value, i = m / TN, j = m % TN;
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    mx_frag(b1[j]), mx_frag(a1[i]), acc[i][j], kE2M1, kE2M1, 1, sb[j], 1, sa[i]);
                load_codes(s + 3, mc);
                if constexpr (m < TN) b0[m] = frag(s + 1, true, m, 0), nb[m] = scale(s + 1, true, m);
                else if constexpr (m < TM + TN)
                    a0[m - TN] = frag(s + 1, false, m - TN, 0), na[m - TN] = scale(s + 1, false, m - TN);
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (Q == 0) load_scales(s / 8 + 1, (s >> 2) & 1);
#pragma unroll
            for (int i = 0; i < TM; ++i) sa[i] = na[i];
#pragma unroll
            for (int j = 0; j < TN; ++j) sb[j] = nb[j];
        };
        int s = 0;
        for (; s + 4 <= nst; s += 4) {
            stage(s, std::integral_constant<int, 0>{});
            stage(s + 1, std::integral_constant<int, 1>{});
            stage(s + 2, std::integral_constant<int, 2>{});
            stage(s + 3, std::integral_constant<int, 3>{});
        }
        if (s < nst) stage(s, std::integral_constant<int, 0>{}), ++s;
        if (s < nst) stage(s, std::integral_constant<int, 1>{}), ++s;
        if (s < nst) stage(s, std::integral_constant<int, 2>{});
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may write LDS after the wave's end
    }

    // Epilogue.  Register r of lane l is column 8 (r / 4) + 4 (l / 32) + r % 4, row l % 32 of its
    // 32 x 32: a wave puts 32 rows of its part of C into LDS (its own piece, behind the barrier
    // that ends the stages' use of it) and stores them from there 16 bytes a lane, a row's 128 or
    // 64 columns contiguous.
    asm volatile("s_barrier" ::: "memory");
    constexpr int kCols = TN * 32, kRowBytes = kCols * (int)sizeof(T) + 16;
    constexpr int kPer = 16 / (int)sizeof(T), kLanes = kCols / kPer, kRowsAtOnce = 64 / kLanes;
    static_assert(4 * 32 * kRowBytes <= Tile::kLds, "the epilogue's rows fit");
    uint8_t* piece = lds + wid * (32 * kRowBytes);
    const int64_t col = n0 + wn * (Tile::kSide / 2) + (lane % kLanes) * kPer;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                put_c4((T*)(piece + li * kRowBytes) + j * 32 + 2 * r + 4 * h, acc[i][j][r], acc[i][j][r + 1],
                       acc[i][j][r + 2], acc[i][j][r + 3]);
        const int64_t row0 = m0 + wm * (Tile::kSide / 2) + i * 32 + lane / kLanes;
#pragma unroll
        for (int k = 0; k < 32 / kRowsAtOnce; ++k) {
            const int4v v = *(const int4v*)(piece + (k * kRowsAtOnce + lane / kLanes) * kRowBytes + (lane % kLanes) * 16);
            const int64_t row = row0 + k * kRowsAtOnce;
            if (row < m1) store_c16<STREAM>(c + row * g.ldc + col, v, g.N - col);
        }
    }
}

template <typename T, int MODE, bool STREAM>
static int launch_tiles(const MxGArgs& g, hipStream_t st) {
    using Tile = MxTile;
    const int64_t tn = (g.N + Tile::kSide - 1) / Tile::kSide, tm = (g.M + Tile::kSide - 1) / Tile::kSide;
    int64_t tiles = tm * tn;
    // every group, and the rows in none, may end in a partial tile
    if (MODE == MxRows) tiles = (g.M / Tile::kSide + (g.n_groups < g.M ? g.n_groups : g.M) + 1) * tn;
    if (MODE == MxK) tiles *= g.n_groups;
    static_assert(Tile::kLds <= kMxMaxLds, "LDS budget");
    if (!mx_grid_fits(tiles, 256)) return NVFP4_ERR_SHAPE;
    const auto kernel = k_mx_tiles<T, MODE, STREAM>;
    static std::atomic<uint64_t> ready{0};
    if (int rc = mx_allow_lds((const void*)kernel, Tile::kLds, ready)) return rc;
    kernel<<<dim3((unsigned)tiles), 256, Tile::kLds, st>>>(g, (unsigned)tn, (unsigned)tm);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// How C is stored.  bfloat16 streams past the caches (grouped 16384 x 4096 x 2048 99 us against
// 103 with ordinary stores, and about the same where a quantizer reads C back: 8192 x 9216 x
// 4096 190 against 186 us, 2048 x 4096 x 2048 20.7 against 22.7).  float32 does where little of C
// would still be in the last-level cache (256 MB) for its reader: 15 gradients of 4096 x 2048
// (503 MB) 130 against 171 us, 15 of 1536 x 2048 (189 MB) 49.5 against 53.2; but 134 MB with a
// reader 84 against 74.
static bool streams(const MxGArgs& g, int mode) {
    return g.M * g.N * 4 * (mode == MxK ? g.n_groups : 1) >= ((int64_t)160 << 20);
}

// Which tile.  256 x 256 tiles run one to a compute unit, 256 at a time; 128 x 128 tiles two to a
// unit.  In percent of a round of the large ones, 512 small ones take 68 and up to 256 of them 45
// (8192^3: 4 rounds 249 us against 8 351 us; 2048 x 2048 x 4096 with 256 small tiles 11.3 us), so
// the small tile wins where the large ones' last round would be mostly empty: 2048 x 9216 x 4096
// (288 large tiles) 51 against 58 us, 1024 x 6144 x 4096 (96) 18 against 24, but 1024 x 9216 x
// 4096 (144 large, 576 small) 30 against 25.  Groups of rows end in half a tile on average.
template <int MODE>
static int launch_gemm(const MxGArgs& g, int c_dtype, hipStream_t st) {
    const auto tiles = [&](int64_t side) {
        int64_t m = (g.M + side - 1) / side;
        if (MODE == MxRows) m = (2 * g.M / side + (g.n_groups < g.M ? g.n_groups : g.M) + 1) / 2;
        return m * ((g.N + side - 1) / side) * (MODE == MxK ? g.n_groups : 1);
    };
    const int64_t big = (tiles(256) + 255) / 256 * 100, n = tiles(128), rest = n % 512;
    const int64_t small = n / 512 * 68 + (rest == 0 ? 0 : rest <= 256 ? 45 : 68);
    if (big <= small) return mx_tile256(g, MODE, c_dtype, streams(g, MODE), st);
    if (c_dtype == NVFP4_BF16) return launch_tiles<uint16_t, MODE, true>(g, st);
    return streams(g, MODE) ? launch_tiles<float, MODE, true>(g, st) : launch_tiles<float, MODE, false>(g, st);
}

// Checks shared by the products; *empty when C has no elements.
static int check_gemm(const mxfp4_tensor* a, const mxfp4_tensor* b, int64_t M, int64_t N, int64_t K,
                      const void* c, int c_dtype, int64_t ldc, bool* empty) {
    if (M < 0 || N < 0 || K < 0 || ldc < N || K > kMxMaxK) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(c_dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    if (int rc = mx_check_tensor(a, M && K)) return rc;
    if (int rc = mx_check_tensor(b, N && K)) return rc;
    *empty = M == 0 || N == 0;
    if (*empty) return NVFP4_OK;
    if (!c) return NVFP4_ERR_NULL;
    return (uintptr_t)c % size ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int mxfp4_gemm(const mxfp4_tensor* a, const mxfp4_tensor* b, int64_t M, int64_t N,
                          int64_t K, void* c, int c_dtype, int64_t ldc, void* stream) {
    bool empty;
    if (int rc = check_gemm(a, b, M, N, K, c, c_dtype, ldc, &empty)) return rc;
    if (empty) return NVFP4_OK;
    const MxGArgs g = {a->codes, a->scales, b->codes, b->scales, M, N, mx_pad(K), 0, c, ldc, nullptr, 0};
    // Up to 16 rows go to the kernel that streams B once (16 x 6144 x 4096 7.3 us against 10.9).
    if (M <= 16 && mx_few_fits(M, g.kp)) return mx_few_packed({g, nullptr, 0, K, 0}, c_dtype, (hipStream_t)stream);
    return launch_gemm<MxDense>(g, c_dtype, (hipStream_t)stream);
}

extern "C" int mxfp4_gemm_grouped(const mxfp4_tensor* a, const mxfp4_tensor* b, const int32_t* offsets,
                                  int64_t n_groups, int64_t M, int64_t N, int64_t K, void* c,
                                  int c_dtype, int64_t ldc, void* stream) {
    bool empty;
    if (int rc = check_gemm(a, b, M, N, K, c, c_dtype, ldc, &empty)) return rc;
    if (n_groups < 1) return NVFP4_ERR_SHAPE;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (empty) return NVFP4_OK;
    const MxGArgs g = {a->codes, a->scales, b->codes, b->scales, M, N, mx_pad(K), 0, c, ldc,
                       offsets, (int)n_groups};
    return launch_gemm<MxRows>(g, c_dtype, (hipStream_t)stream);
}

extern "C" int mxfp4_gemm_grouped_wgrad(const mxfp4_tensor* a, const mxfp4_tensor* b,
                                        const int32_t* offsets, int64_t n_groups, int64_t M, int64_t N,
                                        int64_t rows, void* c, int c_dtype, int64_t ldc, void* stream) {
    bool empty;
    if (rows < 0 || n_groups < 1) return NVFP4_ERR_SHAPE;
    if (int rc = mx_check_groups(offsets, n_groups, rows)) return rc;
    const int64_t kp = mxfp4_grouped_k(rows, n_groups);
    if (int rc = check_gemm(a, b, M, N, kp, c, c_dtype, ldc, &empty)) return rc;
    if (empty) return NVFP4_OK;
    const MxGArgs g = {a->codes, a->scales, b->codes, b->scales, M, N, kp, rows, c, ldc,
                       offsets, (int)n_groups};
    return launch_gemm<MxK>(g, c_dtype, (hipStream_t)stream);
}

static size_t linear_code_bytes(int64_t M, int64_t K) {
    return ((size_t)(M * (mx_pad(K) / 2)) + 255) / 256 * 256;
}

// Few rows are quantized inside the product, which saves a launch and the workspace, as long as
// every workgroup's doing so costs less: 8 rows of 6144 x 4096 10.9 against 10.0 us of GPU time
// with one launch less of host time; 16 rows 16.2 against 10.5.  For groups the same per group:
// 24 rows over 17 groups 21.5 against 22.1 us, 80 rows 27.5 against 22.6.
static bool linear_fused(int64_t M, int64_t K, int64_t n_groups) {
    const int64_t busy = n_groups < M ? n_groups : M;
    return M > 0 && K > 0 && mx_few_fits(M, mx_pad(K)) && (n_groups ? M <= 2 * busy : M <= 8);
}

extern "C" size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    (void)N;
    return M > 0 && K > 0 && !linear_fused(M, K, n_groups) ? linear_code_bytes(M, K) + (size_t)(M * (mx_pad(K) / 32)) : 0;
}

extern "C" int mxfp4_linear(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x,
                            int32_t scale_rule, const mxfp4_tensor* w, int64_t N, const int32_t* offsets,
                            int64_t n_groups, void* c, int c_dtype, int64_t ldc, void* ws,
                            size_t ws_bytes, void* stream) {
    if (M < 0 || K < 0) return NVFP4_ERR_SHAPE;
    const size_t need = mxfp4_linear_workspace_bytes(M, N, K, n_groups);
    if (need && (!ws || ws_bytes < need)) return NVFP4_ERR_WORKSPACE;
    if ((uintptr_t)ws & 255) return NVFP4_ERR_ALIGN;
    const mxfp4_tensor q = {(uint8_t*)ws, (uint8_t*)ws + (need ? linear_code_bytes(M, K) : 0)};
    const mxfp4_quant_params p = {1, 0, scale_rule, NVFP4_RNE, NVFP4_RNE, 0};
    // the product's arguments are checked before the quantization is enqueued (without a workspace
    // there is no packed A to check)
    bool empty;
    if (int rc = check_gemm(need ? &q : w, w, M, N, K, c, c_dtype, ldc, &empty)) return rc;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (x && linear_fused(M, K, n_groups)) {
        if (const int size = mx_dtype_size(dtype); !size) return NVFP4_ERR_DTYPE;
        else if ((uintptr_t)x % size) return NVFP4_ERR_ALIGN;
        if (ld_x < K) return NVFP4_ERR_SHAPE;
        if (scale_rule != MXFP4_SCALE_FLOOR && scale_rule != MXFP4_SCALE_CEIL) return NVFP4_ERR_MODE;
        if (empty) return NVFP4_OK;
        const MxFArgs f = {{nullptr, nullptr, w->codes, w->scales, M, N, mx_pad(K), 0, c, ldc, offsets, (int)n_groups},
                           x, ld_x, K, mx_above(scale_rule)};
        return mx_few_linear(f, dtype, c_dtype, (hipStream_t)stream);
    }
    if (int rc = mxfp4_quantize(x, dtype, 1, M, K, ld_x, 0, nullptr, 0, &p, &q, nullptr, stream)) return rc;
    return n_groups ? mxfp4_gemm_grouped(&q, w, offsets, n_groups, M, N, K, c, c_dtype, ldc, stream)
                    : mxfp4_gemm(&q, w, M, N, K, c, c_dtype, ldc, stream);
}
