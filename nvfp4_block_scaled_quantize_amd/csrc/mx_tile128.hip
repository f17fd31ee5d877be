// mx_tile128.hip -- the small-tile kernel of the MXFP4 products: 128 x 128 tiles of C, a
// workgroup of four waves each, two workgroups a compute unit, for products that have too few
// 256 x 256 tiles to occupy the card.
//
// Wave (wm, wn) computes a 64 x 64 quarter as 2 x 2 accumulators of 32 x 32.  Stages, loads and the
// order of LDS are those of the large tile (mx_tile256.hip): 256 elements of K, 8 rows x 128 bytes
// a load, chunk q of row r at q ^ (r / 2 mod 8).  LDS holds SLOTS stages of codes (32 KiB each) and
// two buffers of scales (16 KiB): two stages for two workgroups a unit, or four for one where there
// are no more tiles than units (1024 x 1024 x 8192 18.0 us against 20.3; 8192 x 1024 x 8192 with
// four 43.4 against 40.1 with two).  A stage is 16 matrix instructions, four for each of its steps.
// While it multiplies, all fragments of the next one are read into a second set of registers; the
// loads of the stage after the next two go where LDS is free.  The barrier at a stage's start
// stands behind the wait for the next stage's loads.
//
// Measured: 8192 x 1024 x 8192 (512 tiles) 40 us, 3.4 PFLOP/s; 2048 x 9216 x 4096 (1152) 49 us;
// 1024 x 1024 x 8192 (64) 18 us, 77 x 4999 x 2056 (40) 9 us.  Bound by LDS: a workgroup's stage
// reads 64 KiB (512 clocks) and takes in 32 KiB (575) for 512 clocks of matrix instructions.
// Stages of 128 elements instead (16 rows x 64 bytes a load) took 45, 54, 20 and 8 us.
#include "mx_tile.h"

namespace nvfp4 {

constexpr int kSide = 128;
constexpr int kOperand = kSide * kRow, kSlot = 2 * kOperand;
constexpr int kScaleBuf = kSide * 32;                // one operand, four stages
constexpr int tile_lds(int slots) { return slots * kSlot + 4 * kScaleBuf; }
static_assert(2 * tile_lds(2) <= kMxMaxLds, "two workgroups a compute unit");

template <typename T, int MODE, bool STREAM, int SLOTS>
__global__ __launch_bounds__(256, SLOTS == 2 ? 2 : 1) void k_mx_tile128(MxGArgs g, unsigned tiles_n, unsigned tiles_m) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wid >> 1, wn = wid & 1, li = lane & 31, h = lane >> 5;
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    constexpr int kScalesAt = SLOTS * kSlot;        // LDS offset of the scale buffers

    // the tile: rows [m0, m1) of A and C, rows [n0, N) of B, K from k0 (in elements)
    unsigned tm, tn;
    int64_t m0, m1 = g.M, k0 = 0;
    int kbytes = (int)(g.kp / 2);       // code bytes of its K range
    const uint8_t *bc = g.bc, *bs = g.bs;
    T* c = (T*)g.c;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, kSide, blockIdx.x, tiles_n, tm, tn, u)) return;
        m0 = u.row0, m1 = u.row0 + u.rows;
        if (u.group == g.n_groups) kbytes = 0;
        else bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
    } else if constexpr (MODE == MxK) {
        mx_tile_of(blockIdx.x, tiles_m * g.n_groups, tiles_n, tm, tn);
        MxUnit u;
        mx_group(g.offsets, g.n_groups, (int)g.k_rows, kMxPad, (int)(tm / tiles_m), u);
        k0 = u.first * kMxPad, kbytes = (int)(mx_blocks(u.rows) * (kMxBlock / 2));
        c += (int64_t)u.group * g.M * g.ldc;
        m0 = (int64_t)(tm % tiles_m) * kSide;
    } else {
        mx_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
        m0 = (int64_t)tm * kSide;
    }
    const int64_t n0 = (int64_t)tn * kSide;

    float16v acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    if (kbytes > 0) {
        const int nst = (kbytes + kRow - 1) / kRow;
        const int ra = (int)(m1 - m0 < kSide ? m1 - m0 : kSide), rb = (int)(g.N - n0 < kSide ? g.N - n0 : kSide);
        const int4v rac = make_rsrc(g.ac + m0 * pitch + k0 / 2 - kBias, (uint32_t)(ra * pitch - k0 / 2 + kBias));
        const int4v rbc = make_rsrc(bc + n0 * pitch + k0 / 2 - kBias, (uint32_t)(rb * pitch - k0 / 2 + kBias));
        // two waves load A's scales and two B's
        const int4v rs = wid < 2 ? make_rsrc(g.as + m0 * spitch + k0 / 32, (uint32_t)(ra * spitch - k0 / 32))
                                 : make_rsrc(bs + n0 * spitch + k0 / 32, (uint32_t)(rb * spitch - k0 / 32));
        const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

        // Code load n of a stage: rows 32 wid + 8 n .. + 7 of A (n < 4), then the same of B.
        const int chunk = ((lane & 7) ^ (lane >> 4)) << 4;              // the lane's, for even n
        uint32_t row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            row[i] = (uint32_t)(wid * 32 + i * 8 + (lane >> 3)) * (uint32_t)pitch + (chunk ^ (i & 1) * 64);
        uint32_t past[2], kat;      // what lanes add for chunks past K (n even, odd); the K position
        const auto enter_stage = [&](int s) {
            const int left = kbytes - s * kRow;
            past[0] = chunk < left ? 0u : kOutOfRange;
            past[1] = (chunk ^ 64) < left ? 0u : kOutOfRange;
            kat = left > 0 ? (uint32_t)(s * kRow) : 0u;
        };
        const auto load_codes = [&](uint32_t slot, auto nc) {
            constexpr int n = decltype(nc)::value, i = n % 4;
            if constexpr (i == 0) set_m0(lds0 + slot + (n < 4 ? 0 : kOperand) + (uint32_t)wid * 4096);
            dma16_at<i * 1024>(n < 4 ? rac : rbc, row[i] + past[i & 1], kat + (kBias - i * 1024));
        };
        // The scales of four stages, two loads of 32 rows x 32 bytes a wave; row r's 16-byte halves are
        // exchanged where r / 8 is odd, for the banks' sake.
        const uint32_t srow = (uint32_t)((wid & 1) * 64 + (lane >> 1));
        const uint32_t soff = srow * (uint32_t)spitch + (((uint32_t)lane ^ (srow >> 3)) & 1) * 16;
        const auto load_scales = [&](int grp) {
            const uint32_t at = lds0 + kScalesAt + (uint32_t)(grp & 1) * 2 * kScaleBuf + (uint32_t)wid * 2048;
            const uint32_t o = grp * (4 * kRow) < kbytes ? soff + (uint32_t)grp * 32 : kOutOfRange;
            dma16(rs, at, o);
            dma16(rs, at + 1024, o + 32 * (uint32_t)spitch);
        };

        // Fragments: [set][step][row group], scales [set][row group].
        const int rowa = wm * 64 + li, rowb = wn * 64 + li;
        const uint32_t swz = (uint32_t)((4 * h) ^ ((li >> 1) & 7)) << 4;
        const uint32_t pa = (uint32_t)rowa * kRow + swz, pb = (uint32_t)rowb * kRow + swz + kOperand;
        const uint32_t qa = (uint32_t)(kScalesAt + rowa * 32 + 4 * h) ^ ((rowa >> 3) & 1) * 16u;
        const uint32_t qb = (uint32_t)(kScalesAt + kScaleBuf + rowb * 32 + 4 * h) ^ ((rowb >> 3) & 1) * 16u;
        int4v fa[2][4][2], fb[2][4][2];
        int sa[2][2], sb[2][2];
        // piece n of step J: B's two, then A's
        const auto read = [&](uint32_t slot, auto setc, auto jc, auto nc) {
            constexpr int set = decltype(setc)::value, J = decltype(jc)::value, n = decltype(nc)::value;
            if constexpr (n < 2) fb[set][J][n] = *(const int4v*)(lds + ((pb ^ (uint32_t)(J << 4)) + slot) + n * (32 * kRow));
            else fa[set][J][n - 2] = *(const int4v*)(lds + ((pa ^ (uint32_t)(J << 4)) + slot) + (n - 2) * (32 * kRow));
        };
        // scale piece n of stage s; 0 (2^-127, of zero codes) past K, where the buffer holds anything
        const auto read_scale = [&](int s, auto setc, auto nc) {
            constexpr int set = decltype(setc)::value, n = decltype(nc)::value;
            const uint32_t at = (uint32_t)((s >> 2) & 1) * 2 * kScaleBuf + (uint32_t)(s & 1) * 8;
            const int x = *(const int*)(lds + (((n < 2 ? qb : qa) ^ (uint32_t)((s >> 1) & 1) * 16) + at) + (n & 1) * (32 * 32));
            const int y = h * 64 < kbytes - s * kRow ? x : 0;
            if constexpr (n < 2) sb[set][n] = y;
            else sa[set][n - 2] = y;
        };

        load_scales(0);
        enter_stage(0);
        static_for<0, 8>([&](auto n) { load_codes(0, n); });
        enter_stage(1);
        static_for<0, 8>([&](auto n) { load_codes(kSlot, n); });
        wait_and_barrier<8>();
        static_for<0, 4>([&](auto n) {
            read_scale(0, Int<0>{}, n);
            static_for<0, 4>([&](auto j) { read(0, Int<0>{}, j, n); });
        });
        if constexpr (SLOTS == 2) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        enter_stage(2);
        static_for<0, 8>([&](auto n) { load_codes(2 * kSlot % (SLOTS * kSlot), n); });

        // Stage s (P = s mod 2), whose fragments are in set P; what is conditional stands before its
        // matrix instructions, which the compiler would move down past a branch.  Two slots: the
        // loads, of stage s + 3, go where the next stage's codes were, behind a second barrier, and
        // have a whole stage of two workgroups to arrive.  Four: they go where the last stage's were, and
        // nothing is waited for in between.
        const auto stage = [&](int s, auto pc) {
            constexpr int P = decltype(pc)::value;
            constexpr Int<1 - P> next;
            // stage s + 1 is there
            if constexpr (SLOTS == 2) wait_and_barrier<8>();
            else asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if constexpr (P == 0)
                if ((s & 3) == 0) load_scales(s / 4 + 1);
            enter_stage(s + 3);
            uint32_t to = (uint32_t)((s + 3) & (SLOTS - 1)) * kSlot, there = (uint32_t)((s + 1) & (SLOTS - 1)) * kSlot;
            asm volatile("" : "+s"(to), "+s"(there));
            static_for<0, 16>([&](auto mc) {
                constexpr int m = decltype(mc)::value, J = m / 4, i = m / 2 % 2, j = m % 2;
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    mx_frag(fb[P][J][j]), mx_frag(fa[P][J][i]), acc[i][j], kE2M1, kE2M1, J, sb[P][j], J, sa[P][i]);
                // 20 reads in the first ten
                if constexpr (m < 8) {
                    read(there, next, Int<m / 2>{}, Int<m % 2 * 2>{});
                    read(there, next, Int<m / 2>{}, Int<m % 2 * 2 + 1>{});
                } else if constexpr (m < 10) {
                    read_scale(s + 1, next, Int<(m - 8) * 2>{});
                    read_scale(s + 1, next, Int<(m - 8) * 2 + 1>{});
                }
                if constexpr (SLOTS == 2) {
                    if constexpr (m == 12) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    if constexpr (m >= 12) {
                        load_codes(to, Int<(m - 12) * 2>{});
                        load_codes(to, Int<(m - 12) * 2 + 1>{});
                    }
                } else {
                    if constexpr (m % 2 == 1) load_codes(to, Int<m / 2>{});
                }
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        int s = 0;
#pragma unroll 1
        for (; s + 2 <= nst; s += 2) {
            stage(s, Int<0>{});
            stage(s + 1, Int<1>{});
        }
        if (s < nst) stage(s, Int<0>{});
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may write LDS after the wave's end
    }

    // C.  Register r of lane l is column 8 (r / 4) + 4 (l / 32) + r % 4, row l % 32 of its 32 x 32: a
    // wave puts 32 rows of its part into LDS (its own piece, behind the barrier that ends the
    // stages' use of it) and stores them from there, 16 bytes a lane, a row's 64 columns contiguous.
    asm volatile("s_barrier" ::: "memory");
    constexpr int kRowBytes = 64 * (int)sizeof(T) + 16, kPer = 16 / (int)sizeof(T), kLanes = 64 / kPer;
    constexpr int kRowsAtOnce = 64 / kLanes;
    static_assert(4 * 32 * kRowBytes <= tile_lds(2), "C's rows fit");
    uint8_t* piece = lds + wid * (32 * kRowBytes);
    const int64_t col = n0 + wn * 64 + (lane % kLanes) * kPer;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                put_c4((T*)(piece + li * kRowBytes) + j * 32 + 2 * r + 4 * h, acc[i][j][r], acc[i][j][r + 1],
                       acc[i][j][r + 2], acc[i][j][r + 3]);
        const int64_t row0 = m0 + wm * 64 + i * 32 + lane / kLanes;
#pragma unroll
        for (int k = 0; k < 32 / kRowsAtOnce; ++k) {
            const int4v v = *(const int4v*)(piece + (k * kRowsAtOnce + lane / kLanes) * kRowBytes + (lane % kLanes) * 16);
            const int64_t r = row0 + k * kRowsAtOnce;
            if (r < m1) store_c16<STREAM>(c + r * g.ldc + col, v, g.N - col);
        }
    }
}

template <typename T, int MODE, bool STREAM, int SLOTS>
static int launch_slots(const MxGArgs& g, int64_t tiles, hipStream_t st) {
    const int64_t tn = (g.N + kSide - 1) / kSide, tm = (g.M + kSide - 1) / kSide;
    const auto kernel = k_mx_tile128<T, MODE, STREAM, SLOTS>;
    static std::atomic<uint64_t> ready{0};
    if (int rc = mx_allow_lds((const void*)kernel, tile_lds(SLOTS), ready)) return rc;
    kernel<<<dim3((unsigned)tiles), 256, tile_lds(SLOTS), st>>>(g, (unsigned)tn, (unsigned)tm);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename T, int MODE, bool STREAM>
static int launch(const MxGArgs& g, hipStream_t st) {
    const int64_t tn = (g.N + kSide - 1) / kSide, tm = (g.M + kSide - 1) / kSide;
    int64_t tiles = tm * tn;
    // every group, and the rows in none, may end in a partial tile
    if (MODE == MxRows) tiles = (g.M / kSide + (g.n_groups < g.M ? g.n_groups : g.M) + 1) * tn;
    if (MODE == MxK) tiles *= g.n_groups;
    if (!mx_grid_fits(tiles, 256)) return NVFP4_ERR_SHAPE;
    const int units = mx_compute_units();
    if (!units) return NVFP4_ERR_HIP;
    // (float32 streams from 128 MB on, which is thousands of tiles)
    if constexpr (sizeof(T) == 2 || !STREAM)
        if (tiles <= units) return launch_slots<T, MODE, STREAM, 4>(g, tiles, st);
    return launch_slots<T, MODE, STREAM, 2>(g, tiles, st);
}

template <typename T, bool STREAM>
static int launch_mode(const MxGArgs& g, int mode, hipStream_t st) {
    return mode == MxDense ? launch<T, MxDense, STREAM>(g, st)
           : mode == MxRows ? launch<T, MxRows, STREAM>(g, st) : launch<T, MxK, STREAM>(g, st);
}

int mx_tile128(const MxGArgs& g, int mode, int c_dtype, bool stream, hipStream_t st) {
    if (c_dtype == NVFP4_BF16) return launch_mode<uint16_t, true>(g, mode, st);
    return stream ? launch_mode<float, true>(g, mode, st) : launch_mode<float, false>(g, mode, st);
}

}  // namespace nvfp4
