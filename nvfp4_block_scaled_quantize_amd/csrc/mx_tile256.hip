// mx_tile256.hip -- the large-tile kernel of the MXFP4 products: 256 x 256 tiles of C, one
// workgroup of four waves a compute unit, each going through its share of the tiles.
//
// Wave (wm, wn) computes a 128 x 128 quarter as 4 x 4 accumulators of 32 x 32.  K advances in
// stages of 256 elements: 128 code bytes a row, one cache line.  Direct global -> LDS loads
// bring a stage as 8 rows x 128 bytes each; from the L2 a compute unit takes in 57 bytes a
// clock that way, but only 30 as 16 rows x 64 bytes.  A row's scale bytes come 32 at a time, for
// four stages.  LDS: two stages of codes (128 KiB) and two buffers of scales (32 KiB).
//
// LDS layout.  Row r's eight 16-byte chunks lie at slots q ^ (r / 2 mod 8): 16 consecutive rows'
// reads of one chunk touch every bank once.  The loads realise that order by which chunk each
// lane fetches.  Rows past the operand, and chunks past its K (K may end in half a stage),
// read as zeros by the loads' range check.
//
// A stage is four steps of 16 matrix instructions: step j multiplies chunk 4h + j of every row
// (h: the lane's half of the wave), whose scale is byte j of the four that the lane holds.
// Fragments are read up to two steps ahead, so that before the end of step 1 all of the stage
// is in registers and a barrier frees its LDS for the stage after next, whose 16 loads (a
// wave's) follow through the stage's end; a second barrier, after step 2, stands behind the wait
// for the next stage, whose first fragments step 3 reads.
//
// One wave a SIMD issues an instruction every four clocks or more, and a matrix instruction
// lasts 32: what stands between two of them has to be short.  So a load's address takes one
// addition: its rows are in eight registers, the K position and the LDS address of four loads in
// scalars, the instruction's offset (which counts for both addresses) tells the four apart, and
// what depends on the tile or on K's end is worked out once a stage.
//
// From tile to tile.  The loads run on into the next tile's first two stages while the last two
// of this one multiply, so that nothing is waited for between tiles but C's way out: through
// the scale buffer that is free then, 32 rows x 128 bytes a wave at a time, a line a row.  The
// stores drain while the next tile multiplies, but not for nothing: all compute units come to the
// end of their tiles together, and of 8192 x 8192 at K 1024, 2048, 4096 and 8192 (58, 84, 135, 238
// us) 33 us do not depend on K, 8 a tile (C alone at the rate of plain writes: 19 us).
//
// Measured, random operands: 8192 x 8192 x 4096 bf16 132 us, 4.2 PFLOP/s (one workgroup a tile with
// stages of 128 elements: 154 us); 8192 x 9216 x 6144 211 us, 4.4 PFLOP/s; 16384 x 4096 x 2048
// over 29 groups 95 us; 15 gradients of 1536 x 2048 over 8192 rows 43 us (189 MB of C: 27 us at
// the rate of plain writes).  Of 8192^3's cycles the matrix units are busy in 0.63, at 1.77 GHz
// with random operands and at 2.19 with zeros: the schedule sets the cycles, power the clock.
// Matrix instructions alone, on all compute units with operands in registers, run at 6.5 PFLOP/s
// (1.6 GHz) on random ones, at 9.3 on zeros.
#include "mx_tile.h"

namespace nvfp4 {

constexpr int kTile = 256;                           // tile side
constexpr int kOperand = kTile * kRow, kSlot = 2 * kOperand;
constexpr int kScaleBuf = kTile * 32;                // one operand, four stages
constexpr int kScalesAt = 2 * kSlot;                 // LDS offset of the scale buffers
constexpr int kTileLds = kScalesAt + 4 * kScaleBuf;
static_assert(kTileLds <= kMxMaxLds, "LDS budget");
// Waits for all but the ten (or, if `more`, the 42) newest operations.
__device__ __forceinline__ void wait_10_or_42_and_barrier(bool more) {
    asm volatile("s_cmp_lg_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(10)\n1:\ts_waitcnt vmcnt(42)\n\ts_barrier"
                 ::"s"(__builtin_amdgcn_readfirstlane((int)more)) : "memory", "scc");
}

// A tile: its descriptors, its extent of K in code bytes and stages (two at least, the second
// all zeros if need be, so that the loads are never more than one tile ahead), its part of C.
struct Tile256 {
    int4v rac, ras, rbc, rbs;
    int kbytes, nst;
    int rows, cols;
    int64_t at;         // element offset of its first element in C
};

template <typename T, int MODE, bool STREAM>
__global__ __launch_bounds__(256, 1) void k_mx_tile256(MxGArgs g, unsigned tiles_n, unsigned tiles_m) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wid >> 1, wn = wid & 1, li = lane & 31, h = lane >> 5;
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    T* const c = (T*)g.c;

    // ---- tiles
    MxSpan span = {};
    if constexpr (MODE != MxDense)
        if (g.n_groups <= 64)
            span = mx_span(g.offsets, g.n_groups, MODE == MxRows ? (int)g.M : (int)g.k_rows,
                           MODE == MxRows ? kTile : kMxPad, 0, 0);
    const auto locate = [&](unsigned v, Tile256& o) -> bool {
        unsigned tm, tn;
        int64_t m0, m1 = g.M, k0 = 0, c0 = 0;
        const uint8_t *bc = g.bc, *bs = g.bs;
        o.kbytes = (int)(g.kp / 2);
        if constexpr (MODE == MxRows) {
            MxUnit u;
            if (!(g.n_groups <= 64 ? mx_span_tile(span, g.n_groups, (int)g.M, kTile, v, tiles_n, tm, tn, u)
                                   : mx_find_tile(g.offsets, g.n_groups, (int)g.M, kTile, v, tiles_n, tm, tn, u)))
                return false;
            m0 = u.row0, m1 = u.row0 + u.rows;
            if (u.group == g.n_groups) o.kbytes = 0;
            else bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
        } else if constexpr (MODE == MxK) {
            if (v >= tiles_m * g.n_groups * tiles_n) return false;
            mx_tile_of(v, tiles_m * g.n_groups, tiles_n, tm, tn);
            MxUnit u;
            if (g.n_groups <= 64) mx_span_group(span, (int)(tm / tiles_m), u);
            else mx_group(g.offsets, g.n_groups, (int)g.k_rows, kMxPad, (int)(tm / tiles_m), u);
            k0 = u.first * kMxPad, o.kbytes = (int)(mx_blocks(u.rows) * (kMxBlock / 2));
            c0 = (int64_t)u.group * g.M * g.ldc;
            m0 = (int64_t)(tm % tiles_m) * kTile;
        } else {
            if (v >= tiles_m * tiles_n) return false;
            mx_tile_of(v, tiles_m, tiles_n, tm, tn);
            m0 = (int64_t)tm * kTile;
        }
        const int64_t n0 = (int64_t)tn * kTile;
        o.rows = (int)(m1 - m0 < kTile ? m1 - m0 : kTile);
        o.cols = (int)(g.N - n0 < kTile ? g.N - n0 : kTile);
        o.at = c0 + m0 * g.ldc + n0;
        o.nst = o.kbytes > kRow ? (o.kbytes + kRow - 1) / kRow : 2;
        // (codes: kBias bytes early, see load_codes)
        o.rac = make_rsrc(g.ac + m0 * pitch + k0 / 2 - kBias, (uint32_t)(o.rows * pitch - k0 / 2 + kBias));
        o.ras = make_rsrc(g.as + m0 * spitch + k0 / 32, (uint32_t)(o.rows * spitch - k0 / 32));
        o.rbc = make_rsrc(bc + n0 * pitch + k0 / 2 - kBias, (uint32_t)(o.cols * pitch - k0 / 2 + kBias));
        o.rbs = make_rsrc(bs + n0 * spitch + k0 / 32, (uint32_t)(o.cols * spitch - k0 / 32));
        return true;
    };
    // The next tile from v on that has anything to multiply (those without are set to 0 here);
    // false, with no bytes of K, if there is none.
    unsigned v = blockIdx.x;
    const auto advance = [&](Tile256& o) -> bool {
        for (;; v += gridDim.x) {
            if (!locate(v, o)) {
                o.kbytes = 0, o.nst = 2;
                return false;
            }
            if (o.kbytes > 0) {
                v += gridDim.x;
                return true;
            }
            for (int r = wid; r < o.rows; r += 4)
                for (int k = lane; k < o.cols; k += 64) store_c(c + o.at + r * g.ldc + k, 0.0f);
        }
    };

    // ---- loads
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    // Code load n of a stage: rows 8 (8 wid + n) .. + 7 of A (n < 8), then the same of B.  The byte of
    // the operand is row[n mod 8] (a register), plus the stage's K position (a scalar), and plus
    // the instruction's offset 1024 (n mod 4), which moves the LDS address on from M0 as well and
    // is taken off again by the scalar and the descriptor's early start (kBias), so that nothing
    // is negative.  The scalar stays below the descriptor's size, as the range check wants it.
    // Chunks past K: 2^31 more, out of range, zeros.
    const int chunk = ((lane & 7) ^ (lane >> 4)) << 4;              // the lane's, for even n
    uint32_t row[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) row[i] = (uint32_t)(wid * 64 + i * 8 + (lane >> 3)) * (uint32_t)pitch + (chunk ^ (i & 1) * 64);
    int4v pra, prb;             // the stage that is being loaded: its tile's descriptors,
    int pk, ps;                 // its tile's bytes of K and its number there,
    uint32_t past[2], kat;      // what its lanes add for chunks past K (n even, odd), its K position
    const auto enter_stage = [&] {
        const int left = pk - ps * kRow;
        past[0] = chunk < left ? 0u : kOutOfRange;
        past[1] = (chunk ^ 64) < left ? 0u : kOutOfRange;
        kat = left > 0 ? (uint32_t)(ps * kRow) : 0u;
    };
    const auto load_codes = [&](uint32_t slot, auto nc) {
        constexpr int n = decltype(nc)::value, i = n % 8, quarter = n % 4;
        if constexpr (quarter == 0)
            set_m0(lds0 + slot + (n < 8 ? 0 : kOperand) + (uint32_t)wid * 8192 + (i & 4) * 1024);
        dma16_at<quarter * 1024>(n < 8 ? pra : prb, row[i] + past[i & 1], kat + (kBias - quarter * 1024));
    };
    // The scales of four stages: a load covers 32 rows x 32 bytes; row r's 16-byte halves are
    // exchanged where r / 8 is odd, for the banks' sake.
    const uint32_t srow = (uint32_t)(wid * 32 + (lane >> 1));
    const uint32_t soff = srow * (uint32_t)spitch + (((uint32_t)lane ^ (srow >> 3)) & 1) * 16;
    const auto load_scales = [&](const int4v& ra, const int4v& rb, int kbytes, int grp, uint32_t buf) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint32_t row = (uint32_t)part * 128, at = lds0 + kScalesAt + buf + (row + (uint32_t)wid * 32) * 32;
            const uint32_t o = grp * (4 * kRow) < kbytes ? soff + row * (uint32_t)spitch + (uint32_t)grp * 32 : kOutOfRange;
            dma16(ra, at, o);
            dma16(rb, at + kScaleBuf, o);
        }
    };

    // ---- fragments: this lane's rows of A and B, 32 apart from one of its four to the next.  The
    // LDS offsets of stages are kept opaque: the compiler would otherwise hold every address of
    // both slots in registers that the fragments need.
    const int rowa = wm * 128 + li, rowb = wn * 128 + li;
    const uint32_t swz = (uint32_t)((4 * h) ^ ((li >> 1) & 7)) << 4;
    const uint32_t pa = (uint32_t)rowa * kRow + swz, pb = (uint32_t)rowb * kRow + swz + kOperand;
    const uint32_t qa = (uint32_t)(kScalesAt + rowa * 32 + 4 * h) ^ ((rowa >> 3) & 1) * 16u;
    const uint32_t qb = (uint32_t)(kScalesAt + kScaleBuf + rowb * 32 + 4 * h) ^ ((rowb >> 3) & 1) * 16u;
    int4v fa[4][4], fb[4][4];           // [step][row group]
    int sa[4], sb[4], na[4], nb[4];     // scales of this stage and of the next
    const auto read = [&](uint32_t slot, auto jc, auto nc) {
        constexpr int J = decltype(jc)::value, n = decltype(nc)::value;
        if constexpr (n < 4) fb[J][n] = *(const int4v*)(lds + ((pb ^ (uint32_t)(J << 4)) + slot) + n * (32 * kRow));
        else if constexpr (n < 8)
            fa[J][n - 4] = *(const int4v*)(lds + ((pa ^ (uint32_t)(J << 4)) + slot) + (n - 4) * (32 * kRow));
    };
    // four scale bytes: at + 8 (stage mod 2) in a buffer, half: 16 (stage / 2 mod 2)
    const auto read_scale = [&](uint32_t at, uint32_t half, auto nc) {
        constexpr int n = decltype(nc)::value;
        const int x = *(const int*)(lds + (((n < 4 ? qb : qa) ^ half) + at) + (n & 3) * (32 * 32));
        if constexpr (n < 4) nb[n] = x;
        else na[n - 4] = x;
    };

    Tile256 cur, nxt;
    if (!advance(cur)) return;
    uint32_t slot = 0, buf = 0;         // LDS offsets of the current stage's codes and scales
    constexpr uint32_t kSlots = kSlot, kBufs = 2 * kScaleBuf;     // the other one: exclusive or
    nxt = cur;
    load_scales(cur.ras, cur.rbs, cur.kbytes, 0, 0);
    pra = cur.rac, prb = cur.rbc, pk = cur.kbytes;
    ps = 0, enter_stage();
    static_for<0, 16>([&](auto n) { load_codes(0, n); });
    ps = 1, enter_stage();
    static_for<0, 16>([&](auto n) { load_codes(kSlot, n); });
    wait_and_barrier<16>();
    static_for<0, 8>([&](auto n) {
        read_scale(0, 0, n);
        read(0, Int<0>{}, n);
    });
    bool flying = false;                // the last tile's stores may still be in flight, 32 at least

    for (;;) {
        const bool more = advance(nxt);
        float16v acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        const auto mma = [&](auto jc, auto mc) {
            constexpr int J = decltype(jc)::value, i = decltype(mc)::value / 4, j = decltype(mc)::value % 4;
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                mx_frag(fb[J][j]), mx_frag(fa[J][i]), acc[i][j], kE2M1, kE2M1, J, sb[j], J, sa[i]);
        };
#pragma unroll 1
        for (int s = 0; s < cur.nst; ++s) {
            // What is conditional stands here, before the first matrix instruction: the compiler moves
            // them down past a branch, away from what they are to run beside.
            // 0 (2^-127, of zero codes) for scales past K, where the buffer holds anything
#pragma unroll
            for (int i = 0; i < 4; ++i) sa[i] = na[i], sb[i] = nb[i];
            if (const int left = cur.kbytes - s * kRow; left < kRow) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sa[i] = h * 64 < left ? sa[i] : 0;
                    sb[i] = h * 64 < left ? sb[i] : 0;
                }
            }
            // the loads go on to stage s + 2, of this tile or the next
            if (s + 2 == cur.nst) pra = nxt.rac, prb = nxt.rbc, pk = nxt.kbytes, ps = 0;
            else ++ps;
            enter_stage();
            // the next four stages' scales
            if ((s & 3) == 0) {
                if (s + 4 < cur.nst) load_scales(cur.ras, cur.rbs, cur.kbytes, s / 4 + 1, buf ^ kBufs);
                else load_scales(nxt.ras, nxt.rbs, nxt.kbytes, 0, buf ^ kBufs);
            }
            uint32_t here = slot, there = slot ^ kSlots;
            asm volatile("" : "+s"(here), "+s"(there));
            // the next stage's scales: another buffer every four stages and with the next tile
            const int s1 = s + 1 < cur.nst ? s + 1 : 0;
            if ((s1 & 3) == 0) buf ^= kBufs;
            const uint32_t sat = buf + (uint32_t)(s1 & 1) * 8, shalf = (uint32_t)((s1 >> 1) & 1) * 16;

            static_for<0, 16>([&](auto m) {
                mma(Int<0>{}, m);
                if constexpr (m < 8) read(here, Int<1>{}, m);
                else read(here, Int<2>{}, Int<m - 8>{});
                __builtin_amdgcn_sched_barrier(0);
            });
            static_for<0, 16>([&](auto m) {
                mma(Int<1>{}, m);
                read(here, Int<3>{}, m);
                if constexpr (m == 12) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // its LDS is free
                if constexpr (m == 13) load_codes(here, Int<0>{});
                if constexpr (m == 15) load_codes(here, Int<1>{});
                __builtin_amdgcn_sched_barrier(0);
            });
            static_for<0, 16>([&](auto m) {
                mma(Int<2>{}, m);
                if constexpr (m % 2 == 1) load_codes(here, Int<2 + m / 2>{});
                __builtin_amdgcn_sched_barrier(0);
            });
            // Stage s + 1 is there (and the scales): in flight are the ten loads after it and, in a
            // tile's first stage, whose stage 1 was asked for before them, 32 stores of the last tile's.
            wait_10_or_42_and_barrier(s == 0 && flying);
            static_for<0, 16>([&](auto m) {
                mma(Int<3>{}, m);
                read(there, Int<0>{}, m);
                if constexpr (m % 2 == 1) read_scale(sat, shalf, Int<m / 2>{});
                if constexpr (m % 3 == 0) load_codes(here, Int<10 + m / 3>{});
                __builtin_amdgcn_sched_barrier(0);
            });
            slot ^= kSlots;
        }

        // ---- C.  Register r of lane l is column 8 (r / 4) + 4 (l / 32) + r % 4, row l % 32 of its 32 x
        // 32.  A wave's piece of the free scale buffer takes 32 rows x 128 bytes, chunk q of row r
        // at q ^ (r mod 8), and is stored from there, a line a row.
        uint8_t* piece = lds + kScalesAt + (buf ^ kBufs) + wid * 4096;
        constexpr int kN = 128 / (int)sizeof(T), kPer = 16 / (int)sizeof(T);     // columns of a piece, of a lane
        const bool whole = cur.rows == kTile && cur.cols == kTile;
        int rr = lane >> 3, cc = wn * 128 + (lane & 7) * kPer, lr = li;     // opaque, as above: addresses
        asm volatile("" : "+v"(rr), "+v"(cc), "+v"(lr));                    // are made where they are used
        // the accumulators as they stand: the compiler would otherwise take them apart and shuffle
        // them on their way out of the loop
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));
        T* const first = c + cur.at + (int64_t)(wm * 128 + rr) * g.ldc + cc;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 128 / kN; ++q) {
#pragma unroll
                for (int j = 0; j < kN / 32; ++j)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const int byte = (j * 32 + 2 * r + 4 * h) * (int)sizeof(T);
                        const float16v& x = acc[i][q * (kN / 32) + j];
                        put_c4((T*)(piece + lr * 128 + (((byte >> 4) ^ (lr & 7)) << 4) + (byte & 15)), x[r], x[r + 1],
                               x[r + 2], x[r + 3]);
                    }
                // row k * 8 + rr of the piece (rr < 8)
                const uint8_t* from = piece + rr * 128 + (((lane & 7) ^ rr) << 4);
                T* p = first + ((int64_t)(i * 32) * g.ldc + q * kN);
                if (whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        using Vec = typename Oct<T>::Vec;
                        const int4v x = *(const int4v*)(from + k * 1024);
                        if constexpr (STREAM) __builtin_nontemporal_store((Vec)x, (Vec*)p);
                        else *(Vec*)p = x;
                        p += 8 * g.ldc;
                    }
                } else {
                    int row = wm * 128 + i * 32 + rr, left = cur.cols - cc - q * kN;
                    asm volatile("" : "+v"(row), "+v"(left));
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int4v x = *(const int4v*)(from + k * 1024);
                        if (row < cur.rows) store_c16<STREAM>(p, x, left);
                        row += 8, p += 8 * g.ldc;
                    }
                }
                __builtin_amdgcn_sched_barrier(0);      // not all accumulators into registers at once
            }
        if (!more) break;
        flying = whole;
        cur = nxt;
        // every wave is done with its piece of the scale buffer, which the next stage fills
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no load may write LDS after the wave's end
}

template <typename T, int MODE, bool STREAM>
static int launch(const MxGArgs& g, hipStream_t st) {
    const int64_t tn = (g.N + kTile - 1) / kTile, tm = (g.M + kTile - 1) / kTile;
    int64_t tiles = tm * tn;
    // every group, and the rows in none, may end in a partial tile
    if (MODE == MxRows) tiles = (g.M / kTile + (g.n_groups < g.M ? g.n_groups : g.M) + 1) * tn;
    if (MODE == MxK) tiles *= g.n_groups;
    if (tiles > 0x7FFFFFFF - 0x10000) return NVFP4_ERR_SHAPE;      // tile numbers are 32 bits
    const auto kernel = k_mx_tile256<T, MODE, STREAM>;
    static std::atomic<uint64_t> ready{0};
    if (int rc = mx_allow_lds((const void*)kernel, kTileLds, ready)) return rc;
    const int units = mx_compute_units();
    if (!units) return NVFP4_ERR_HIP;
    kernel<<<dim3((unsigned)(tiles < units ? tiles : units)), 256, kTileLds, st>>>(g, (unsigned)tn, (unsigned)tm);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename T, bool STREAM>
static int launch_mode(const MxGArgs& g, int mode, hipStream_t st) {
    return mode == MxDense ? launch<T, MxDense, STREAM>(g, st)
           : mode == MxRows ? launch<T, MxRows, STREAM>(g, st) : launch<T, MxK, STREAM>(g, st);
}

int mx_tile256(const MxGArgs& g, int mode, int c_dtype, bool stream, hipStream_t st) {
    if (c_dtype == NVFP4_BF16) return launch_mode<uint16_t, true>(g, mode, st);
    return stream ? launch_mode<float, true>(g, mode, st) : launch_mode<float, false>(g, mode, st);
}

}  // namespace nvfp4
