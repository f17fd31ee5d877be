// mx_common.h -- what the MXFP4 kernels share: the block scale, groups of rows, host checks.
#pragma once
#include "mxfp4.h"
#include "device_common.h"

namespace nvfp4 {

constexpr uint32_t kTagMxSR = 0x4D585352u;
constexpr int kMxBlock = 32;    // elements per E8M0 scale
constexpr int kMxPad = 128;     // a copy's K extent is a multiple of this
constexpr int64_t kMxMaxK = (int64_t)1 << 23;   // 256 rows of codes stay within 2^30 bytes

inline int64_t mx_pad(int64_t k) { return (k + kMxPad - 1) / kMxPad * kMxPad; }

// E8M0 code of a block from the binary32 bits of its largest magnitude (magnitudes order as
// their bits do, infinities and NaN above every finite one).  With e the exponent field:
// FLOOR is 2^(e - 127 - 2), code e - 2; CEIL is one more when amax > 1.5 * 2^(e - 127), i.e.
// amax > 6 * 2^(e - 127 - 2).  Subnormal maxima have e = 0 and take code 0 (2^-127), which
// both rules' lower bound gives: amax < 2^-126 <= 6 * 2^-127.  `above`: the largest fraction
// field that does not round up, kMxCeilAbove or kMxFloorAbove.
constexpr uint32_t kMxCeilAbove = 0x400000u, kMxFloorAbove = 0x7FFFFFu;
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits, uint32_t above) {
    uint32_t e = amax_bits >> 23;
    if (e == 255u) return 255u;
    e += (amax_bits & 0x7FFFFFu) > above ? 1u : 0u;
    return (e > 2u ? e : 2u) - 2u;
}

// 2^(code - 127) as binary32 for codes 0..254 (0 gives the subnormal 2^-127).
__device__ __forceinline__ float mx_scale_value(uint32_t code) {
    const uint32_t b = code << 23;
    return __uint_as_float(b > 0x400000u ? b : 0x400000u);
}

// A unit (`unit` consecutive rows, or fewer at a group's end) of the rows of a grouped matrix.
struct MxUnit {
    int group;        // n_groups for the rows past the last group
    int64_t row0;     // first row of the unit
    int64_t rows;     // rows in the unit (<= unit)
    int64_t first;    // units of the groups before this one
    int64_t group_row0, group_rows;
};

// Blocks of a group of `rows` rows in a grouped columnwise copy.
__device__ __forceinline__ int64_t mx_blocks(int64_t rows) {
    return (rows + kMxPad - 1) / kMxPad * (kMxPad / kMxBlock);
}

// DPP moves: quads, rows of 16 lanes, whole wave.  Lanes without a source (or masked rows)
// take `old`.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ int dpp(int old, int v) {
    return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128, kWaveShr1 = 0x138;

// Inclusive scan over the wave's 64 lanes of non-negative values: within rows of 16, then the
// last lane of rows 0 and 2 into rows 1 and 3, then lane 31 into the upper half.
template <typename Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, dpp<0x111>(0, v));
    v = op(v, dpp<0x112>(0, v));
    v = op(v, dpp<0x114>(0, v));
    v = op(v, dpp<0x118>(0, v));
    v = op(v, dpp<0x142, 0xA>(0, v));
    return op(v, dpp<0x143, 0xC>(0, v));
}

// The value of one lane, as a scalar (the descriptors of direct loads must be scalars).
__device__ __forceinline__ int lane_value(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// 64 consecutive groups, one per lane: rows [s, e), their units n and the inclusive count p of
// units.  Offsets are clamped to [0, rows] and made non-decreasing.
struct MxSpan {
    int s, e, n, p;
};
__device__ __forceinline__ MxSpan mx_span(const int32_t* offsets, int n_groups, int rows, int unit, int base,
                                          int end) {
    const int g = base + (threadIdx.x & 63);
    int e = g < n_groups ? offsets[g + 1] : 0;
    e = e < rows ? e : rows;
    e = e > end ? e : end;
    MxSpan x;
    x.e = wave_scan(e, [](int a, int b) { return a > b ? a : b; });
    x.s = dpp<kWaveShr1>(end, x.e);
    x.n = (x.e - x.s + unit - 1) / unit;
    x.p = wave_scan(x.n, [](int a, int b) { return a + b; });
    return x;
}

// Unit `u` of the groups' units in order (each group ceil(rows / unit) of them, then those of
// the rows in no group), which exists.  `u` is uniform over the wave; all 64 lanes call.
__device__ __forceinline__ void mx_find_unit(const int32_t* offsets, int n_groups, int rows, int unit, int64_t u,
                                             MxUnit& out) {
    int end = 0;          // end of the groups before `base`
    int64_t units = 0;    // their units
    for (int base = 0; base < n_groups; base += 64) {
        const MxSpan x = mx_span(offsets, n_groups, rows, unit, base, end);
        const uint64_t hit = __builtin_amdgcn_ballot_w64(units + x.p > u);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            const int gs = lane_value(x.s, at), ge = lane_value(x.e, at);
            out.group = base + at;
            out.first = units + lane_value(x.p - x.n, at);
            out.group_row0 = gs;
            out.group_rows = ge - gs;
            out.row0 = gs + (u - out.first) * unit;
            out.rows = ge - out.row0 < unit ? ge - out.row0 : unit;
            return;
        }
        end = lane_value(x.e, 63);
        units += lane_value(x.p, 63);
    }
    out.group = n_groups;
    out.first = units;
    out.group_row0 = end;
    out.group_rows = rows - end;
    out.row0 = end + (u - units) * unit;
    out.rows = rows - out.row0 < unit ? rows - out.row0 : unit;
}

// All units of the groups and of the rows in none.  All 64 lanes call.
__device__ __forceinline__ int64_t mx_units(const int32_t* offsets, int n_groups, int rows, int unit) {
    int end = 0;
    int64_t units = 0;
    for (int base = 0; base < n_groups; base += 64) {
        const MxSpan x = mx_span(offsets, n_groups, rows, unit, base, end);
        units += lane_value(x.p, 63);
        end = lane_value(x.e, 63);
    }
    return units + (rows - end + unit - 1) / unit;
}

// Group g's rows and the number of `unit`-row units before it.  All 64 lanes call.
__device__ __forceinline__ void mx_group(const int32_t* offsets, int n_groups, int rows, int unit, int g,
                                         MxUnit& out) {
    int end = 0;
    int64_t units = 0;
    for (int base = 0;; base += 64) {
        const MxSpan x = mx_span(offsets, n_groups, rows, unit, base, end);
        if (g < base + 64) {
            const int at = g - base;
            out.group = g;
            out.first = units + lane_value(x.p - x.n, at);
            out.group_row0 = out.row0 = lane_value(x.s, at);
            out.group_rows = out.rows = lane_value(x.e, at) - out.row0;
            return;
        }
        end = lane_value(x.e, 63);
        units += lane_value(x.p, 63);
    }
}

// Tile id -> (tm, tn) as in the NVFP4 product: workgroups go to the eight XCDs in turn, XCD x
// takes a contiguous range of ids, and ids walk down groups of 8 tile rows column by column,
// so that the tiles an XCD runs at once share operand rows (and output lines) in its L2.
__device__ __forceinline__ void mx_tile_of(unsigned bid, unsigned tiles_m, unsigned tiles_n, unsigned& tm,
                                           unsigned& tn) {
    const unsigned total = tiles_m * tiles_n, q = total / 8, r = total % 8, x = bid % 8;
    const unsigned id = x * q + (x < r ? x : r) + bid / 8;
    const unsigned group = id / (8 * tiles_n), first = group * 8;
    const unsigned rows = tiles_m - first < 8 ? tiles_m - first : 8, in = id - group * 8 * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

// The tile of workgroup `bid` when the rows are grouped: tiles_n columns of units.  False past
// the last unit (grids are sized for the worst offsets).  With up to 64 groups the offsets are
// read and scanned once.
__device__ __forceinline__ bool mx_find_tile(const int32_t* offsets, int n_groups, int rows, int unit,
                                             unsigned bid, unsigned tiles_n, unsigned& tm, unsigned& tn,
                                             MxUnit& out) {
    if (n_groups > 64) {
        const unsigned units = (unsigned)mx_units(offsets, n_groups, rows, unit);
        if (bid >= units * tiles_n) return false;
        mx_tile_of(bid, units, tiles_n, tm, tn);
        mx_find_unit(offsets, n_groups, rows, unit, tm, out);
        return true;
    }
    const MxSpan x = mx_span(offsets, n_groups, rows, unit, 0, 0);
    const int grouped = lane_value(x.p, 63), end = lane_value(x.e, 63);
    const unsigned units = (unsigned)(grouped + (rows - end + unit - 1) / unit);
    if (bid >= units * tiles_n) return false;
    mx_tile_of(bid, units, tiles_n, tm, tn);
    const bool in = tm < (unsigned)grouped;
    const int at = in ? (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(x.p > (int)tm)) : 0;
    const int gs = in ? lane_value(x.s, at) : end, ge = in ? lane_value(x.e, at) : rows;
    out.group = in ? at : n_groups;
    out.first = in ? lane_value(x.p - x.n, at) : grouped;
    out.group_row0 = gs;
    out.group_rows = ge - gs;
    out.row0 = gs + (tm - out.first) * unit;
    out.rows = ge - out.row0 < unit ? ge - out.row0 : unit;
    return true;
}

// ---------------------------------------------------------------- host checks
// `used`: the copy has elements, so its arrays must exist.
inline int mx_check_tensor(const mxfp4_tensor* t, bool used) {
    if (!t || (used && (!t->codes || !t->scales))) return NVFP4_ERR_NULL;
    if (((uintptr_t)t->codes & 15) || ((uintptr_t)t->scales & 3)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}
inline int mx_dtype_size(int dtype) {
    return dtype == NVFP4_F32 ? 4 : dtype == NVFP4_BF16 ? 2 : 0;
}
// Groups: an offsets array goes with n_groups >= 1, none with 0; row numbers are int32.
inline int mx_check_groups(const int32_t* offsets, int64_t n_groups, int64_t rows) {
    if (n_groups < 0 || n_groups > 65536 || (n_groups && rows > 0x7FFFFFFF - 65536))
        return NVFP4_ERR_SHAPE;
    if (n_groups && !offsets) return NVFP4_ERR_NULL;
    if (!n_groups && offsets) return NVFP4_ERR_MODE;
    if ((uintptr_t)offsets & 3) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

}  // namespace nvfp4
