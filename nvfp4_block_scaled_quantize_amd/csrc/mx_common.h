// mx_common.h -- what the MXFP4 kernels share: the block scale, groups of rows, host checks.
#pragma once
#include "mxfp4.h"
#include "device_common.h"

#include <atomic>

namespace nvfp4 {

constexpr uint32_t kTagMxSR = 0x4D585352u;
constexpr int kMxBlock = 32;    // elements per E8M0 scale
constexpr int kMxPad = 128;     // a copy's K extent is a multiple of this
constexpr int64_t kMxMaxK = (int64_t)1 << 23;   // 256 rows of codes stay within 2^30 bytes

typedef int int8v __attribute__((ext_vector_type(8)));

// No extent is larger: a quarter of a padded row (the decode's pieces) and what a workgroup adds to it
// are counted in 32 bits.
constexpr int64_t kMxMaxExtent = ((int64_t)1 << 34) - (1 << 13);
constexpr int64_t kMxMaxC = (int64_t)1 << 40;   // elements of a product's C, so that counts of them stay in 64 bits

inline int64_t mx_pad(int64_t k) { return (k + kMxPad - 1) / kMxPad * kMxPad; }

// E8M0 code of a block from the binary32 bits of its largest magnitude (magnitudes order as
// their bits do, infinities and NaN above every finite one).  With e the exponent field:
// FLOOR is 2^(e - 127 - 2), code e - 2; CEIL is one more when amax > 1.5 * 2^(e - 127), i.e.
// amax > 6 * 2^(e - 127 - 2).  Subnormal maxima have e = 0 and take code 0 (2^-127), which
// both rules' lower bound gives: amax < 2^-126 <= 6 * 2^-127.  `above`: the largest fraction
// field that does not round up, kMxCeilAbove or kMxFloorAbove.
constexpr uint32_t kMxCeilAbove = 0x400000u, kMxFloorAbove = 0x7FFFFFu;
inline uint32_t mx_above(int rule) { return rule == MXFP4_SCALE_CEIL ? kMxCeilAbove : kMxFloorAbove; }
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

// ---------------------------------------------------------------- elements
// Eight consecutive elements of a block.
typedef int int4_by2 __attribute__((ext_vector_type(4), aligned(2)));
typedef int int4_by4 __attribute__((ext_vector_type(4), aligned(4)));
template <typename T> struct Oct {};
template <> struct Oct<uint16_t> { uint32_t w[4]; using Vec = int4_by2; };
template <> struct Oct<float> { float v[8]; using Vec = int4_by4; };

// Loads of any alignment: rows may start at any element, and the hardware splits what
// straddles.  left: elements up to the row's end (may be <= 0); the rest are zeros.  STREAM:
// past the caches.
template <typename T, bool STREAM = false>
__device__ __forceinline__ Oct<T> load_oct(const T* p, int64_t left) {
    using Vec = typename Oct<T>::Vec;
    Oct<T> o;
    if (left >= 8) {
        int4v v[sizeof(o) / 16];
#pragma unroll
        for (unsigned i = 0; i < sizeof(o) / 16; ++i)
            v[i] = STREAM ? __builtin_nontemporal_load((const Vec*)p + i) : ((const Vec*)p)[i];
        __builtin_memcpy(&o, v, sizeof(o));
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < left ? p[i] : (T)0;
        __builtin_memcpy(&o, e, sizeof(o));
    }
    return o;
}

typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// Magnitude bits of two packed bfloat16 each: they order as the values do.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2v, a),
                                                                  __builtin_bit_cast(ushort2v, b)));
}

// binary32 bits of the largest magnitude
__device__ __forceinline__ uint32_t max_bits(const Oct<uint16_t>& o) {
    uint32_t m = o.w[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max_bf16x2(m, o.w[i] & 0x7FFF7FFFu);
    return max(m << 16, m & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t max_bits(const Oct<float>& o) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(o.v[i]) & 0x7FFFFFFFu);
    return m;
}

__device__ __forceinline__ float value(const Oct<uint16_t>& o, int i) {
    return __uint_as_float((i & 1) ? o.w[i >> 1] & 0xFFFF0000u : o.w[i >> 1] << 16);
}
__device__ __forceinline__ float value(const Oct<float>& o, int i) { return o.v[i]; }

// Nearest even: eight codes of o / cs (cs a power of two).
__device__ __forceinline__ uint32_t codes_rne(const Oct<uint16_t>& o, float cs) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, o.w[0]), cs, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, o.w[1]), cs, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, o.w[2]), cs, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2v, o.w[3]), cs, 3);
}
__device__ __forceinline__ uint32_t codes_rne(const Oct<float>& o, float cs) {
    uint32_t w = 0;
    w = cvt_fp4x2<0>(w, o.v[0], o.v[1], cs);
    w = cvt_fp4x2<1>(w, o.v[2], o.v[3], cs);
    w = cvt_fp4x2<2>(w, o.v[4], o.v[5], cs);
    return cvt_fp4x2<3>(w, o.v[6], o.v[7], cs);
}

// ---------------------------------------------------------------- groups of rows
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

// Largest over the four lanes of a quad, which hold one block.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)dpp<kXor1>(0, (int)m));
    return max(m, (uint32_t)dpp<kXor2>(0, (int)m));
}

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
// the last unit (grids are sized for the worst offsets).  x: the span of all (at most 64) groups.
__device__ __forceinline__ bool mx_span_tile(const MxSpan& x, int n_groups, int rows, int unit, unsigned bid,
                                             unsigned tiles_n, unsigned& tm, unsigned& tn, MxUnit& out) {
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

// mx_group from the span of all (at most 64) groups.
__device__ __forceinline__ void mx_span_group(const MxSpan& x, int g, MxUnit& out) {
    out.group = g;
    out.first = lane_value(x.p - x.n, g);
    out.group_row0 = out.row0 = lane_value(x.s, g);
    out.group_rows = out.rows = lane_value(x.e, g) - out.row0;
}

// mx_span_tile for any number of groups: with up to 64 the offsets are read and scanned once.
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
    return mx_span_tile(mx_span(offsets, n_groups, rows, unit, 0, 0), n_groups, rows, unit, bid, tiles_n, tm, tn, out);
}

// ---------------------------------------------------------------- products
// A product.  Groups: rows (A's and C's rows [offsets[g], offsets[g+1]) with B's matrix g) or
// ragged K (K positions of group g, C's matrix g).
enum { MxDense = 0, MxRows = 1, MxK = 2 };
struct MxGArgs {
    const uint8_t *ac, *as, *bc, *bs;
    int64_t M, N, kp;           // kp: K extent of both operands' rows (a multiple of 128)
    int64_t k_rows;             // MxK: rows that the groups divide
    void* c;
    int64_t ldc;
    const int32_t* offsets;
    int n_groups;
};

// A product for mx_few.hip: A packed (x null), or x to quantize rowwise.
struct MxFArgs {
    MxGArgs g;
    const void* x;
    int64_t ldx, K;
    uint32_t above;
};
// A packed, or quantized from x; dense or grouped.
int mx_few_packed(const MxFArgs& f, int c_dtype, hipStream_t st);
int mx_few_linear(const MxFArgs& f, int x_dtype, int c_dtype, hipStream_t st);
// Whether 16 rows of A fit into a workgroup's LDS, and whether a dense product of A packed belongs
// here: up to 16 rows, or no more than two workgroups (of 32 x 32) a compute unit.
bool mx_few_fits(int64_t M, int64_t kp);
bool mx_few_dense(int64_t M, int64_t N, int64_t kp);
// Elements of x that a workgroup of a dense product quantizes, times the workgroups a compute unit.
int64_t mx_few_quantized(int64_t M, int64_t N, int64_t kp);

constexpr int kMxMaxLds = 160 * 1024;
// Lets a kernel use `bytes` of LDS, once per device (a bit of `ready` each).
inline int mx_allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return NVFP4_ERR_HIP;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (dev < 64 && (ready.load(std::memory_order_relaxed) & bit)) return NVFP4_OK;
    if (hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return NVFP4_ERR_HIP;
    ready.fetch_or(bit, std::memory_order_relaxed);
    return NVFP4_OK;
}

// The 256 x 256 tiles (mx_tile256.hip).  mode: MxDense, MxRows, MxK; stream: float32 C past the
// caches.
int mx_tile256(const MxGArgs& g, int mode, int c_dtype, bool stream, hipStream_t st);
// The same with 128 x 128 tiles (mx_tile128.hip).
int mx_tile128(const MxGArgs& g, int mode, int c_dtype, bool stream, hipStream_t st);

// Compute units of the current device, rounded down to a multiple of the 8 XCDs; 0 on an error.
inline int mx_compute_units() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed))) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    n = n > 8 ? n / 8 * 8 : 8;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// A grid's threads are counted in 32 bits.  (Wide: products of extents.)
inline bool mx_grid_fits(__int128 blocks, int threads) { return blocks * threads < ((__int128)1 << 32); }

typedef float float4v __attribute__((ext_vector_type(4)));

// An operand fragment: the instruction's E2M1 form reads the first four of eight registers.
__device__ __forceinline__ int8v mx_frag(int4v v) {
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
constexpr int kE2M1 = 4;

__device__ __forceinline__ void store_c(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_c(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }
// Four consecutive elements of C into LDS.
__device__ __forceinline__ void put_c4(float* p, float a, float b, float c, float d) {
    *(float4v*)p = float4v{a, b, c, d};
}
__device__ __forceinline__ void put_c4(uint16_t* p, float a, float b, float c, float d) {
    typedef __bf16 bf16x4v __attribute__((ext_vector_type(4)));
    *(bf16x4v*)p = bf16x4v{(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d};
}
// 16 bytes of a row of C, of which `left` elements exist.  STREAM: past the caches.
template <bool STREAM, typename T>
__device__ __forceinline__ void store_c16(T* p, int4v v, int64_t left) {
    using Vec = typename Oct<T>::Vec;
    constexpr int n = 16 / (int)sizeof(T);
    if (left >= n) {
        if constexpr (STREAM) __builtin_nontemporal_store((Vec)v, (Vec*)p);
        else *(Vec*)p = v;
    } else {
        T e[n];
        __builtin_memcpy(e, &v, sizeof(e));
#pragma unroll
        for (int i = 0; i < n - 1; ++i)
            if (i < left) p[i] = e[i];
    }
}

// ---------------------------------------------------------------- host checks
inline bool mx_extent(int64_t n) { return n >= 0 && n <= kMxMaxExtent; }
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
