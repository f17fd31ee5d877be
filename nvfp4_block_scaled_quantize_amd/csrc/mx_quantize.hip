// mx_quantize.hip -- MXFP4 quantization and its inverse.
//
// x_hat = E2M1(x / s) s with s = 2^(code - 127) from the block's largest magnitude (32
// elements).  Division by s is exact, so the only rounding is E2M1's.
#include "mx_common.h"

namespace nvfp4 {

struct MxQArgs {
    const void* x;
    int64_t batch, rows, cols, ld, stride;
    const int32_t* offsets;
    int n_groups;
    uint8_t *rc, *rs, *cc, *cs;
    int64_t row_kp, col_kp;     // K extents of the two copies
    uint32_t k0, k1;            // Philox key
};

// ROUND: NVFP4_RNE or NVFP4_SR.  Quantizes one block of 32 values and stores its 16 code bytes
// and its scale; e0: index of the block's first element (a multiple of 32).
template <int RULE, int ROUND>
__device__ __forceinline__ void quantize_block(const float (&v)[32], uint8_t* codes, uint8_t* scale,
                                               int64_t e0, uint32_t copy, uint32_t k0, uint32_t k1) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const uint32_t code = mx_scale_code<RULE>(m);
    const float cs = mx_scale_value(code);
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t word = 0;
        if constexpr (ROUND == NVFP4_RNE) {
            word = cvt_fp4x2<0>(word, v[8 * q + 0], v[8 * q + 1], cs);
            word = cvt_fp4x2<1>(word, v[8 * q + 2], v[8 * q + 3], cs);
            word = cvt_fp4x2<2>(word, v[8 * q + 4], v[8 * q + 5], cs);
            word = cvt_fp4x2<3>(word, v[8 * q + 6], v[8 * q + 7], cs);
        } else {
            const U4 c = {(uint32_t)((e0 >> 3) + q), (uint32_t)(((e0 >> 3) + q) >> 32), copy, kTagMxSR};
            const U4 r = philox10(c, k0, k1);
            const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
            // x / s in binary32 (exact but for results below 2^-126, which round to 0 either
            // way), then the conversion at unit scale
            const float inv = __uint_as_float((254u - code) << 23);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = (i & 1) ? rw[i >> 1] & 0xFFFF0000u : rw[i >> 1] << 16;
                word |= (cvt_fp4_sr(v[8 * q + i] * inv, bits) & 0xFu) << (4 * i);
            }
        }
        w[q] = code == 255u ? 0u : word;
    }
    *(uint4*)codes = make_uint4(w[0], w[1], w[2], w[3]);
    *scale = (uint8_t)code;
}

template <typename T> __device__ __forceinline__ float load_value(const T* p);
template <> __device__ __forceinline__ float load_value<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float load_value<uint16_t>(const uint16_t* p) {
    return bf16_to_f32(*p);
}

// One thread per block of the rowwise copy.
template <typename T, int RULE, int ROUND>
__global__ void k_mx_rows(MxQArgs g) {
    const int64_t per = g.row_kp / kMxBlock;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= g.batch * g.rows * per) return;
    const int64_t r = i / per, k = (i - r * per) * kMxBlock;
    const T* p = (const T*)g.x + r / g.rows * g.stride + r % g.rows * g.ld + k;
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = k + j < g.cols ? load_value(p + j) : 0.0f;
    quantize_block<RULE, ROUND>(v, g.rc + i * 16, g.rs + i, r * g.row_kp + k, 0, g.k0, g.k1);
}

// One thread per column of a 128-row unit of the columnwise copy.
template <typename T, int RULE, int ROUND>
__global__ void k_mx_cols(MxQArgs g, int64_t units, unsigned col_blocks) {
    const unsigned cb = blockIdx.x % col_blocks, ub = blockIdx.x / col_blocks;
    const int64_t b = ub / units, u = ub % units;
    int64_t row0 = u * kMxPad, rows = g.rows - row0, kp0 = u * kMxPad;
    if (g.n_groups) {
        MxUnit m;
        if (!mx_find_unit(g.offsets, g.n_groups, (int)g.rows, kMxPad, u, m) || m.group == g.n_groups)
            return;
        row0 = m.row0, rows = m.rows;
    }
    const int64_t c = (int64_t)cb * blockDim.x + threadIdx.x;
    if (c >= g.cols) return;
    const T* p = (const T*)g.x + b * g.stride + row0 * g.ld + c;
    for (int q = 0; q < kMxPad / kMxBlock; ++q) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = q * 32 + j < rows ? load_value(p + (q * 32 + j) * g.ld) : 0.0f;
        const int64_t e = (b * g.cols + c) * g.col_kp + kp0 + q * 32;
        quantize_block<RULE, ROUND>(v, g.cc + e / 2, g.cs + e / 32, e, 1, g.k0, g.k1);
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

__device__ __forceinline__ void store_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_value(uint16_t* p, float v) {
    // exact for copies of bf16 values; nearest even otherwise
    *p = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// One thread per 8 elements; a workgroup decodes 16 rows of a 128-wide unit of K.
template <typename T>
__global__ void k_mx_decode(MxDArgs g, unsigned units) {
    const int64_t u = blockIdx.x % units;
    int64_t k0 = u * kMxPad, left = g.k - k0;
    bool zero = false;
    if (g.n_groups) {
        MxUnit m;
        if (!mx_find_unit(g.offsets, g.n_groups, (int)g.k, kMxPad, u, m)) return;
        k0 = m.row0, left = m.rows, zero = m.group == g.n_groups;
    }
    const int64_t r = (int64_t)(blockIdx.x / units) * 16 + (threadIdx.x >> 4);
    const int j = (int)(threadIdx.x & 15) * 8;
    if (r >= g.n || j >= left) return;
    const int64_t e = r * g.kp + u * kMxPad + j;
    uint32_t w = 0, code = 0;
    if (!zero) w = *(const uint32_t*)(g.codes + e / 2), code = g.scales[e / 32];
    const float s = code == 255u ? __builtin_nanf("") : mx_scale_value(code);
    const float2v p[4] = {fp4x2_to_f32<0>(w), fp4x2_to_f32<1>(w), fp4x2_to_f32<2>(w), fp4x2_to_f32<3>(w)};
    T* o = (T*)g.out + r * g.ld + k0 + j;
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (j + q < left) store_value(o + q, p[q >> 1][q & 1] * s);
}

template <typename T, int RULE, int ROUND>
static void launch_rows(const MxQArgs& g, hipStream_t st) {
    const int64_t n = g.batch * g.rows * (g.row_kp / kMxBlock);
    k_mx_rows<T, RULE, ROUND><<<dim3((unsigned)((n + 255) / 256)), 256, 0, st>>>(g);
}
template <typename T, int RULE, int ROUND>
static void launch_cols(const MxQArgs& g, hipStream_t st) {
    const int64_t units = g.col_kp / kMxPad;
    const int64_t col_blocks = (g.cols + 255) / 256;
    k_mx_cols<T, RULE, ROUND><<<dim3((unsigned)(col_blocks * units * g.batch)), 256, 0, st>>>(
        g, units, (unsigned)col_blocks);
}

template <typename T, int RULE>
static void launch_quantize(const MxQArgs& g, const mxfp4_quant_params* p, hipStream_t st) {
    if (p->rowwise) {
        if (p->round_row == NVFP4_RNE) launch_rows<T, RULE, NVFP4_RNE>(g, st);
        else launch_rows<T, RULE, NVFP4_SR>(g, st);
    }
    if (p->colwise) {
        if (p->round_col == NVFP4_RNE) launch_cols<T, RULE, NVFP4_RNE>(g, st);
        else launch_cols<T, RULE, NVFP4_SR>(g, st);
    }
}

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
    if (batch < 0 || rows < 0 || cols < 0 || ld_x < cols) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    const auto flag = [](int32_t v) { return v == 0 || v == 1; };
    if (!flag(p->rowwise) || !flag(p->colwise) || !(p->rowwise || p->colwise) || !flag(p->scale_rule) ||
        !flag(p->round_row) || !flag(p->round_col))
        return NVFP4_ERR_MODE;
    if (int rc = mx_check_groups(offsets, n_groups, rows)) return rc;
    if (n_groups && batch != 1) return NVFP4_ERR_MODE;
    const bool used = batch && rows && cols;
    if (p->rowwise)
        if (int rc = mx_check_tensor(row_out, used)) return rc;
    if (p->colwise)
        if (int rc = mx_check_tensor(col_out, used)) return rc;
    MxQArgs g = {};
    g.row_kp = mx_pad(cols);
    g.col_kp = n_groups ? mxfp4_grouped_k(rows, n_groups) : mx_pad(rows);
    if (!used) return NVFP4_OK;
    if (!x) return NVFP4_ERR_NULL;
    if ((uintptr_t)x % size) return NVFP4_ERR_ALIGN;
    g.x = x, g.batch = batch, g.rows = rows, g.cols = cols, g.ld = ld_x, g.stride = batch_stride;
    g.offsets = offsets, g.n_groups = (int)n_groups;
    if (p->rowwise) g.rc = row_out->codes, g.rs = row_out->scales;
    if (p->colwise) g.cc = col_out->codes, g.cs = col_out->scales;
    g.k0 = (uint32_t)p->seed, g.k1 = (uint32_t)(p->seed >> 32);
    const hipStream_t st = (hipStream_t)stream;
    const bool ceil = p->scale_rule == MXFP4_SCALE_CEIL;
    if (dtype == NVFP4_BF16)
        ceil ? launch_quantize<uint16_t, MXFP4_SCALE_CEIL>(g, p, st)
             : launch_quantize<uint16_t, MXFP4_SCALE_FLOOR>(g, p, st);
    else
        ceil ? launch_quantize<float, MXFP4_SCALE_CEIL>(g, p, st)
             : launch_quantize<float, MXFP4_SCALE_FLOOR>(g, p, st);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

extern "C" int mxfp4_dequantize(const mxfp4_tensor* q, int64_t n, int64_t k, const int32_t* offsets,
                                int64_t n_groups, int out_dtype, void* out, int64_t ld_out,
                                void* stream) {
    if (n < 0 || k < 0 || ld_out < k) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(out_dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    if (int rc = mx_check_groups(offsets, n_groups, k)) return rc;
    if (int rc = mx_check_tensor(q, n && k)) return rc;
    if (n == 0 || k == 0) return NVFP4_OK;
    if (!out) return NVFP4_ERR_NULL;
    if ((uintptr_t)out % size) return NVFP4_ERR_ALIGN;
    MxDArgs g = {q->codes, q->scales, n, k, n_groups ? mxfp4_grouped_k(k, n_groups) : mx_pad(k),
                 offsets, (int)n_groups, out, ld_out};
    // one unit more than the copy holds: the rows in no group
    const unsigned units = (unsigned)(g.kp / kMxPad + (n_groups ? 1 : 0));
    const dim3 grid((unsigned)((n + 15) / 16 * units));
    const hipStream_t st = (hipStream_t)stream;
    if (out_dtype == NVFP4_BF16) k_mx_decode<uint16_t><<<grid, 256, 0, st>>>(g, units);
    else k_mx_decode<float><<<grid, 256, 0, st>>>(g, units);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}
