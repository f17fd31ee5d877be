// mx8.hip -- 8-bit (MXFP8) activation checkpoints: made of a tensor, decoded, and read by the backward
// pass of the gated product from a dH in memory.
//
// x_hat = E4M3(x / s) s with s = 2^(code - 127) the smallest power of two with amax <= 448 s, 32 elements a
// block.  Division by s is exact, so the only rounding is E4M3's.
//
// All three are bound by memory: an element costs 33/32 bytes of the checkpoint and what the tensors
// beside it take.  From memory, 8192 x 4096 bfloat16: made in 16.4 us (102 MB, 6.2 TB/s), decoded in 15.6
// (6.5); the backward pass of 8192 x 9216 with H 129 us, 760 MB, 5.9 TB/s.  1021 x 1531 float32 4.2 and 3.8
// us, an empty kernel 2.4.
#include "mx_ffn.h"
#include "mx_pieces.h"

namespace nvfp4 {

struct Mx8Args {
    const void* x;
    int64_t batch, rows, cols, ld, stride;
    uint8_t *codes, *scales;
    int64_t kp;
};

// A lane per eight elements, a quad per block; a workgroup takes kSteps8 times 256 consecutive octs of the
// padded checkpoint, all loaded before the first is used.
constexpr int kSteps8 = 4;
template <typename T>
__global__ __launch_bounds__(256) void k_mx8_quantize(Mx8Args g) {
    const uint32_t per = (uint32_t)(g.kp / 8);      // octs of a row
    const int64_t first = (int64_t)blockIdx.x * (256 * kSteps8), total = g.batch * g.rows * per;
    const int64_t row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    Oct<T> o[kSteps8];
#pragma unroll
    for (int i = 0; i < kSteps8; ++i) {
        const uint32_t at = rem + threadIdx.x + 256 * i, dr = at / per;
        const int64_t r = row0 + dr, k = (int64_t)(at - dr * per) * 8;
        const int64_t b = g.batch == 1 ? 0 : r / g.rows;
        const bool in = first + threadIdx.x + 256 * i < total;
        o[i] = load_oct((const T*)g.x + b * g.stride + (r - b * g.rows) * g.ld + k, in ? g.cols - k : 0);
    }
#pragma unroll
    for (int i = 0; i < kSteps8; ++i) {
        const int64_t at = first + threadIdx.x + 256 * i;   // oct of the checkpoint
        const uint32_t code = mx8_scale_code(quad_max(max_bits(o[i])));
        const float scale = mx_scale_value(code);
        uint32_t w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            w[j] = mx8_codes(value(o[i], 4 * j), value(o[i], 4 * j + 1), value(o[i], 4 * j + 2), value(o[i], 4 * j + 3), scale);
            if (code == 255u) w[j] = 0;
        }
        if (at < total) {
            *(uint2*)(g.codes + at * 8) = make_uint2(w[0], w[1]);
            if ((threadIdx.x & 3) == 0) g.scales[at >> 2] = (uint8_t)code;
        }
    }
}

// n codes (4 or 8) of a row, those past `left` zero.
template <int n>
__device__ __forceinline__ void load_codes8(const uint8_t* p, int64_t left, uint32_t (&w)[n / 4]) {
#pragma unroll
    for (int i = 0; i < n / 4; ++i) w[i] = left > 0 ? ((const uint32_t*)p)[i] : 0u;
}

template <typename T>
__device__ __forceinline__ int4v pack_piece(const float (&v)[Piece<T>::n]) {
    T e[Piece<T>::n];
#pragma unroll
    for (int i = 0; i < Piece<T>::n; ++i) {
        if constexpr (sizeof(T) == 2) e[i] = __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        else e[i] = v[i];
    }
    int4v d;
    __builtin_memcpy(&d, e, sizeof(d));
    return d;
}

// A lane per 16 bytes of output.
template <typename T>
__global__ __launch_bounds__(256) void k_mx8_decode(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                                    int64_t kp, T* out, int64_t ld) {
    constexpr int n = Piece<T>::n;
    const uint32_t per = (uint32_t)(kp / n);
    const int64_t first = (int64_t)blockIdx.x * (256 * kSteps8), total = rows * per;
    const int64_t row0 = first / per;
    const uint32_t rem = (uint32_t)(first - row0 * per);
    uint32_t w[kSteps8][n / 4], code[kSteps8];
#pragma unroll
    for (int i = 0; i < kSteps8; ++i) {
        const int64_t at = first + threadIdx.x + 256 * i;
        load_codes8<n>(codes + at * n, total - at, w[i]);
        code[i] = at < total ? scales[at / (32 / n)] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kSteps8; ++i) {
        const uint32_t at = rem + threadIdx.x + 256 * i, dr = at / per;
        const int64_t r = row0 + dr, k = (int64_t)(at - dr * per) * n;
        const bool in = first + threadIdx.x + 256 * i < total;
        const float s = mx8_factor(code[i]);
        float v[n];
#pragma unroll
        for (int j = 0; j < n / 4; ++j) {
            const Quad q = mx8_values(w[i][j], s);
#pragma unroll
            for (int m = 0; m < 4; ++m) v[4 * j + m] = q.v[m];
        }
        store_piece(pack_piece<T>(v), out + r * ld + k, in ? cols - k : 0, k == 0 || (threadIdx.x & 63) == 0);
    }
}

// n elements of a row of dH, those past `left` zero.
template <int n>
__device__ __forceinline__ void load_row(const uint16_t* p, int64_t left, float (&v)[n]) {
    if (left >= n) {
        uint32_t w[n / 2];
        __builtin_memcpy(w, p, sizeof(w));
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = i < left ? bf16_to_f32(p[i]) : 0.0f;
    }
}
template <int n>
__device__ __forceinline__ void load_row(const float* p, int64_t left, float (&v)[n]) {
    if (left >= n) {
        __builtin_memcpy(v, p, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = i < left ? p[i] : 0.0f;
    }
}

// A lane per 16 bytes of dG, of dU and of H.
template <typename T, typename XT, int ACT>
__global__ __launch_bounds__(256) void k_mx8_gated_backward(MxFfnArgs f, const XT* dh, int64_t ld_dh) {
    constexpr int n = Piece<T>::n;
    const MxGArgs& g = f.g;
    const uint32_t per = (uint32_t)(f.np / n);
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, total = g.M * per;
    const int64_t r = at / per, k = (at - r * per) * n, second = g.M * f.np;
    const int64_t left = at < total ? g.N - k : 0;
    float d[n];
    load_row<n>(dh + r * ld_dh + k, left, d);
    uint32_t gw[n / 4], uw[n / 4];
    load_codes8<n>(f.kc + at * n, left, gw);
    load_codes8<n>(f.kc + second + at * n, left, uw);
    const float gs = mx8_factor(left > 0 ? f.ks[at / (32 / n)] : 0u), us = mx8_factor(left > 0 ? f.ks[second / 32 + at / (32 / n)] : 0u);
    float dg[n], du[n], x[n];
#pragma unroll
    for (int j = 0; j < n / 4; ++j) {
        const Quad gq = mx8_values(gw[j], gs), uq = mx8_values(uw[j], us);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Act a = act_both<ACT>(gq.v[i]);
            du[4 * j + i] = d[4 * j + i] * a.a;
            dg[4 * j + i] = d[4 * j + i] * uq.v[i] * a.slope;
            x[4 * j + i] = a.a * uq.v[i];
        }
    }
    const bool start = k == 0 || (threadIdx.x & 63) == 0;
    T* const p = (T*)g.c + r * g.ldc + k;
    store_piece(pack_piece<T>(dg), p, left, start);
    store_piece(pack_piece<T>(du), p + g.N, left, start);
    if (f.h) store_piece(pack_piece<T>(x), (T*)f.h + r * f.ldh + k, left, start);
}

template <typename T, typename XT>
static int launch_backward(const MxFfnArgs& f, const void* dh, int64_t ld_dh, int act, hipStream_t st) {
    const __int128 grid = ((__int128)f.g.M * (f.np / Piece<T>::n) + 255) / 256;
    if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
    const auto kernel = act == MXFP4_SILU ? k_mx8_gated_backward<T, XT, MXFP4_SILU> : k_mx8_gated_backward<T, XT, MXFP4_GELU>;
    kernel<<<dim3((unsigned)grid), 256, 0, st>>>(f, (const XT*)dh, ld_dh);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <typename T>
static int launch_decode(const mxfp8_tensor* q, int64_t n, int64_t k, void* out, int64_t ld, hipStream_t st) {
    const int64_t kp = mx_pad(k), per = 256 * kSteps8;
    const __int128 grid = ((__int128)n * (kp / Piece<T>::n) + per - 1) / per;
    if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
    k_mx8_decode<T><<<dim3((unsigned)grid), 256, 0, st>>>(q->codes, q->scales, n, k, kp, (T*)out, ld);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int mxfp8_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld_x,
                              int64_t batch_stride, const mxfp8_tensor* q, void* stream) {
    if (!mx_extent(batch) || !mx_extent(rows) || !mx_extent(cols) || ld_x < cols) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    const bool used = batch && rows && cols;
    if (int rc = mx8_check_tensor(q, used)) return rc;
    if (!used) return NVFP4_OK;
    if (!x) return NVFP4_ERR_NULL;
    if ((uintptr_t)x % size) return NVFP4_ERR_ALIGN;
    const Mx8Args g = {x, batch, rows, cols, ld_x, batch_stride, q->codes, q->scales, mx_pad(cols)};
    const int per = 256 * kSteps8;
    const __int128 grid = ((__int128)batch * rows * (g.kp / 8) + per - 1) / per;
    if (!mx_grid_fits(grid, 256)) return NVFP4_ERR_SHAPE;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == NVFP4_BF16) k_mx8_quantize<uint16_t><<<dim3((unsigned)grid), 256, 0, st>>>(g);
    else k_mx8_quantize<float><<<dim3((unsigned)grid), 256, 0, st>>>(g);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

extern "C" int mxfp8_dequantize(const mxfp8_tensor* q, int64_t n, int64_t k, int out_dtype, void* out, int64_t ld_out,
                                void* stream) {
    if (!mx_extent(n) || !mx_extent(k) || ld_out < k) return NVFP4_ERR_SHAPE;
    const int size = mx_dtype_size(out_dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    if (int rc = mx8_check_tensor(q, n && k)) return rc;
    if (n == 0 || k == 0) return NVFP4_OK;
    if (!out) return NVFP4_ERR_NULL;
    if ((uintptr_t)out % size) return NVFP4_ERR_ALIGN;
    const hipStream_t st = (hipStream_t)stream;
    return out_dtype == NVFP4_BF16 ? launch_decode<uint16_t>(q, n, k, out, ld_out, st) : launch_decode<float>(q, n, k, out, ld_out, st);
}

extern "C" int mxfp8_gated_backward(const void* dh, int dh_dtype, int64_t ld_dh, int64_t M, int64_t N, int32_t activation,
                                    const mxfp8_tensor* checkpoint, void* dgu, int dtype, int64_t ld, void* h, int64_t ldh,
                                    void* stream) {
    if (!mx_extent(M) || !mx_extent(N) || ld_dh < N || ld < 2 * N || (h && ldh < N)) return NVFP4_ERR_SHAPE;
    if (!mx_activation(activation)) return NVFP4_ERR_MODE;
    const int size = mx_dtype_size(dtype), dh_size = mx_dtype_size(dh_dtype);
    if (!size || !dh_size) return NVFP4_ERR_DTYPE;
    const bool used = M && N;
    if (int rc = mx8_check_tensor(checkpoint, used)) return rc;
    if (!used) return NVFP4_OK;
    if (!dh || !dgu) return NVFP4_ERR_NULL;
    if ((uintptr_t)dh % dh_size || (uintptr_t)dgu % size || (uintptr_t)h % size) return NVFP4_ERR_ALIGN;
    MxFfnArgs f = {};
    f.g.M = M, f.g.N = N, f.g.c = dgu, f.g.ldc = ld;
    f.kc = checkpoint->codes, f.ks = checkpoint->scales, f.np = mx_pad(N), f.h = h, f.ldh = ldh;
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == NVFP4_BF16)
        return dh_dtype == NVFP4_BF16 ? launch_backward<uint16_t, uint16_t>(f, dh, ld_dh, activation, st)
                                      : launch_backward<uint16_t, float>(f, dh, ld_dh, activation, st);
    return dh_dtype == NVFP4_BF16 ? launch_backward<float, uint16_t>(f, dh, ld_dh, activation, st)
                                  : launch_backward<float, float>(f, dh, ld_dh, activation, st);
}
