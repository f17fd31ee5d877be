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

typedef int int8v __attribute__((ext_vector_type(8)));

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

// An operand fragment: the instruction's E2M1 form reads the first four of eight registers.
__device__ __forceinline__ int8v mx_frag(int4v v) {
    return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}
constexpr int kE2M1 = 4;

__device__ __forceinline__ void store_c(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_c(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// One wave per 32 x 32 tile of C.
template <typename T, int MODE>
__global__ __launch_bounds__(64) void k_mx_gemm(MxGArgs g, unsigned tiles_n, unsigned tiles_m) {
    const unsigned tn = blockIdx.x % tiles_n, tq = blockIdx.x / tiles_n;
    const int lane = threadIdx.x, li = lane & 31, h = lane >> 5;
    int64_t m0 = (int64_t)(tq % tiles_m) * 32, m1 = g.M, kb0 = 0, kb1 = g.kp / 32;
    const uint8_t *bc = g.bc, *bs = g.bs;
    T* c = (T*)g.c;
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_unit(g.offsets, g.n_groups, (int)g.M, 32, tq, u)) return;
        m0 = u.row0, m1 = u.row0 + u.rows;
        if (u.group == g.n_groups) kb1 = 0;
        bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
    } else if constexpr (MODE == MxK) {
        MxUnit u;
        mx_group(g.offsets, g.n_groups, (int)g.k_rows, kMxPad, (int)(tq / tiles_m), u);
        kb0 = u.first * (kMxPad / 32), kb1 = kb0 + mx_blocks(u.rows);
        c += (int64_t)u.group * g.M * g.ldc;
    }
    const int64_t n0 = (int64_t)tn * 32;
    const int64_t am = m0 + li < m1 ? m0 + li : m1 - 1, bn = n0 + li < g.N ? n0 + li : g.N - 1;
    float16v acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
    for (int64_t kb = kb0 + h; kb < kb1 + h; kb += 2) {
        const int4v a = *(const int4v*)(g.ac + am * pitch + kb * 16);
        const int4v b = *(const int4v*)(bc + bn * pitch + kb * 16);
        const int sa = g.as[am * spitch + kb], sb = bs[bn * spitch + kb];
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_frag(a), mx_frag(b), acc, kE2M1, kE2M1, 0,
                                                              sa, 0, sb);
    }
    // register r of lane l is row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int64_t row = m0 + 8 * (r >> 2) + 4 * h + (r & 3), col = n0 + li;
        if (row < m1 && col < g.N) store_c(c + row * g.ldc + col, acc[r]);
    }
}

template <int MODE>
static int launch_gemm(const MxGArgs& g, int c_dtype, hipStream_t st) {
    const int64_t tn = (g.N + 31) / 32;
    int64_t tm = (g.M + 31) / 32, tiles = tm * tn;
    if (MODE == MxRows) tiles = (g.M / 32 + (g.n_groups < g.M ? g.n_groups : g.M) + 1) * tn;
    if (MODE == MxK) tiles *= g.n_groups;
    const dim3 grid((unsigned)tiles);
    if (c_dtype == NVFP4_BF16) k_mx_gemm<uint16_t, MODE><<<grid, 64, 0, st>>>(g, (unsigned)tn, (unsigned)tm);
    else k_mx_gemm<float, MODE><<<grid, 64, 0, st>>>(g, (unsigned)tn, (unsigned)tm);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
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

extern "C" size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    (void)N, (void)n_groups;
    return M > 0 && K > 0 ? linear_code_bytes(M, K) + (size_t)(M * (mx_pad(K) / 32)) : 0;
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
    // the product's arguments are checked before the quantization is enqueued
    bool empty;
    if (int rc = check_gemm(&q, w, M, N, K, c, c_dtype, ldc, &empty)) return rc;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (int rc = mxfp4_quantize(x, dtype, 1, M, K, ld_x, 0, nullptr, 0, &p, &q, nullptr, stream)) return rc;
    return n_groups ? mxfp4_gemm_grouped(&q, w, offsets, n_groups, M, N, K, c, c_dtype, ldc, stream)
                    : mxfp4_gemm(&q, w, M, N, K, c, c_dtype, ldc, stream);
}
