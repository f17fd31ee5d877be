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

// How C is stored.  bfloat16 always streams past the caches: where no kernel reads C next that
// gains (grouped 16384 x 4096 x 2048 95 us against 100 with ordinary stores), where a quantizer
// does it loses less (8192 x 9216 x 4096 with its reader 186 against 182, 2048 x 4096 x 2048 the
// same), and the call does not know which.  float32 does where C is larger than the last-level
// cache (256 MB), so that no reader could find much of it there: 15 gradients of 4096 x 2048 (503
// MB) 109 us against 141, 8192 x 9216 x 4096 (302 MB) with its reader 227 against 242; but 268 MB
// (8192 x 8192 x 2048) with a reader 157 against 145, 134 MB 109 against 100.  Gradients of groups
// are read after the whole backward pass: they do from half of that on, which leaves the cache to
// the next layer's operands (measured at one size, 15 of 1536 x 2048, 189 MB: 43 us either way, a
// step of their layer 164 against 187).  A dense float32 C may be Y or dX, which are read next: it
// keeps the upper bound.
static bool streams(const MxGArgs& g, int mode) {
    return mode == MxK ? g.M * g.N * 4 * g.n_groups > ((int64_t)128 << 20) : g.M * g.N * 4 > ((int64_t)256 << 20);
}

// Which tile.  256 x 256 tiles run one to a compute unit, 256 at a time (these rules count
// workgroups for an MI355X's 256 units); 128 x 128 tiles two to a unit.  In percent of a round of
// the large ones, 512 small ones take 68 and up to 256 of them 45 (8192^3: 4 rounds 232 us against
// 8 299 us; 2048 x 2048 x 4096: 64 large 25.1 us, 256 small 12.5), so the small tile wins where the
// large ones' last round would be mostly empty: 2048 x 9216 x 4096 (288 large tiles) 49 against 56
// us, 1024 x 6144 x 4096 (96) 19.6 against 24.9, but 1024 x 9216 x 4096 (144 large, 576 small) 30.3
// against 25.8.  Groups of rows end in half a tile on average: 2048 rows over 29 groups (x 4096 x
// 2048) 27.6 against 36.3, 16384 rows 105.7 against 95.7.
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
    return mx_tile128(g, MODE, c_dtype, streams(g, MODE), st);
}

// Whether a product's extents are ones that the launch code can count with.
static bool gemm_extents(int64_t M, int64_t N, int64_t K) {
    return mx_extent(M) && mx_extent(N) && K >= 0 && K <= kMxMaxK && (N == 0 || M <= kMxMaxC / N);
}

// Checks shared by the products; *empty when C has no elements.
static int check_gemm(const mxfp4_tensor* a, const mxfp4_tensor* b, int64_t M, int64_t N, int64_t K,
                      const void* c, int c_dtype, int64_t ldc, bool* empty) {
    if (!gemm_extents(M, N, K) || ldc < N) return NVFP4_ERR_SHAPE;
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
    // Few rows, and products of few tiles, go to the kernel that splits K over the waves of a
    // workgroup: 16 x 6144 x 4096 6.1 us against 10.7, 77 x 4999 x 2056 (471 of its workgroups) 6.0
    // against 8.9, 256 x 1024 x 4096 (256) 5.8 against 10.7; but 64 x 9216 x 2048 (576) 7.8 either way,
    // 128 x 6144 x 4096 (768) 12.8 against 11.5.
    if (K > 0 && mx_few_dense(M, N, g.kp)) return mx_few_packed({g, nullptr, 0, K, 0}, c_dtype, (hipStream_t)stream);
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
    const int64_t busy = n_groups < M ? n_groups : M;
    // Up to 48 Ki elements of A a group, or a row, go to the kernel that streams B (4096 x 2048, 17
    // groups: 80 rows 14.2 us against 19.8, 400 rows 17.8 against 20.2; 2048 x 6144, 8 groups: 16 rows
    // 11.4 against 15.0; 9216 x 4096, 4 groups: 32 rows 17.3 against 19.3, 64 rows (64 Ki a group)
    // 21.2 against 19.5).
    if (K > 0 && M * g.kp <= busy * (g.kp > 48 << 10 ? g.kp : 48 << 10) && mx_few_fits(M, g.kp))
        return mx_few_packed({g, nullptr, 0, K, 0}, c_dtype, (hipStream_t)stream);
    return launch_gemm<MxRows>(g, c_dtype, (hipStream_t)stream);
}

extern "C" int mxfp4_gemm_grouped_wgrad(const mxfp4_tensor* a, const mxfp4_tensor* b,
                                        const int32_t* offsets, int64_t n_groups, int64_t M, int64_t N,
                                        int64_t rows, void* c, int c_dtype, int64_t ldc, void* stream) {
    bool empty;
    if (!mx_extent(rows) || n_groups < 1) return NVFP4_ERR_SHAPE;
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

// Few rows are quantized inside the product, which saves a launch (about 3 us) and the workspace,
// as long as every workgroup's doing so costs less.  Dense: a workgroup's elements times the
// workgroups a compute unit, up to 48 Ki.  64 x 1024 x 2048 (32 Ki) 5.6 us of GPU time against 6.4
// as two kernels, 32 x 4096 x 1024 (32 Ki) 6.0 against 6.5, 12 x 4096 x 4096 (48 Ki) 7.0 against
// 6.9 and a launch less; 32 x 1024 x 4096 (64 Ki) 8.2 against 7.0, 16 x 9216 x 2048 (72 Ki) 10.0
// against 7.6.  One or two rows cost less than the launch whatever their length: 1 x 50000 x 4096
// 20.2 against 23.2, 2 x 21.5 against 23.3, 4 x 26.4 against 23.7.  Grouped: up to 8 Ki elements,
// or a row, a group.  Of N x K 4096 x 2048 and 17 groups 40 rows (5 Ki a group) 16.2 against 17.0,
// 60 rows (7 Ki) 18.0 against 17.3 and a launch less; of 1536 x 2048 and 29 groups 64 rows 12.0
// against 13.3, 128 rows (9 Ki) 15.4 against 14.2; of 9216 x 4096 and 4 groups 8 rows 16.0 against
// 18.2, 16 rows (16 Ki) 21.4 against 19.4.
static bool linear_fused(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    const int64_t kp = mx_pad(K), busy = n_groups < M ? n_groups : M;
    if (M <= 0 || K <= 0) return false;
    if (n_groups) return M * kp <= busy * (kp > 8192 ? kp : 8192) && mx_few_fits(M, kp);
    return mx_few_dense(M, N, kp) && (M <= 2 || mx_few_quantized(M, N, kp) <= 48 << 10);
}

extern "C" size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    if (!gemm_extents(M, N, K)) return 0;       // mxfp4_linear refuses them
    return M > 0 && K > 0 && !linear_fused(M, N, K, n_groups) ? linear_code_bytes(M, K) + (size_t)(M * (mx_pad(K) / 32)) : 0;
}

extern "C" int mxfp4_linear(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x,
                            int32_t scale_rule, const mxfp4_tensor* w, int64_t N, const int32_t* offsets,
                            int64_t n_groups, void* c, int c_dtype, int64_t ldc, void* ws,
                            size_t ws_bytes, void* stream) {
    if (!gemm_extents(M, N, K)) return NVFP4_ERR_SHAPE;
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
    if (x && linear_fused(M, N, K, n_groups)) {
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
