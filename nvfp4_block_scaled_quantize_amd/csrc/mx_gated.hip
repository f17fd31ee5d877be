// mx_gated.hip -- the gated feed-forward block on MXFP4 products: the entry points.
//
// Forward: G and U are the products of A with the two halves of W, H = a(G) U.  Backward: dH is a
// product, dG and dU follow from it and the checkpoint's G and U.  Either way what is done to an
// element needs no other but those of its block of 32, which a lane pair holds, so it is done to the
// accumulators and nothing but the results goes to memory.
#include "mx_ffn.h"

namespace nvfp4 {

// Which tile of the forward, in percent of a round of 256 large ones (the rule of mx_gemm.hip; the epilogues of 512
// small ones run beside each other's products): 512 small ones take 55, up to 256 of them 37.  8192 x 9216 x 4096
// 318 us against 345 with small ones, 4096 x 4096 x 8192 132 against 148, 8192 x 2048 x 2048 44 against 46; but
// 2048 x 9216 x 4096 (576 large tiles) 115 against 92.  Where rows are grouped a large tile's ends cost a little
// more: H over 8 groups, 32768 rows, 4608 x 4096, 747 against 794, over 2, 8192, 9216 x 4096, 391 against 403; over 4, 16384,
// 2048 x 4096, 190 against 188 (and the packed copy 193 against 179), 8191 over 15 of 16, 1536 x 2048, 52 against 47.  (Few
// rows in each of many groups it judges a little too well for the small ones: 16384 over 60 of 64, 4096 x 2048, 290,
// 277 with large ones.)  float32 H is left to the small ones: 8192 x 9216 x 4096 375, with large ones 345.
static int launch_forward(const MxFfnArgs& f, int dtype, int act, hipStream_t st) {
    const MxGArgs& g = f.g;
    const int mode = g.n_groups ? MxRows : MxDense;
    const auto tiles = [&](int64_t side) {
        int64_t m = (g.M + side - 1) / side;
        if (mode == MxRows) m = (2 * g.M / side + (g.n_groups < g.M ? g.n_groups : g.M) + 1) / 2;
        return m * ((2 * g.N + side - 1) / side);
    };
    const int64_t big = (tiles(256) + 255) / 256 * (mode == MxRows ? 102 : 100), n = tiles(128), rest = n % 512;
    const int64_t small = n / 512 * 55 + (rest == 0 ? 0 : rest <= 256 ? 37 : 55);
    if (dtype == NVFP4_BF16 && big <= small) return mx_forward256(f, mode, act, st);
    return mx_forward128(f, mode, dtype, act, st);
}

// Whether H alone, of A packed, goes to the kernel for few rows.  Dense: up to 16 rows, or as long as no compute unit
// gets a second workgroup (17 x 4096 x 4096, 256 workgroups, 7.5 us against 11.6 by tiles, 256 x 512 x 4096 6.6
// against 11.2; but 77 x 4999 x 2056, 471, 11.0 against 9.3, 64 x 9216 x 4096, 576, 25 against 13).  Groups: up to 48
// Ki elements of A a group, or a row (1536 x 2048, 17 groups: 80 rows 13.6 against 14.2, 400 over 29 groups 20.6
// against 23.4, 800 24.9 against 24.1).  (A group: on average.  Which of them hold rows is known on the device alone.)
static bool few_packed(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    const int64_t kp = mx_pad(K), busy = n_groups < M ? n_groups : M;
    if (M <= 0 || N <= 0 || K <= 0) return false;
    if (n_groups) return M * kp <= busy * (kp > 48 << 10 ? kp : 48 << 10) && mx_few_rows(M, N, kp, n_groups);
    return mx_ffn_few_dense(M, N, kp);
}
// Whether x is quantized inside it: as long as that costs every workgroup less than a launch.  Dense: a workgroup's
// elements times the workgroups a compute unit up to 48 Ki, or two rows (16 x 2048 x 2048, 32 Ki, 6.3 us
// against 7.2 as two kernels; 64 x 4096 x 2048, 64 Ki, 10.0 against 8.7); groups: up to 8 Ki elements a group, or a row
// (24 rows over 17 of 32 groups, 1536 x 2048, 13.0 against 15.4; 400 over 29 28.0 against 23.8).
static bool few_fused(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    const int64_t kp = mx_pad(K), busy = n_groups < M ? n_groups : M;
    if (!few_packed(M, N, K, n_groups)) return false;
    if (n_groups) return M * kp <= busy * (kp > 8192 ? kp : 8192);
    return M <= 2 || mx_ffn_few_quantized(M, N, kp) <= 48 << 10;
}

// Whether the backward goes there, where its epilogue costs less than on tiles.  Dense: what the plain products send,
// or up to 800 workgroups of 32 x 32 (300 x 1500 x 1000, 470 of them, 6.2 us against 12.7, 700 x 777 x 1300, 550, 10.3
// against 13.4, 1000 x 777 x 489, 800, 9.6 against 11.7; but 512 x 2048 x 2048, 1024, 12.7 against 11.5).  Groups: up
// to 48 Ki elements of dY a group, or a row (400 rows over 29 groups, 1536 x 2048, 16.0 against 19.5; 600 over 15, 77
// Ki, 15.4 against 13.7), or up to 1024 such workgroups (1000 x 600 x 700 over 6 groups, 703, 7.0 against 11.8; 600 x
// 1024 x 2048 over 12, 960, 13.0 either way).  Of either only where workgroups (of groups: the usual number, half of
// the last ones full) times K are below 2.5 Mi, or 2.25 Mi: longer rows take more of a compute unit's LDS, so that from
// K = 4096 on two workgroups of it run at once, at 8192 one, while tiles gain.  Dense 2000 x 300 x 4096, 630 of them,
// 15.4 against 18.6, but 1000 x 800 x 4096, 800, 18.6 against 17.7, 600 x 1024 x 8192, 608, 27.7 against 22.5; 300 x
// 1500 x 4096 over 4 groups, 517, 15.1 against 18.4, 350 x 473 x 7017 over 16, 270, 12.6 against 22.5, but 512 x 1024 x
// 4096 over 4, 576, 19.1 against 16.6, 1000 x 800 over 6, 850, K = 2048 13.1 against 14.2, K = 4096 18.8 against 17.7, K =
// 8192 38.9 against 24.4.  (The forward on as few of these in groups wins at short rows alone: 3000 x 100 x 300
// over 10 5.2 against 6.7, 5000 x 64 x 4096 over 12 18.1 against 12.3.)
static bool few_backward(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    const int64_t kp = mx_pad(K), busy = n_groups < M ? n_groups : M, cols = (N + 31) / 32;
    if (M <= 0 || N <= 0 || K <= 0) return false;
    if (n_groups) {
        const int64_t most = (M / 32 + busy) * cols, usual = (2 * (M / 32) + busy) / 2 * cols;
        return (M * kp <= busy * (kp > 48 << 10 ? kp : 48 << 10) || (most <= 1024 && usual * kp < 9 << 18)) &&
               mx_few_rows(M, N, kp, n_groups);
    }
    const int64_t workgroups = (M + 31) / 32 * cols;
    return mx_few_dense(M, N, kp) || (workgroups <= 800 && workgroups * kp < 5 << 19 && mx_few_two_fit(M, kp));
}

// Extents as in mxfp4_gemm, for a product of 2 N columns.
static bool ffn_extents(int64_t M, int64_t N, int64_t K) {
    return mx_extent(M) && mx_extent(N) && mx_extent(2 * N) && K >= 0 && K <= kMxMaxK &&
           (N == 0 || M <= kMxMaxC / (2 * mx_pad(N)));
}
// A result of row pitch ld >= cols.
static int check_result(const void* p, int dtype, int64_t ld, int64_t cols, bool used) {
    const int size = mx_dtype_size(dtype);
    if (!size) return NVFP4_ERR_DTYPE;
    if (ld < cols) return NVFP4_ERR_SHAPE;
    if (used && !p) return NVFP4_ERR_NULL;
    return (uintptr_t)p % size ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int mxffn_abi_version(void) { return MXFFN_ABI_VERSION; }

extern "C" int mxfp4_gated(const mxfp4_tensor* a, const mxfp4_tensor* w, const int32_t* offsets, int64_t n_groups,
                           int64_t M, int64_t N, int64_t K, int32_t activation, void* h, int h_dtype, int64_t ldh,
                           int32_t scale_rule, const mxfp4_tensor* h_copy, const mxfp8_tensor* checkpoint,
                           void* stream) {
    if (!ffn_extents(M, N, K)) return NVFP4_ERR_SHAPE;
    if (!mx_activation(activation)) return NVFP4_ERR_MODE;
    if (scale_rule != MXFP4_SCALE_FLOOR && scale_rule != MXFP4_SCALE_CEIL) return NVFP4_ERR_MODE;
    const bool used = M && N;
    if (used && !h && !h_copy && !checkpoint) return NVFP4_ERR_NULL;
    if (h)
        if (int rc = check_result(h, h_dtype, ldh, N, used)) return rc;
    if (int rc = mx_check_tensor(a, M && K)) return rc;
    if (int rc = mx_check_tensor(w, N && K)) return rc;
    if (h_copy)
        if (int rc = mx_check_tensor(h_copy, used)) return rc;
    if (checkpoint)
        if (int rc = mx8_check_tensor(checkpoint, used)) return rc;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (!used) return NVFP4_OK;
    MxFfnArgs f = {{a->codes, a->scales, w->codes, w->scales, M, N, mx_pad(K), 0, h, ldh, offsets, (int)n_groups},
                   mx_above(scale_rule), nullptr, nullptr, nullptr, nullptr, mx_pad(N), nullptr, 0};
    if (h_copy) f.qc = h_copy->codes, f.qs = h_copy->scales;
    if (checkpoint) f.kc = checkpoint->codes, f.ks = checkpoint->scales;
    if (!h_copy && !checkpoint && few_packed(M, N, K, n_groups))
        return mx_ffn_few({f.g, nullptr, 0, K, 0}, 0, h_dtype, activation, (hipStream_t)stream);
    return launch_forward(f, h ? h_dtype : NVFP4_BF16, activation, (hipStream_t)stream);
}

static size_t linear_code_bytes(int64_t M, int64_t K) {
    return ((size_t)(M * (mx_pad(K) / 2)) + 255) / 256 * 256;
}

extern "C" size_t mxfp4_gated_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    if (!ffn_extents(M, N, K)) return 0;        // mxfp4_gated_linear refuses them
    return M > 0 && K > 0 && !few_fused(M, N, K, n_groups) ? linear_code_bytes(M, K) + (size_t)(M * (mx_pad(K) / 32)) : 0;
}

extern "C" int mxfp4_gated_linear(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x, int32_t scale_rule,
                                  const mxfp4_tensor* w, int64_t N, const int32_t* offsets, int64_t n_groups,
                                  int32_t activation, void* h, int h_dtype, int64_t ldh, void* ws, size_t ws_bytes,
                                  void* stream) {
    if (!ffn_extents(M, N, K)) return NVFP4_ERR_SHAPE;
    if (!mx_activation(activation)) return NVFP4_ERR_MODE;
    const size_t need = mxfp4_gated_linear_workspace_bytes(M, N, K, n_groups);
    if (need && (!ws || ws_bytes < need)) return NVFP4_ERR_WORKSPACE;
    if ((uintptr_t)ws & 255) return NVFP4_ERR_ALIGN;
    // the product's arguments are checked before the quantization is enqueued
    const bool used = M && N;
    if (int rc = check_result(h, h_dtype, ldh, N, used)) return rc;
    if (int rc = mx_check_tensor(w, N && K)) return rc;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (x && few_fused(M, N, K, n_groups)) {
        if (const int size = mx_dtype_size(dtype); !size) return NVFP4_ERR_DTYPE;
        else if ((uintptr_t)x % size) return NVFP4_ERR_ALIGN;
        if (ld_x < K) return NVFP4_ERR_SHAPE;
        if (scale_rule != MXFP4_SCALE_FLOOR && scale_rule != MXFP4_SCALE_CEIL) return NVFP4_ERR_MODE;
        const MxFArgs f = {{nullptr, nullptr, w->codes, w->scales, M, N, mx_pad(K), 0, h, ldh, offsets, (int)n_groups},
                           x, ld_x, K, mx_above(scale_rule)};
        return mx_ffn_few(f, dtype, h_dtype, activation, (hipStream_t)stream);
    }
    const mxfp4_tensor q = {(uint8_t*)ws, (uint8_t*)ws + (need ? linear_code_bytes(M, K) : 0)};
    const mxfp4_quant_params p = {1, 0, scale_rule, NVFP4_RNE, NVFP4_RNE, 0};
    if (int rc = mxfp4_quantize(x, dtype, 1, M, K, ld_x, 0, nullptr, 0, &p, &q, nullptr, stream)) return rc;
    return mxfp4_gated(&q, w, offsets, n_groups, M, N, K, activation, h, h_dtype, ldh, scale_rule, nullptr, nullptr, stream);
}

extern "C" int mxfp4_gated_backward(const mxfp4_tensor* dy, const mxfp4_tensor* w, const int32_t* offsets,
                                    int64_t n_groups, int64_t M, int64_t N, int64_t K, int32_t activation,
                                    const mxfp8_tensor* checkpoint, void* dgu, int dtype, int64_t ld, void* h,
                                    int64_t ldh, void* stream) {
    if (!ffn_extents(M, N, K)) return NVFP4_ERR_SHAPE;
    if (!mx_activation(activation)) return NVFP4_ERR_MODE;
    const bool used = M && N;
    if (int rc = check_result(dgu, dtype, ld, 2 * N, used)) return rc;
    if (h)
        if (int rc = check_result(h, dtype, ldh, N, used)) return rc;
    if (int rc = mx_check_tensor(dy, M && K)) return rc;
    if (int rc = mx_check_tensor(w, N && K)) return rc;
    if (int rc = mx8_check_tensor(checkpoint, used)) return rc;
    if (int rc = mx_check_groups(offsets, n_groups, M)) return rc;
    if (!used) return NVFP4_OK;
    const MxFfnArgs f = {{dy->codes, dy->scales, w->codes, w->scales, M, N, mx_pad(K), 0, dgu, ld, offsets, (int)n_groups},
                         0, nullptr, nullptr, checkpoint->codes, checkpoint->scales, mx_pad(N), h, ldh};
    if (few_backward(M, N, K, n_groups)) return mx_ffn_few_backward(f, K, dtype, activation, (hipStream_t)stream);
    return mx_backward128(f, n_groups ? MxRows : MxDense, dtype, activation, (hipStream_t)stream);
}
