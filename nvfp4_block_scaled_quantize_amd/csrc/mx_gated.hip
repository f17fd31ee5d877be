// mx_gated.hip -- the gated feed-forward block on MXFP4 products: the entry points, and a plain kernel.
//
// Forward: G and U are the products of A with the two halves of W, H = a(G) U.  Backward: dH is a
// product, dG and dU follow from it and the checkpoint's G and U.  Either way what is done to an
// element needs no other but those of its block of 32, which a lane pair holds, so it is done to the
// accumulators and nothing but the results goes to memory.
//
// The plain kernel: a wave computes 32 x 32 of H, or of dH, with its operands straight from memory.
#include "mx_ffn.h"

namespace nvfp4 {

// A fragment's 16 bytes for a lane: row `row` of an operand, K step s (of 64 elements).
__device__ __forceinline__ int4v plain_codes(const uint8_t* p, int64_t row, int64_t pitch, int64_t s, int h) {
    return *(const int4v*)(p + row * pitch + s * 32 + h * 16);
}

template <typename T, int ACT, bool BACK, bool GROUPS>
__global__ __launch_bounds__(256) void k_mx_gated(MxFfnArgs f, unsigned tiles_n, int64_t width) {
    const MxGArgs& g = f.g;
    const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 31, h = lane >> 5;
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    unsigned tm, tn;
    int64_t m0, rows;
    const uint8_t *bc = g.bc, *bs = g.bs;
    int64_t steps = g.kp / 64;
    bool none = false;
    if constexpr (GROUPS) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, 32, blockIdx.x, tiles_n, tm, tn, u)) return;
        m0 = u.row0, rows = u.rows, none = u.group == g.n_groups;
        if (none) steps = 0;
        else bc += u.group * (BACK ? 1 : 2) * g.N * pitch, bs += u.group * (BACK ? 1 : 2) * g.N * spitch;
    } else {
        mx_tile_of(blockIdx.x, (unsigned)((g.M + 31) / 32), tiles_n, tm, tn);
        m0 = (int64_t)tm * 32, rows = g.M - m0 < 32 ? g.M - m0 : 32;
    }
    const int64_t c0 = ((int64_t)tn * 4 + wid) * 32;
    if (c0 >= width) return;
    // rows and columns past the end repeat the last: their results are not stored
    const int64_t ra = m0 + (li < rows ? li : rows - 1), rb = c0 + li < g.N ? c0 + li : g.N - 1;
    float16v acc[BACK ? 1 : 2] = {};
    for (int64_t s = 0; s < steps; ++s) {
        const int4v a = plain_codes(g.ac, ra, pitch, s, h);
        const int sa = g.as[ra * spitch + s * 2 + h];
#pragma unroll
        for (int j = 0; j < (BACK ? 1 : 2); ++j) {
            const int64_t r = rb + j * g.N;
            acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_frag(plain_codes(bc, r, pitch, s, h)), mx_frag(a), acc[j],
                                                                     kE2M1, kE2M1, 0, bs[r * spitch + s * 2 + h], 0, sa);
        }
    }
    const bool in = li < rows;
    const int left = (int)(g.N - c0 < 32 ? g.N - c0 : 32);
    if constexpr (BACK) put_backward<T, ACT>(f, acc[0], m0 + li, in, c0, left, h, none);
    else put_forward<T, ACT>(f, acc[0], acc[1], m0 + li, in, c0, left, h);
}

template <typename T, int ACT, bool BACK>
static int launch_plain(const MxFfnArgs& f, hipStream_t st) {
    const MxGArgs& g = f.g;
    const int64_t width = f.qc || f.kc ? f.np : g.N, tn = (width + 127) / 128;
    // every group, and the rows in none, may end in a partial unit
    const int64_t units = g.offsets ? g.M / 32 + (g.n_groups < g.M ? g.n_groups : g.M) + 1 : (g.M + 31) / 32;
    if (!mx_grid_fits((__int128)units * tn, 256)) return NVFP4_ERR_SHAPE;
    const auto kernel = g.offsets ? k_mx_gated<T, ACT, BACK, true> : k_mx_gated<T, ACT, BACK, false>;
    kernel<<<dim3((unsigned)(units * tn)), 256, 0, st>>>(f, (unsigned)tn, width);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <bool BACK>
static int launch_any(const MxFfnArgs& f, int dtype, int act, hipStream_t st) {
    if (act == MXFP4_SILU)
        return dtype == NVFP4_BF16 ? launch_plain<uint16_t, MXFP4_SILU, BACK>(f, st) : launch_plain<float, MXFP4_SILU, BACK>(f, st);
    return dtype == NVFP4_BF16 ? launch_plain<uint16_t, MXFP4_GELU, BACK>(f, st) : launch_plain<float, MXFP4_GELU, BACK>(f, st);
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
    return launch_any<false>(f, h ? h_dtype : NVFP4_F32, activation, (hipStream_t)stream);
}

static size_t linear_code_bytes(int64_t M, int64_t K) {
    return ((size_t)(M * (mx_pad(K) / 2)) + 255) / 256 * 256;
}

extern "C" size_t mxfp4_gated_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups) {
    if (!ffn_extents(M, N, K)) return 0;        // mxfp4_gated_linear refuses them
    return M > 0 && K > 0 ? linear_code_bytes(M, K) + (size_t)(M * (mx_pad(K) / 32)) : 0;
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
    return launch_any<true>(f, dtype, activation, (hipStream_t)stream);
}
