// mx_ffn_few.hip -- the gated feed-forward block with few rows or few tiles (kernel: mx_few.h).
#include "mx_few.h"

namespace nvfp4 {

template <int KIND, typename XT, int MODE, int NT, int WAVES, int BLOCKS = 1>
static int launch(const few::FfnArgs& a, int64_t units, hipStream_t st) {
    return few::launch<float, XT, MODE, NT, WAVES, BLOCKS, KIND>(a, units, st);
}

// The tile of a dense product.  Up to 16 rows: eight columns of H a workgroup, the work of 16 columns of a plain
// product (1 x 9216 x 4096 9.2 us; with 16 columns 10.7, with 32 12.5), with four waves from 448 workgroups
// on (1 x 16384 x 2048 8.1 us against 10.8 with eight; 1 x 4096 x 2048, 512 of them, 4.3 against 4.8; but 16 x 1024 x
// 8192, 128, 7.8 against 6.6).  (Eight columns' operands lie N rows apart in one buffer, which has to be below 2^31
// bytes; else 16.)  More rows, and the backward: the tiles of the plain products (mx_few.hip).
struct FewTile {
    int blocks, cols;
    int64_t units, workgroups;
};
template <int KIND>
static FewTile few_tile(int64_t M, int64_t N, int64_t kp) {
    const int64_t units = (M + 15) / 16, pairs = (M + 31) / 32, tn = (N + 15) / 16;
    if (KIND == kForward && units == 1 && 2 * N * (kp / 2) < 0x7FFFFFE0 - (1 << 22)) return {1, 8, 1, (N + 7) / 8};
    if (units == 1 || units * tn <= 256) return {1, 16, units, units * tn};
    if (pairs * tn <= 256) return {2, 16, pairs, pairs * tn};
    return {2, 32, pairs, pairs * ((N + 31) / 32)};
}
template <int KIND, typename XT>
static int launch_dense(const few::FfnArgs& a, hipStream_t st) {
    const FewTile t = few_tile<KIND>(a.f.g.M, a.f.g.N, a.f.g.kp);
    if (t.cols == 32) return launch<KIND, XT, MxDense, 32, 8, 2>(a, t.units, st);
    if (t.blocks == 2) return launch<KIND, XT, MxDense, 16, 8, 2>(a, t.units, st);
    if constexpr (KIND == kForward)
        if (t.cols == 8) return t.workgroups > 448 ? launch<KIND, XT, MxDense, 8, 4>(a, t.units, st) : launch<KIND, XT, MxDense, 8, 8>(a, t.units, st);
    if (t.workgroups > 448) return launch<KIND, XT, MxDense, 16, 4>(a, t.units, st);
    return launch<KIND, XT, MxDense, 16, 8>(a, t.units, st);
}
template <int KIND, typename XT>
static int launch_rows(const few::FfnArgs& a, hipStream_t st) {
    const MxGArgs& g = a.f.g;
    const few::RowsTile t = few::rows_tile(g.M, g.N, g.kp, g.n_groups);
    if (t.cols == 64) return launch<KIND, XT, MxRows, 64, 4, 2>(a, t.units, st);
    if (t.cols == 16) return launch<KIND, XT, MxRows, 16, 4>(a, t.units, st);
    return launch<KIND, XT, MxRows, 32, 4>(a, t.units, st);
}
template <int KIND, typename XT>
static int launch_x(const few::FfnArgs& a, hipStream_t st) {
    return a.f.g.n_groups ? launch_rows<KIND, XT>(a, st) : launch_dense<KIND, XT>(a, st);
}

int mx_ffn_few(const MxFArgs& f, int x_dtype, int dtype, int act, hipStream_t st) {
    const few::FfnArgs a = {f, act, dtype == NVFP4_BF16, {}};
    if (!f.x) return launch_x<kForward, uint8_t>(a, st);
    return x_dtype == NVFP4_BF16 ? launch_x<kForward, uint16_t>(a, st) : launch_x<kForward, float>(a, st);
}

int mx_ffn_few_backward(const MxFfnArgs& f, int64_t K, int dtype, int act, hipStream_t st) {
    const few::FfnArgs a = {{f.g, nullptr, 0, K, 0}, act, dtype == NVFP4_BF16, {f.kc, f.ks, f.np, f.h, f.ldh}};
    return launch_x<kBackward, uint8_t>(a, st);
}

bool mx_ffn_few_dense(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile<kForward>(M, N, kp);
    return (M <= 16 || t.workgroups <= 256) && few::few_fits(kp, M, t.blocks) && few::few_launches(t.workgroups);
}

int64_t mx_ffn_few_quantized(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile<kForward>(M, N, kp);
    const int64_t rows = M < 16 * t.blocks ? M : 16 * t.blocks;
    return rows * kp * (t.workgroups > 256 ? t.workgroups : 256) / 256;
}

}  // namespace nvfp4
