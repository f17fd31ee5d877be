// mx_few.hip -- the plain products with few rows or few tiles (kernel: mx_few.h).
#include "mx_few.h"

namespace nvfp4 {
using namespace few;

// The tile of a dense product (counts of workgroups: for an MI355X's 256 compute units).  Up to 16
// rows: 16 columns a workgroup.  Eight waves halve a wave's K (1 x 1024 x 8192 4.6 against 5.0 us,
// 16 x 6144 x 4096 6.1 against 6.3), but with more than about 448 workgroups four are enough and
// start sooner (1 x 16384 x 2048 5.3 against 6.5 us, 4 x 9216 x 2048 4.9 against 5.2).  More rows:
// the smallest tile that leaves no compute unit two workgroups, or else 32 x 32.  Packed, 32 x 1024
// x 4096: 16 x 16 4.0 us, 32 x 16 4.5; 128 x 1024 x 4096: 5.5, 4.7, 32 x 32 5.7; 64 x 6144 x 4096:
// 13.0, 9.4, 9.1.
struct FewTile {
    int blocks, cols;
    int64_t units, workgroups;
};
static FewTile few_tile(int64_t M, int64_t N) {
    const int64_t units = (M + 15) / 16, pairs = (M + 31) / 32, tn = (N + 15) / 16;
    if (units == 1 || units * tn <= 256) return {1, 16, units, units * tn};
    if (pairs * tn <= 256) return {2, 16, pairs, pairs * tn};
    return {2, 32, pairs, pairs * ((N + 31) / 32)};
}
template <typename T, typename XT>
static int launch_dense(const MxFArgs& f, hipStream_t st) {
    const FewTile t = few_tile(f.g.M, f.g.N);
    if (t.cols == 32) return launch<T, XT, MxDense, 32, 8, 2>(f, t.units, st);
    if (t.blocks == 2) return launch<T, XT, MxDense, 16, 8, 2>(f, t.units, st);
    if (t.workgroups > 448) return launch<T, XT, MxDense, 16, 4>(f, t.units, st);
    return launch<T, XT, MxDense, 16, 8>(f, t.units, st);
}

template <typename T, typename XT>
static int launch_rows(const MxFArgs& f, hipStream_t st) {
    const RowsTile t = rows_tile(f.g.M, f.g.N, f.g.kp, f.g.n_groups);
    if (t.cols == 64) return launch<T, XT, MxRows, 64, 4, 2>(f, t.units, st);
    if (t.cols == 16) return launch<T, XT, MxRows, 16, 4>(f, t.units, st);
    return launch<T, XT, MxRows, 32, 4>(f, t.units, st);
}

bool mx_few_rows(int64_t M, int64_t N, int64_t kp, int64_t n_groups) {
    return few_fits(kp, M, 1) && few_launches(rows_tile(M, N, kp, n_groups).workgroups);
}
bool mx_few_two_fit(int64_t M, int64_t kp) { return few_fits(kp, M, 2); }

bool mx_few_dense(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile(M, N);
    return (M <= 16 || t.workgroups <= 512) && few_fits(kp, M, t.blocks) && few_launches(t.workgroups);
}

int64_t mx_few_quantized(int64_t M, int64_t N, int64_t kp) {
    const FewTile t = few_tile(M, N);
    const int64_t rows = M < kFewRows * t.blocks ? M : kFewRows * t.blocks;
    return rows * kp * (t.workgroups > 256 ? t.workgroups : 256) / 256;
}

template <typename XT>
static int launch_x(const MxFArgs& f, int c_dtype, hipStream_t st) {
    if (f.g.n_groups) return c_dtype == NVFP4_BF16 ? launch_rows<uint16_t, XT>(f, st) : launch_rows<float, XT>(f, st);
    return c_dtype == NVFP4_BF16 ? launch_dense<uint16_t, XT>(f, st) : launch_dense<float, XT>(f, st);
}

int mx_few_packed(const MxFArgs& f, int c_dtype, hipStream_t st) { return launch_x<uint8_t>(f, c_dtype, st); }

int mx_few_linear(const MxFArgs& f, int x_dtype, int c_dtype, hipStream_t st) {
    return x_dtype == NVFP4_BF16 ? launch_x<uint16_t>(f, c_dtype, st) : launch_x<float>(f, c_dtype, st);
}

}  // namespace nvfp4
