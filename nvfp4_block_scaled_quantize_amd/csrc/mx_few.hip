// mx_few.hip -- MXFP4 products with few rows of A: the forward for single tokens and small
// batches, dense or grouped by expert, with A packed or quantized on the way.
//
// C[m][n] = Q(x_m) . w_n is bound by reading W once (17/32 byte per element).  A workgroup takes
// 16 rows and NT columns of C; each of its waves takes 16 of the columns and a part of K.  W's
// fragments come straight from memory into registers, a batch of K steps ahead (a load covers 16
// rows x 64 contiguous bytes); the rows of A are put into LDS once per workgroup, quantized
// there from x while the first of W is on its way; the waves' partial sums meet in LDS at the
// end, in wave order.  v_mfma_scale_f32_16x16x128: lane l holds row l mod 16 and the 32 elements
// of K at 32 (l / 16), with their scale byte.
//
// Measured (GPU time per call in a replayed graph, three sets of operands in turn): 1 x 6144 x
// 4096, x in bfloat16, 5.7 us (W alone at the card's copy rate: 2.8 us, an empty kernel: about
// 2.4 us) against 8.4 us as quantize and packed product; 16 rows 9.5 us, packed, the quantize
// included, against 13.7 us by tiles; 24 rows over 17 groups (4096 x 2048, 71 MB of W) 15.3 us.
#include "mx_common.h"

#include <atomic>

namespace nvfp4 {

constexpr int kFewRows = 16;
constexpr int kFewBatch = 4;                 // K steps of 128 in one batch of loads (of scales: 16 bytes)
// LDS row strides of A: 64 and 4 bytes past the row, so that 16 rows' reads spread over the banks
__host__ __device__ constexpr int few_code_stride(int kp) { return kp / 2 + 64; }
__host__ __device__ constexpr int few_scale_stride(int kp) { return kp / 32 + 4; }
inline int64_t few_lds(int64_t kp, int64_t rows, int waves) {
    const int64_t a = rows * (kp / 2 + 64 + kp / 32 + 4), sums = waves * 16 * 17 * 4;
    return a > sums ? a : sums;
}

// XT: uint8_t (A packed), uint16_t or float (x).
template <typename T, typename XT, int MODE, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_mx_few(MxFArgs f, unsigned tiles_n) {
    constexpr int kThreads = 64 * WAVES;
    constexpr int kSubs = NT / 16, kSplit = WAVES / kSubs;      // the waves' columns and K parts
    const MxGArgs& g = f.g;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63, wid = __builtin_amdgcn_readfirstlane(t >> 6);
    const int li = lane & 15, q = lane >> 4, sub = wid % kSubs, part = wid / kSubs;
    unsigned tn, tu;
    int64_t m0 = 0;
    int rows = (int)g.M, steps = (int)(g.kp / 128);
    const int64_t pitch = g.kp / 2, spitch = g.kp / 32;
    const uint8_t *bc = g.bc, *bs = g.bs;
    if constexpr (MODE == MxRows) {
        MxUnit u;
        if (!mx_find_tile(g.offsets, g.n_groups, (int)g.M, kFewRows, blockIdx.x, tiles_n, tu, tn, u)) return;
        m0 = u.row0, rows = (int)u.rows;
        if (u.group == g.n_groups) steps = 0;
        else bc += u.group * g.N * pitch, bs += u.group * g.N * spitch;
    } else {
        tn = blockIdx.x;
    }
    const int64_t n0 = (int64_t)tn * NT + sub * 16, n = n0 + li < g.N ? n0 + li : g.N - 1;
    const uint8_t* wc = bc + n * pitch + q * 16;
    const uint8_t* ws = bs + n * spitch;
    const int s0 = steps * part / kSplit, s1 = steps * (part + 1) / kSplit;

    // A load of 16 rows costs the address unit as much for 4 bytes a row as for 64, so a batch's
    // scales come in one, unless that would reach past the row's end.
    struct Batch {
        int4v w[kFewBatch];
        int s[kFewBatch];
    };
    const auto load = [&](Batch& b, int s) {
#pragma unroll
        for (int i = 0; i < kFewBatch; ++i)
            if (s + i < s1) b.w[i] = *(const int4v*)(wc + (int64_t)(s + i) * 64);
        if (s + kFewBatch <= steps) {
            const int4v v = *(const int4_by4*)(ws + (int64_t)s * 4);
#pragma unroll
            for (int i = 0; i < kFewBatch; ++i) b.s[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < kFewBatch; ++i)
                if (s + i < s1) b.s[i] = *(const int*)(ws + (int64_t)(s + i) * 4);
        }
    };
    // The first of x is asked for before W: loads return in order, and x has to be quantized
    // while W is on its way.  A lane takes eight elements, a quad a block.
    const int per = (int)(g.kp / 8), octs = steps ? rows * per : 0;
    const auto load_x = [&](int i) -> Oct<XT> {
        const int r = i / per, k = (i - r * per) * 8;
        if constexpr (sizeof(XT) > 1) return load_oct((const XT*)f.x + (m0 + r) * f.ldx + k, i < octs ? f.K - k : 0);
    };
    constexpr int kAhead = 4;
    [[maybe_unused]] Oct<XT> o[kAhead];
    if constexpr (sizeof(XT) > 1) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j * kThreads < octs) o[j] = load_x(t + j * kThreads);
    }
    Batch cur = {};
    if (s0 < s1) load(cur, s0);

    // A's rows into LDS
    uint8_t* ac = lds;
    const int cstride = few_code_stride((int)g.kp), sstride = few_scale_stride((int)g.kp);
    uint8_t* as = lds + rows * cstride;
    if constexpr (sizeof(XT) == 1) {
        const int n = (int)(pitch / 16), sn = (int)(spitch / 4);
        for (int r = wid; r < (steps ? rows : 0); r += WAVES) {
            for (int i = lane; i < n; i += 64)
                *(uint4*)(ac + r * cstride + i * 16) = *(const uint4*)(g.ac + (m0 + r) * pitch + i * 16);
            for (int i = lane; i < sn; i += 64)
                *(uint32_t*)(as + r * sstride + i * 4) = *(const uint32_t*)(g.as + (m0 + r) * spitch + i * 4);
        }
    } else {
        const auto put_x = [&](int i, const Oct<XT>& x) {
            const int r = i / per, k = (i - r * per) * 8;
            const uint32_t code = mx_scale_code(quad_max(max_bits(x)), f.above);
            const uint32_t w = codes_rne(x, mx_scale_value(code));
            if (i >= octs) return;
            *(uint32_t*)(ac + r * cstride + k / 2) = code == 255u ? 0u : w;
            if ((t & 3) == 0) as[r * sstride + k / 32] = (uint8_t)code;
        };
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j * kThreads < octs) put_x(t + j * kThreads, o[j]);
        for (int i = t + kAhead * kThreads; i - t < octs; i += kThreads) put_x(i, load_x(i));
    }
    __syncthreads();

    float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t* pa = ac + li * cstride + q * 16;
    const uint8_t* ps = as + li * sstride + q;
    for (int s = s0; s < s1; s += kFewBatch) {
        Batch next;
        if (s + kFewBatch < s1) load(next, s + kFewBatch);
#pragma unroll
        for (int i = 0; i < kFewBatch; ++i) {
            if (s + i >= s1) break;
            int4v a = {0, 0, 0, 0};
            int sa = 0;
            if (li < rows) {
                a = *(const int4v*)(pa + (s + i) * 64);
                sa = ps[(s + i) * 4];
            }
            acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_frag(cur.w[i]), mx_frag(a), acc, kE2M1,
                                                                   kE2M1, 0, cur.s[i] >> (8 * q), 0, sa);
        }
        cur = next;
    }
    __syncthreads();        // A's rows are done with: their LDS takes the partial sums

    // register i of lane l: column 4 (l / 16) + i, row l mod 16
    float* sums = (float*)lds;
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[(wid * 16 + li) * 17 + 4 * q + i] = acc[i];
    __syncthreads();
    for (int i = t; i < 16 * NT; i += kThreads) {
        const int row = i / NT, col = i % NT;
        const float* p = sums + ((col >> 4) * 16 + row) * 17 + (col & 15);
        float v = p[0];
#pragma unroll
        for (int w = 1; w < kSplit; ++w) v += p[w * kSubs * 16 * 17];
        const int64_t c = (int64_t)tn * NT + col;
        if (row < rows && c < g.N) store_c((T*)g.c + (m0 + row) * g.ldc + c, v);
    }
}

template <typename T, typename XT, int MODE, int NT, int WAVES>
static int launch(const MxFArgs& f, int64_t units, hipStream_t st) {
    const int64_t tn = (f.g.N + NT - 1) / NT;
    if (!mx_grid_fits(units * tn, 64 * WAVES)) return NVFP4_ERR_SHAPE;
    const int lds = (int)few_lds(f.g.kp, f.g.M < kFewRows ? f.g.M : kFewRows, WAVES);
    const auto kernel = k_mx_few<T, XT, MODE, NT, WAVES>;
    static std::atomic<uint64_t> ready{0};
    if (lds > 64 * 1024)
        if (int rc = mx_allow_lds((const void*)kernel, kMxMaxLds, ready)) return rc;
    kernel<<<dim3((unsigned)(units * tn)), 64 * WAVES, lds, st>>>(f, (unsigned)tn);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

// Dense: 16 columns a workgroup.  Eight waves halve a wave's K (1 x 1024 x 8192 5.3 against 6.4
// us, 16 x 6144 x 4096 9.5 against 11.3), but with more than about 448 workgroups four are enough
// and start sooner (1 x 16384 x 2048 5.8 against 6.2 us, 4 x 9216 x 2048 5.5 either way).
template <typename T, typename XT>
static int launch_dense(const MxFArgs& f, hipStream_t st) {
    if ((f.g.N + 15) / 16 > 448) return launch<T, XT, MxDense, 16, 4>(f, 1, st);
    return launch<T, XT, MxDense, 16, 8>(f, 1, st);
}

// Grouped: four waves on 32 columns, two of them sharing K (24 rows over 17 groups, 4096 x 2048:
// 15.2 us against 17.1 with 16 columns and 16.8 with 64, which need no split), or on 16 where that
// leaves compute units without work (4 rows over 4 groups, 1024 x 2048: 3.8 us against 4.6).
template <typename T, typename XT>
static int launch_rows(const MxFArgs& f, hipStream_t st) {
    // every group, and the rows in none, may end in a partial unit
    const int64_t units = f.g.M / kFewRows + (f.g.n_groups < f.g.M ? f.g.n_groups : f.g.M) + 1;
    if (units * ((f.g.N + 31) / 32) < 256) return launch<T, XT, MxRows, 16, 4>(f, units, st);
    return launch<T, XT, MxRows, 32, 4>(f, units, st);
}

bool mx_few_fits(int64_t M, int64_t kp) {
    return few_lds(kp, M < kFewRows ? M : kFewRows, 8) <= kMxMaxLds;
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
