/*
 * mxfp4.h -- C ABI of the microscaled 4-bit (MXFP4) operators: quantization, the products
 * of quantized operands, and the same products grouped by expert.  Part of libnvfp4.so.
 *
 * Format (OCP Microscaling Formats v1.0, MXFP4): E2M1 elements, one E8M0 scale per block of
 * 32 along a copy's rows, no tensor scale: x_hat = x_E2M1 * 2^(code - 127).  Unlike NVFP4's
 * E4M3 scales per 16 elements, this is the operand format of gfx950's block-scaled matrix
 * instructions, and quantizing it needs no pass for a tensor maximum.
 *
 * Conventions are those of nvfp4.h (device pointers, streams, statuses, argument errors
 * returned before anything is enqueued; no allocation, no synchronisation).  The calls hold
 * no state at all: any number of them may run at once on distinct buffers.
 *
 * Layout of one copy: an n x k matrix quantized along its rows, with kp = k rounded up to a
 * multiple of 128 (mxfp4_padded_k), has
 *   codes  uint8 [n][kp/2]   element 2i in the low nibble, 2i+1 in the high nibble; a nibble
 *                            is sign<<3 | exponent<<1 | mantissa; 16-byte aligned
 *   scales uint8 [n][kp/32]  E8M0 codes; 0..254 stand for 2^(code-127), 255 for NaN; 4-byte
 *                            aligned
 * Elements past k are zero codes; blocks wholly past k have scale code 0.  The rowwise copy
 * of an R x C matrix X is X quantized along its rows (n = R, k = C); the columnwise copy is
 * X^T quantized along its rows (n = C, k = R).  Extents may be any size, row pitches any
 * pitch of at least a row, and inputs need only their element's alignment.  Only sizes far
 * past a device's memory, or made almost wholly of padding, are refused (NVFP4_ERR_SHAPE): an
 * extent above 2^34 - 2^13, a C of more than 2^40 elements, a launch of 2^32 threads or more
 * (such as 2^30 rows of one column).
 *
 * Groups.  `offsets` is a device array of n_groups + 1 int32: group g holds the rows
 * [offsets[g], offsets[g+1]) of a matrix (an expert's tokens).  offsets[0] is read as 0;
 * entries are clamped to [0, rows] and to be non-decreasing, so that no value makes a kernel
 * leave its buffers.  A group may be empty.  Rows from the last offset on belong to no group.
 * A grouped columnwise copy restarts its blocks at each group: group g's rows start at k
 * position P_g = the sum over earlier groups of their row counts rounded up to 128, and the
 * copy's pitch is kp = mxfp4_grouped_k(rows, n_groups), which suffices for any offsets;
 * positions past the last group are not written, and never read.
 */
#ifndef MXFP4_H
#define MXFP4_H
#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MXFP4_ABI_VERSION 1

/* Scale of a block whose largest magnitude is amax > 0:
 *   FLOOR  2^(floor(log2 amax) - 2): the OCP rule; magnitudes above 6 scales saturate
 *   CEIL   the smallest power of two s with amax <= 6 s: nothing saturates, so that
 *          stochastic rounding is unbiased
 * at least 2^-127 either way, and 2^-127 when amax = 0.  A block that holds an infinity or
 * a NaN gets scale code 255 and zero codes: it decodes to, and multiplies as, NaN. */
enum mxfp4_scale_rule { MXFP4_SCALE_FLOOR = 0, MXFP4_SCALE_CEIL = 1 };

/* Options of one mxfp4_quantize call.
 *   rowwise, colwise   produce the rowwise and/or the columnwise copy (at least one)
 *   scale_rule         enum mxfp4_scale_rule
 *   round_row/col      NVFP4_RNE (to nearest even, saturating at 6) or NVFP4_SR: with u the
 *                      scaled magnitude and f its position between its two grid neighbours,
 *                      up iff floor(f 2^16) + r >= 2^16 with 16 Philox bits r per element
 *   seed               key of the Philox4x32-10 generator; element (i, j) of copy c (0
 *                      rowwise, 1 columnwise) at e = i kp + j takes half (e mod 2) of word
 *                      ((e/2) mod 4) of the block with counter (lo32(e/8), hi32(e/8), c,
 *                      0x4D585352) */
typedef struct {
    int32_t rowwise, colwise;
    int32_t scale_rule;
    int32_t round_row, round_col;
    uint64_t seed;
} mxfp4_quant_params;

/* One copy (pointers to device memory; see the layout above). */
typedef struct {
    uint8_t* codes;
    uint8_t* scales;
} mxfp4_tensor;

/* k rounded up to a multiple of 128: the K extent of a copy's rows. */
int64_t mxfp4_padded_k(int64_t k);
/* K extent of a grouped columnwise copy of `rows` rows in n_groups groups: the largest sum of
 * the groups' row counts rounded up to 128 that any offsets can give. */
int64_t mxfp4_grouped_k(int64_t rows, int64_t n_groups);

/* Quantize `batch` matrices X[rows][cols] (bf16 or f32 per `dtype`; row pitch ld_x >= cols,
 * batch_stride elements from one matrix to the next, ignored for batch 1), both copies from
 * one read.
 *   row_out  rowwise copies [batch][rows][...]; may be NULL when p->rowwise == 0
 *   col_out  columnwise copies [batch][cols][...]; may be NULL when p->colwise == 0
 *   offsets  NULL (n_groups 0), or the groups of X's rows, with batch == 1: the columnwise
 *            copy is then the grouped one; the rowwise copy covers all rows either way */
int mxfp4_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols,
                   int64_t ld_x, int64_t batch_stride, const int32_t* offsets, int64_t n_groups,
                   const mxfp4_quant_params* p, const mxfp4_tensor* row_out,
                   const mxfp4_tensor* col_out, void* stream);

/* Decode one copy: out[n][k] (f32 or bf16 per out_dtype, row pitch ld_out >= k) gets the
 * values the codes stand for, exact in f32 and, for a copy made of bf16 values, in bf16; but
 * 2^128 and more, to which CEIL can round magnitudes above 1.5 * 2^127, become infinite.  For
 * a grouped columnwise copy pass its offsets and k = the number of rows; positions of rows in
 * no group get 0. */
int mxfp4_dequantize(const mxfp4_tensor* q, int64_t n, int64_t k, const int32_t* offsets,
                     int64_t n_groups, int out_dtype, void* out, int64_t ld_out, void* stream);

/* C[M][N] = A B^T over two copies (A: M x K, B: N x K), FP32 accumulation, each element
 * rounded once to c_dtype (f32 or bf16), row pitch ldc >= N.  Products of elements are exact
 * and block scales are powers of two; the only rounding is the accumulation, whose accuracy
 * assumes the products of scales to be normal binary32 (smaller ones may flush to 0).  The
 * three products of a linear layer Y = X W^T are this call: Y on the rowwise copies of X and
 * W, dX = dY W on dY's rowwise and W's columnwise copy (K = N), dW = dY^T X on the columnwise
 * copies (K = tokens).  K <= 2^23. */
int mxfp4_gemm(const mxfp4_tensor* a, const mxfp4_tensor* b, int64_t M, int64_t N, int64_t K,
               void* c, int c_dtype, int64_t ldc, void* stream);

/* The product grouped by expert: rows [offsets[g], offsets[g+1]) of C[M][N] are those rows
 * of A (M x K) times B_g^T, B holding n_groups matrices N x K one after the other.  Rows in
 * no group are set to 0.  Forward (B: rowwise copies of the experts' weights) and input
 * gradient (B: their columnwise copies). */
int mxfp4_gemm_grouped(const mxfp4_tensor* a, const mxfp4_tensor* b, const int32_t* offsets,
                       int64_t n_groups, int64_t M, int64_t N, int64_t K, void* c, int c_dtype,
                       int64_t ldc, void* stream);

/* The products over ragged K: C_g[M][N] = A_g B_g^T for g = 0 .. n_groups - 1, A_g and B_g the
 * spans of group g in two grouped columnwise copies (A: M x rows, B: N x rows, both made with
 * these offsets).  C is [n_groups][M][N] with row pitch ldc; an empty group's C_g is 0.  The
 * experts' weight gradients dW_g = dY_g^T X_g. */
int mxfp4_gemm_grouped_wgrad(const mxfp4_tensor* a, const mxfp4_tensor* b, const int32_t* offsets,
                             int64_t n_groups, int64_t M, int64_t N, int64_t rows, void* c,
                             int c_dtype, int64_t ldc, void* stream);

/* The forward of a layer in one call: C[M][N] = Q(X) W^T with X (bf16 or f32, M x K, row pitch
 * ld_x) quantized rowwise to nearest even by scale_rule, W a copy N x K; or, with offsets,
 * grouped as in mxfp4_gemm_grouped with W holding n_groups matrices.  The result is that of
 * mxfp4_quantize followed by the product, bit for bit.
 *   ws  device workspace of mxfp4_linear_workspace_bytes() bytes, 256-byte aligned (0 bytes,
 *       NULL allowed, for the few rows that are quantized inside the product's kernel, and for
 *       sizes that the call refuses) */
size_t mxfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups);
int mxfp4_linear(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x, int32_t scale_rule,
                 const mxfp4_tensor* w, int64_t N, const int32_t* offsets, int64_t n_groups,
                 void* c, int c_dtype, int64_t ldc, void* ws, size_t ws_bytes, void* stream);

/* MXFP4_ABI_VERSION of the loaded library. */
int mxfp4_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif
