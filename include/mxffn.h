/*
 * mxffn.h -- C ABI of the gated feed-forward block on MXFP4 products, forward and backward, and
 * of the 8-bit (MXFP8) activation checkpoints that its backward pass reads.  Part of libnvfp4.so.
 *
 * The block:  G = A Wg^T,  U = A Wu^T,  H = a(G) U (element by element),  Y = H W2^T.
 * Both projections, the activation a and the product are one kernel; G and U never reach memory,
 * but for the checkpoint that a training step asks for.  Its backward pass is one kernel too:
 * dH = dY W2, and with the checkpoint's values g and u
 *   dU = dH a(g),   dG = dH u a'(g),   H = a(g) u (for dW2 = dY^T H).
 * What remains of the backward pass are products of mxfp4.h: with [dG dU] as one matrix M x 2N and
 * W = [Wg; Wu] as one 2N x K, dX = [dG dU] W and dW = [dG dU]^T X are one product each.
 *
 * Format of a checkpoint (OCP Microscaling Formats v1.0, MXFP8 with E4M3 elements): one E8M0 scale
 * per block of 32 along the rows, x_hat = x_E4M3 * 2^(code - 127).  The scale is the smallest power of
 * two s >= 2^-127 with amax <= 448 s, so that nothing saturates; elements are rounded to nearest even.
 * A block that holds an infinity or a NaN gets scale code 255 and zero codes: it decodes to NaN.
 *
 * Conventions, offsets of groups and layouts are those of mxfp4.h, except that a code is a byte:
 * an n x k checkpoint has, with kp = mxfp4_padded_k(k),
 *   codes  uint8 [n][kp]     OCP E4M3 "fn"; 16-byte aligned
 *   scales uint8 [n][kp/32]  E8M0; 4-byte aligned
 * Elements past k are zero codes; blocks wholly past k have scale code 0.  (Codes 0x7F and 0xFF, which
 * no call here writes, decode to NaN.)
 */
#ifndef MXFFN_H
#define MXFFN_H
#include "mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MXFFN_ABI_VERSION 1

/* a(x):  SILU  x / (1 + e^-x)
 *        GELU  x (1 + tanh z) / 2,  z = sqrt(2 / pi) (x + 0.044715 x^3)  (the tanh form)
 * Both in binary32.  Where x is infinite, a(x) or a'(x) may be NaN. */
enum mxffn_activation { MXFP4_SILU = 0, MXFP4_GELU = 1 };

/* One checkpoint (pointers to device memory; see the layout above). */
typedef struct {
    uint8_t* codes;
    uint8_t* scales;
} mxfp8_tensor;

/* Checkpoint of `batch` matrices X[rows][cols] (bf16 or f32; row pitch ld_x >= cols, batch_stride
 * elements from one matrix to the next, ignored for batch 1): q is [batch][rows][...]. */
int mxfp8_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t ld_x,
                   int64_t batch_stride, const mxfp8_tensor* q, void* stream);

/* out[n][k] (f32 or bf16, row pitch ld_out >= k) gets a checkpoint's values: exact in f32, and in
 * bf16 but for values below 2^-126, which may be rounded (to nearest even), as 2^128 is to infinity. */
int mxfp8_dequantize(const mxfp8_tensor* q, int64_t n, int64_t k, int out_dtype, void* out,
                     int64_t ld_out, void* stream);

/* MXFP4 copies of a checkpoint's values, as mxfp4_quantize makes them of the matrices that
 * mxfp8_dequantize gives in bf16, bit for bit: the operands of the backward pass (the columnwise
 * copy that dW = dY^T X multiplies) from the input that the forward pass kept.  Arguments after q
 * as in mxfp4_quantize. */
int mxfp8_to_mxfp4(const mxfp8_tensor* q, int64_t batch, int64_t rows, int64_t cols,
                   const int32_t* offsets, int64_t n_groups, const mxfp4_quant_params* p,
                   const mxfp4_tensor* row_out, const mxfp4_tensor* col_out, void* stream);

/* H[M][N] = a(A Wg^T) (A Wu^T) from packed operands: A is M x K; w is 2N x K, the rows of Wg before
 * those of Wu.  With offsets, w holds n_groups such matrices one after the other and rows
 * [offsets[g], offsets[g+1]) of A go with matrix g; rows in no group give 0, checkpoint included.
 * At least one of three results, each computed from the FP32 sums:
 *   h           H in h_dtype (f32 or bf16), row pitch ldh >= N, rounded once; or NULL
 *   h_copy      the rowwise MXFP4 copy of H (M x N), rounded to nearest even by scale_rule from the
 *               FP32 values, not from bf16 ones: the operand of Y = H W2^T; or NULL
 *   checkpoint  G and U, as two M x N checkpoints one after the other ([2][M][...]); or NULL
 * Accuracy as mxfp4_gemm.  K <= 2^23. */
int mxfp4_gated(const mxfp4_tensor* a, const mxfp4_tensor* w, const int32_t* offsets, int64_t n_groups,
                int64_t M, int64_t N, int64_t K, int32_t activation, void* h, int h_dtype, int64_t ldh,
                int32_t scale_rule, const mxfp4_tensor* h_copy, const mxfp8_tensor* checkpoint,
                void* stream);

/* The same from activations in one call, for serving: X (bf16 or f32, M x K, row pitch ld_x) is
 * quantized rowwise to nearest even by scale_rule.  The result is that of mxfp4_quantize followed by
 * mxfp4_gated with h alone, bit for bit.
 *   ws  device workspace of mxfp4_gated_linear_workspace_bytes() bytes, 256-byte aligned (0 bytes,
 *       NULL allowed, for the few rows that are quantized inside the product's kernel, and for sizes
 *       that the call refuses) */
size_t mxfp4_gated_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t n_groups);
int mxfp4_gated_linear(const void* x, int dtype, int64_t M, int64_t K, int64_t ld_x, int32_t scale_rule,
                       const mxfp4_tensor* w, int64_t N, const int32_t* offsets, int64_t n_groups,
                       int32_t activation, void* h, int h_dtype, int64_t ldh, void* ws, size_t ws_bytes,
                       void* stream);

/* The backward pass through down projection, product and activation: dH[M][N] = dY W2 from packed
 * operands (dy: dY's rowwise copy, M x K; w: W2's columnwise copy, N x K, or n_groups of them with
 * offsets, K the width of Y), and from it and the checkpoint ([2][M][...], as mxfp4_gated writes it)
 *   dgu  [M][2N], row pitch ld >= 2N: dG in columns 0 .. N-1, dU in columns N .. 2N-1
 *   h    H = a(g) u, [M][N], row pitch ldh >= N; or NULL
 * in `dtype` (f32 or bf16), each rounded once; dH itself is not rounded.  Rows in no group give 0. */
int mxfp4_gated_backward(const mxfp4_tensor* dy, const mxfp4_tensor* w, const int32_t* offsets,
                         int64_t n_groups, int64_t M, int64_t N, int64_t K, int32_t activation,
                         const mxfp8_tensor* checkpoint, void* dgu, int dtype, int64_t ld, void* h,
                         int64_t ldh, void* stream);

/* The same from dH (dh_dtype, M x N, row pitch ld_dh >= N), whatever product made it. */
int mxfp8_gated_backward(const void* dh, int dh_dtype, int64_t ld_dh, int64_t M, int64_t N,
                         int32_t activation, const mxfp8_tensor* checkpoint, void* dgu, int dtype,
                         int64_t ld, void* h, int64_t ldh, void* stream);

/* MXFFN_ABI_VERSION of the loaded library. */
int mxffn_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif
