/*
 * libgemm, microscaled operands -- block-scaled 4- and 8-bit matrices for a
 * linear layer's forward and backward products on MI355X (gfx950).
 *
 * The format (OCP Microscaling Formats, v1.0)
 * -------------------------------------------
 * A coded matrix has `rows` rows of `cols` values, held in blocks of 32
 * consecutive columns.  The last block of a row is filled up with zeros, so
 * that a row is nb = ceil(cols / 32) whole blocks.  Block j of row i has
 *   - one scale byte s = scales[i*lds + j]: E8M0, the factor 2^(s - 127);
 *     255 is NaN (every value of the block is NaN);
 *   - 32 element codes:
 *       GEMM_MX_E2M1  4 bits (values 0, .5, 1, 1.5, 2, 3, 4, 6 and their
 *                     negatives), 16 bytes at codes[i*ldq + 16j], element c
 *                     in byte c/2, the even element in the low half;
 *       GEMM_MX_E4M3  one OCP FP8 E4M3 byte each, 32 bytes at
 *                     codes[i*ldq + 32j].
 * A value is its element times its block's factor.
 *
 * Conventions
 * -----------
 * Those of gemm.h: row-major device memory owned by the caller, leading
 * dimensions in elements (codes and scales: in bytes), calls enqueue on
 * `stream` and return, argument errors are found on the host before any
 * launch, gemm_last_error() has the reason.  Codes are 16-byte aligned with
 * ldq a multiple of 16 (else UNSUPPORTED); everything else may have any
 * alignment.  Sizes are up to 2^31-1.  Results are bit-reproducible: no
 * sum's order depends on timing.  Elements that a call does not describe
 * (columns past `cols`, bytes past a row's blocks) are never written.
 * Errors:
 *   a size < 0 or > 2^31-1, a leading dimension below its row's length, a
 *   NULL operand, an unknown format or type               -> INVALID_ARG
 *   codes not 16-byte aligned or ldq % 16 != 0            -> UNSUPPORTED
 *   an output overlapping an input                        -> ALIAS
 *   launch failure                                        -> HIP
 */
#ifndef DENSE_GEMM_ROW_AMD_GEMM_MX_H
#define DENSE_GEMM_ROW_AMD_GEMM_MX_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm_mx_format {
    GEMM_MX_E2M1 = 0, /* 4-bit elements (MXFP4) */
    GEMM_MX_E4M3 = 1  /* 8-bit elements (MXFP8) */
} gemm_mx_format_t;

/*
 * Quantisation of the rows x cols matrix X of type dtype (GEMM_DTYPE_F32,
 * _F16 or _BF16).  trans = 0: codes are rows x cols, blocks along X's rows.
 * trans = 1: codes are those of X^T (cols x rows), blocks down X's columns:
 * the layout in which a product sums over X's rows.
 *
 * With amax the largest magnitude of a block, its factor 2^e has
 *   E2M1  e = floor(log2(amax)) - 2: the OCP conversion.  Magnitudes above
 *         6 * 2^e saturate at it.
 *   E4M3  the smallest e with amax <= 448 * 2^e, so that nothing saturates
 *         and every value is within 2^-4 of itself (or half a step of the
 *         block's smallest, 2^(e-10)).
 * (e clamped to [-127, 127]; -127 for a block of zeros), and each element is
 * x / 2^e rounded to the nearest code, ties to even.  A block that holds an
 * infinity or NaN gets scale 255 and zero codes.  The zeros that fill up
 * the last block are written.
 */
gemm_status_t gemm_mx_quantize(int32_t dtype, int32_t format, int32_t trans,
                               int64_t rows, int64_t cols, const void *X, int64_t ldx,
                               uint8_t *codes, int64_t ldq, uint8_t *scales, int64_t lds,
                               void *stream);

/*
 * The values of a coded matrix, as the rows x cols matrix X of type dtype
 * (F32, F16, BF16): trans = 0 from codes that are rows x cols, trans = 1
 * from codes of X^T (cols x rows).  Rounded to nearest even where the type
 * cannot hold a value exactly (F16 out of its range gives infinities).
 */
gemm_status_t gemm_mx_dequantize(int32_t dtype, int32_t format, int32_t trans,
                                 int64_t rows, int64_t cols,
                                 const uint8_t *codes, int64_t ldq,
                                 const uint8_t *scales, int64_t lds,
                                 void *X, int64_t ldx, void *stream);

/*
 * Product of two E2M1 matrices: C = act(alpha * (A x Bt^T) + beta * C +
 * bias), A coded M x K, Bt coded N x K (both blocks along k; a row-major
 * K x N weight matrix is coded with trans = 1), C of type c_dtype (F32, F16,
 * BF16), accumulated in FP32 on the block-scaled matrix instruction and
 * rounded once.  epi NULL: C = A x Bt^T (C is not read); otherwise as
 * gemm_*_epi (beta == 0: C is not read; bias overlapping C -> ALIAS).
 * K == 0: the empty sum.
 *
 * Speed: the fast kernels take scales (A's and Bt's) that are 4-byte aligned
 * with rows of a multiple of 4 bytes, best of 16; the bytes behind a row's
 * blocks may be anything.  Other scales, code rows 2^23 - 2^12 bytes apart or
 * more (16 rows or fewer: 2^26) and rows of C 2^21 - 2^10 elements apart or
 * more take a general kernel (8192 x 8192 x 8160 with rows of 255 scales: 1190 us
 * against 296 with rows of 256).
 * 16-byte groups of X's rows and words of scales are read whole where one of
 * their values is in the matrix; what lies behind the matrix is not used.
 */
gemm_status_t gemm_mx_matmul(int32_t c_dtype, int64_t M, int64_t N, int64_t K,
                             const uint8_t *A, int64_t lda, const uint8_t *As, int64_t ldas,
                             const uint8_t *Bt, int64_t ldbt, const uint8_t *Bs, int64_t ldbs,
                             void *C, int64_t ldc, void *stream, const gemm_epilogue_t *epi);

/*
 * The same product with A = X quantised to E2M1 on the way (X is M x K of
 * type a_dtype: F32, F16, BF16): the sums that gemm_mx_quantize and
 * gemm_mx_matmul give one after the other, and bit for bit the same where
 * both ways take the same kernel (X and all scales laid out as the fast
 * kernels take them); another kernel adds in another order.  Up to 16 rows, a decoding step's, are encoded
 * inside the product, in one launch, if X's rows are 16-byte aligned, Bt's
 * scale rows 4-byte aligned, every row stride below 2^26 bytes and N at most
 * 2^26 - 16; `workspace` may be NULL then.  Otherwise the codes go through it
 * (gemm_mx_matmul_values_workspace_bytes bytes, 16-byte aligned, not
 * overlapping the operands; too small a one -> INVALID_ARG).
 */
gemm_status_t gemm_mx_matmul_values(int32_t a_dtype, int32_t c_dtype, int64_t M, int64_t N, int64_t K,
                                    const void *X, int64_t ldx,
                                    const uint8_t *Bt, int64_t ldbt, const uint8_t *Bs, int64_t ldbs,
                                    void *C, int64_t ldc, void *workspace, int64_t workspace_bytes,
                                    void *stream, const gemm_epilogue_t *epi);

/* Bytes of that workspace; -1 for a size that gemm_mx_matmul_values refuses. */
int64_t gemm_mx_matmul_values_workspace_bytes(int64_t M, int64_t K);

/*
 * Weight gradient from an 8-bit activation checkpoint: dW = alpha * X^T x dY
 * + beta * dW.  The checkpoint is x (T tokens x F features) quantised with
 * GEMM_MX_E4M3 and trans = 1: codes F x T, blocks of 32 tokens of one
 * feature.  dY is T x N of type y_dtype, dW F x N of type c_dtype (F32, F16,
 * BF16 each).  The codes enter the bfloat16 matrix instruction exactly; dY
 * does too: bfloat16 as it is, binary16 as the sum of two bfloat16 terms,
 * FP32 as the sum of three (bits below 2^-133, bfloat16's smallest step, are
 * dropped).  Accumulated in FP32, rounded once.  beta == 0:
 * dW is not read.  T == 0: the empty sum.
 *
 * `workspace` (gemm_mx_wgrad_workspace_bytes bytes, 16-byte aligned, not
 * overlapping the operands) takes two things: dY's bfloat16 terms, where dY
 * is not bfloat16 or N is no multiple of 8, and, where few outputs have many
 * tokens, the FP32 sums of S chunks of tokens, which are added in chunk
 * order.  The workspace may be NULL, or smaller than that: then a slower
 * kernel runs that needs none (as for a bfloat16 dY of rows that are not
 * 16-byte aligned though N is a multiple of 8, or scales off 4-byte words):
 * 8192 tokens, 4096 x 4096, rows of 4099: 1840 us against 201.
 */
gemm_status_t gemm_mx_wgrad(int32_t y_dtype, int32_t c_dtype, int64_t T, int64_t F, int64_t N,
                            const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                            const void *dY, int64_t ldy, void *dW, int64_t ldw,
                            float alpha, float beta,
                            void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of that workspace (0: none is used); -1 for an unknown type or a
 * size that gemm_mx_wgrad refuses. */
int64_t gemm_mx_wgrad_workspace_bytes(int32_t y_dtype, int64_t T, int64_t F, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_ROW_AMD_GEMM_MX_H */
