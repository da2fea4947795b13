/*
 * libgemm, integer 4-bit weights -- weights in 4 bits with a scale (and zero
 * point) for every group of inputs, and the products of few rows with them
 * (a decoding step's), for one layer or a layer of experts, on MI355X
 * (gfx950).
 *
 * The format
 * ----------
 * A weight matrix is held by outputs: N rows of K values, in groups of
 * `group` (32, 64 or 128) consecutive k; ng = ceil(K / group).  The last group
 * of a row may be shorter.  Group j of row i has
 *   - codes q of 0 .. 15, two a byte: element k in byte codes[i*ldq + k/2],
 *     the even k in the low half.  A row is filled up to whole 32 k, so it is
 *     16 * ceil(K / 32) bytes; what the filling holds does not matter;
 *   - a scale, scales[i*lds + j], of the type of the activations (or F16 /
 *     BF16 as given);
 *   - a zero point, the byte zeros[i*ldz + j] of 0 .. 15, where `zeros` is not
 *     NULL; otherwise 8.
 * A value is scale * (q - zero point).  G matrices of one size are one
 * operand, `stride_*` apart (in bytes for codes and zeros, elements for
 * scales).
 *
 * Conventions
 * -----------
 * Those of gemm_grouped.h, `offsets` among them.  Codes are 16-byte aligned,
 * ldq and stride_q multiples of 16 (else UNSUPPORTED).  Types of activations
 * and scales are GEMM_DTYPE_F16 or _BF16.  Errors besides: a group size that
 * is not 32, 64 or 128, or K above 2^30 -> INVALID_ARG.
 *
 * Speed: products of few rows (see GEMM_W4_ROWS) read codes, activations,
 * scales and zero points in whole pieces wherever their rows begin.  Fastest are
 * rows of X that begin on 16 bytes with K % 8 == 0, and scales (and zero points) a
 * row of which is whole runs of 256 k, aligned to such a run.  Rows of X that
 * begin on 4 bytes take up to 30 % longer; on 2 bytes, or with K odd, 5 to 30 %
 * longer, but 8 to 32 rows of narrow layers 1.3 to 3 times as long (16 rows, 4096 x
 * 4096: 10 us; 4096 x 4095: 30).  Scales off their runs cost up to 15 %.  Scales of
 * rows of fewer than 256 k, and leading dimensions from 2^22 on, are read by
 * element.
 */
#ifndef DENSE_GEMM_ROW_AMD_GEMM_W4_H
#define DENSE_GEMM_ROW_AMD_GEMM_W4_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A coded weight operand (see above); strides are read where G matters. */
typedef struct gemm_w4 {
    const uint8_t *codes;
    int64_t ldq, stride_q;
    const void *scales;
    int64_t lds, stride_s;
    const uint8_t *zeros; /* or NULL: every zero point is 8 */
    int64_t ldz, stride_z;
    int32_t group;
} gemm_w4_t;

/*
 * The coded form, with scales of type s_dtype (F16, BF16), of a matrix of type
 * dtype (F32, F16, BF16).  trans = 0: X is N x K, as the codes are; trans = 1:
 * X is K x N (a row-major weight of the other entry points).  Writes what `q`
 * describes (its pointers are outputs here; its strides are not read).
 *
 * With zero points: lo = min(0, least value), hi = max(0, greatest value) of
 * a group; the scale is (hi - lo) / 15, each operation rounded to FP32, then
 * rounded to its type; the zero point is -lo / scale and a code w / scale +
 * zero point, both ratios rounded to the nearest whole number, ties to even,
 * and the results kept within 0 .. 15.  Without: the scale is (largest
 * magnitude) / 7, rounded alike, and a code w / scale + 8 alike.
 * A scale beyond its type's range is the type's largest.  Where it is 0, codes
 * and zero points are 0 (without zero points codes are 8).  A group that
 * holds an infinity or NaN gets a NaN scale, codes 0 and zero point 0.
 */
gemm_status_t gemm_w4_quantize(int32_t dtype, int32_t s_dtype, int32_t trans, int64_t N, int64_t K,
                               const void *X, int64_t ldx, const gemm_w4_t *q, void *stream);

/* The values of a coded N x K matrix as X (N x K) of type dtype (F32, F16,
 * BF16), rounded to nearest even where the type cannot hold one. */
gemm_status_t gemm_w4_dequantize(int32_t dtype, int32_t s_dtype, int64_t N, int64_t K, const gemm_w4_t *q,
                                 void *X, int64_t ldx, void *stream);

/*
 * Y = X x W^T: X is M x K and Y M x N of type dtype, W the coded N x K matrix
 * with scales of that type.  Up to GEMM_W4_ROWS rows, the codes enter the matrix
 * core as the whole numbers 16 + q (exact in both types), each group's sum is
 * accumulated in FP32, 16 + zero point times the sum of its activations is
 * taken off and the scale applied in FP32; the result is rounded once.  (Where
 * these sums are not finite, for an infinite activation or one near the end of
 * bfloat16's range, a result is taken from sum s (q - zero point) x in 64 bits
 * instead: infinities and NaN are those of the definition, and such a result
 * takes K / 32 steps of one thread.)  With more rows the weights are
 * dequantised first, rounded to dtype (which makes results off by about a third
 * more than their own rounding; call with up to GEMM_W4_ROWS rows at a time where
 * that counts), into `workspace`
 * (gemm_w4_matmul_workspace_bytes bytes, 16-byte aligned, not overlapping the
 * operands; too small a one -> INVALID_ARG) and multiplied as gemm_*_bt does;
 * for fewer it may be NULL.
 */
#define GEMM_W4_ROWS 128
gemm_status_t gemm_w4_matmul(int32_t dtype, int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                             const gemm_w4_t *q, void *Y, int64_t ldy, void *workspace, int64_t workspace_bytes,
                             void *stream);

/* Bytes of that workspace (0: none is used); -1 for a size that
 * gemm_w4_matmul refuses. */
int64_t gemm_w4_matmul_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The same by groups: Y[t] = X[t] x W_g^T for every row t of every group g
 * (X T x K, Y T x N; `offsets` and `fill` as in gemm_grouped_matmul).  Up to
 * GEMM_W4_ROWS rows a group on average (T <= GEMM_W4_ROWS * G) the codes are
 * read by the product itself, each group's codes once for every 16, 32 or 64 of
 * its rows; beyond, all G matrices are dequantised into `workspace`, which must
 * not overlap `offsets` either, and multiplied as gemm_grouped_matmul does.
 */
gemm_status_t gemm_w4_grouped(int32_t dtype, int64_t G, int64_t T, int64_t N, int64_t K, const int32_t *offsets,
                              const void *X, int64_t ldx, const gemm_w4_t *q, void *Y, int64_t ldy, int32_t fill,
                              void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of that workspace (0: none is used); -1 for a size that
 * gemm_w4_grouped refuses. */
int64_t gemm_w4_grouped_workspace_bytes(int64_t G, int64_t T, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_ROW_AMD_GEMM_W4_H */
