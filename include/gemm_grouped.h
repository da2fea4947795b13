/*
 * libgemm, grouped products -- the products of a layer of experts on MI355X
 * (gfx950): rows sorted by group, one weight matrix a group, group sizes that
 * only the device knows.
 *
 * Groups
 * ------
 * `offsets` is G + 1 int32 values in device memory.  Rows offsets[g] ..
 * offsets[g+1] - 1 of the T rows are group g's; a group may be empty.  Rows
 * before offsets[0] and from offsets[G] on belong to no group (padding).  An
 * offset below 0 or above T counts as 0 or T, one below an earlier offset as
 * that one, so that no contents of `offsets` reach past the operands.
 *
 * Conventions
 * -----------
 * Those of gemm.h: row-major device memory owned by the caller, leading
 * dimensions and strides in elements, calls enqueue on `stream` and return,
 * argument errors are found on the host before any launch, gemm_last_error()
 * has the reason.  No call reads device memory on the host, allocates or
 * needs a workspace, so all can be captured into a graph and replayed with
 * other offsets.  dtype is GEMM_DTYPE_F32, _F16 or _BF16, the type of both
 * operands; c_dtype, the result's, is dtype or GEMM_DTYPE_F32.  Sums are
 * accumulated in FP32 and rounded once; their order depends on the sizes
 * alone, so results are bit-reproducible.  A row's result does not depend on
 * the other rows' values.
 * T, N and K are 0 .. 2^31-1, G is 0 .. 65535.  Errors:
 *   a size outside its range, a leading dimension below its row's length, a
 *   negative stride, results of two groups that overlap or lie between one
 *   another's rows (stride_w of dW below a matrix's extent), a NULL operand, an
 *   unknown type                                          -> INVALID_ARG
 *   an operand not aligned to its elements                -> UNSUPPORTED
 *   an output overlapping an input                        -> ALIAS
 *   launch failure                                        -> HIP
 *
 * Speed: 16-bit operands run on pipelined matrix-core kernels where X's and
 * W's (the gradient's X's and dY's) rows begin on 16 bytes (pointers, leading
 * dimensions and strides) and are whole 16-byte pieces long (K % 8 == 0, and
 * N % 8 == 0 but for trans_w = 1), with leading dimensions below 2^20; the
 * result may lie anywhere.  Everything else runs on a general kernel, at about
 * half their rate for large products and gradients.
 */
#ifndef DENSE_GEMM_ROW_AMD_GEMM_GROUPED_H
#define DENSE_GEMM_ROW_AMD_GEMM_GROUPED_H

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Y[t] = X[t] x W_g for every row t of every group g: X is T x K, Y is T x N.
 * trans_w = 0: W_g is the K x N matrix at W + g * stride_w (rows of ldw);
 * trans_w = 1: W_g is given transposed, N x K (the input's gradient, or
 * weights stored by outputs).  stride_w may be 0 (one matrix for all).
 * fill = 1: rows of no group are set to zero; fill = 0: they are not touched.
 * K == 0: the empty sum.
 */
gemm_status_t gemm_grouped_matmul(int32_t dtype, int32_t c_dtype, int32_t trans_w,
                                  int64_t G, int64_t T, int64_t N, int64_t K, const int32_t *offsets,
                                  const void *X, int64_t ldx, const void *W, int64_t ldw, int64_t stride_w,
                                  void *Y, int64_t ldy, int32_t fill, void *stream);

/*
 * dW_g = alpha * X_g^T x dY_g + beta * dW_g for every group: X is T x K, dY
 * is T x N, dW_g the K x N matrix at dW + g * stride_w.  beta == 0: dW is not
 * read.  A group without rows has the empty sum.  (For weights stored N x K,
 * give dY as X and X as dY.)
 */
gemm_status_t gemm_grouped_wgrad(int32_t dtype, int32_t c_dtype, int64_t G, int64_t T, int64_t K, int64_t N,
                                 const int32_t *offsets, const void *X, int64_t ldx, const void *dY, int64_t ldy,
                                 void *dW, int64_t ldw, int64_t stride_w, float alpha, float beta, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_ROW_AMD_GEMM_GROUPED_H */
