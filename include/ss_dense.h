/*
 * ss_dense.h -- C ABI of libss.so, part 9: the weight gradient of a dense
 * layer y = x W^T + b whose input x was kept in 8 bits (ss_rows8.h).
 *
 *   dW[i][j] = sum over rows m of dy[m][i] x[m][j],   db[i] = sum of dy[m][i]
 *
 * x[m][j] is q s as it is held.  Every product is exact (x in bfloat16, dy as the sum of one,
 * two or three bfloat16 values, which float16 and float32 values are but for what a float32 has
 * below 2^-133, which is left out), infinite and NaN where dy x is; sums are float32,
 * in the tensor cores for up to 2048 rows (16,384 where dweight has 16 bits), which cut
 * off what float32's last place does not hold, and rounded to nearest from there on.  The rows
 * are split by the sizes, the types and the alignment: with those the same, the same
 * inputs give the same bits.  (Scales below 2^-111, which packing does not make, may leave x
 * bfloat16's subnormals.)  Should one of the kernels' waits run out, dweight and
 * dbias read NaN where it was, which nothing else tells of.
 *
 * Conventions are those of ss.h; rows and strides those of ss_embed.h.
 */
#ifndef SS_DENSE_H
#define SS_DENSE_H

#include "ss.h"
#include "ss_dtype.h"
#include "ss_rows8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace ss_dense_grad8 needs for these sizes (fewer rows may need more);
 * 0 for sizes or types outside the limits. */
size_t ss_dense_grad8_workspace_bytes(int64_t n, int32_t N, int32_t D, ss_dtype dtype,
                                      ss_dtype grad_dtype);

/* dy: device [n][N] of `dtype`; *x: n rows of D; dweight: device [N][D] of
 * grad_dtype (SS_F32 or `dtype`), dbias: device [N] of grad_dtype, NULL if not
 * wanted; both are overwritten (n = 0: with zeros).  workspace: device, 256-byte
 * aligned, >= ss_dense_grad8_workspace_bytes.
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n < 2^31, 1 <= N <= 65536 and
 * 1 <= D <= 65536; SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an unknown type or
 * format, a stride too small, a small or misaligned workspace. */
ss_status ss_dense_grad8(const void *dy, ss_dtype dtype, int64_t dy_stride, const ss_rows8 *x,
                         int64_t n, int32_t N, int32_t D, void *dweight, int64_t dweight_stride,
                         void *dbias, ss_dtype grad_dtype, void *workspace,
                         size_t workspace_bytes, ss_stream_t stream);

/* Test hook for failure detection, not part of the path: ss_dense_grad8 with copies
 * that stop after the first stage of each range of rows (32 or 64 of them), so that the waits
 * for the next one give up, after a few thousand tries; rows that no copies bring (dy or x
 * off 16-byte boundaries, in weights of one tile) are worked on as ever. */
ss_status ss_test_dense_wait_timeout(const void *dy, ss_dtype dtype, int64_t dy_stride,
                                     const ss_rows8 *x, int64_t n, int32_t N, int32_t D,
                                     void *dweight, int64_t dweight_stride, void *dbias,
                                     ss_dtype grad_dtype, void *workspace, size_t workspace_bytes,
                                     ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_DENSE_H */
