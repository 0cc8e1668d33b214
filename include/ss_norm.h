/*
 * ss_norm.h -- C ABI of libss.so, part 5: layer normalisation of rows, and
 * its gradient with the weights' gradients.
 *
 *   mu = mean_j x_j,  r = 1 / sqrt(mean_j (x_j - mu)^2 + eps)
 *   forward   y_j = (x_j - mu) r gamma_j + beta_j
 *   backward  with h_j = (x_j - mu) r and a_j = dy_j gamma_j:
 *             dx_j = r (a_j - mean_k a_k - h_j mean_k a_k h_k)
 *             dgamma_j = sum over rows of dy_j h_j,  dbeta_j = sum of dy_j
 *
 * The variance is taken from the centred values (a second look at the row,
 * held in registers), never as a difference of moments.  Statistics and sums
 * are float32; where mu is far from the row's spread its rounding is averaged
 * out of the centred values, so that a row of one value gives y = beta.
 * The weights' sums run along splits that depend on the sizes, on how the rows
 * are aligned and on the device: with those the same, the same inputs give the
 * same bits.
 *
 * Conventions are those of ss.h; rows and strides those of ss_embed.h.
 */
#ifndef SS_NORM_H
#define SS_NORM_H

#include "ss.h"
#include "ss_dtype.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x, y: device [n][D] of `dtype` (y may be x, row for row); gamma, beta: device [D] of
 * param_dtype (SS_F32 or `dtype`), NULL for 1 and 0; mean, rstd: device float
 * [n], each NULL if not wanted.  n = 0 does nothing.
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n < 2^31 and 1 <= D <= 65536;
 * SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an unknown type, a
 * stride below D, eps negative or not finite. */
ss_status ss_layer_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D,
                            const void *gamma, const void *beta, ss_dtype param_dtype, float eps,
                            void *y, int64_t y_stride, float *mean, float *rstd,
                            ss_stream_t stream);

/* Bytes of workspace ss_layer_norm_bwd needs; 0 for sizes outside the limits. */
size_t ss_layer_norm_workspace_bytes(int64_t n, int32_t D);

/* dy, x, dx: device [n][D] of `dtype` (dx may be dy or x, row for row); mean, rstd: the
 * forward's; dgamma, dbeta: device [D] of param_dtype, overwritten (n = 0:
 * with zeros), both NULL if not wanted; workspace: device, 256-byte aligned,
 * >= ss_layer_norm_workspace_bytes (not read where dgamma and dbeta are
 * NULL).  Errors as above. */
ss_status ss_layer_norm_bwd(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride,
                            ss_dtype dtype, int64_t n, int32_t D, const void *gamma,
                            ss_dtype param_dtype, const float *mean, const float *rstd, void *dx,
                            int64_t dx_stride, void *dgamma, void *dbeta, void *workspace,
                            size_t workspace_bytes, ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_NORM_H */
