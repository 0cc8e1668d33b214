/*
 * ss_rms.h -- C ABI of libss.so, part 8: root-mean-square norm of rows with
 * the residual's addition, its output in the rows' type or in 8 bits; and the
 * gradients of this norm and of the layer norm (ss_norm.h) from rows kept in
 * 8 bits (ss_rows8.h).
 *
 *   forward   h = x + residual, rounded to the rows' type (h = x without one)
 *             r = 1 / sqrt(mean_j h_j^2 + eps)
 *             y_j = h_j r gamma_j
 *   backward  with a_j = dy_j gamma_j and g_j = h_j r:
 *             dx_j = dsum_j + r (a_j - g_j mean_k a_k g_k)
 *             dgamma_j = sum over rows of dy_j g_j
 *
 * dsum is the gradient that reaches h on its other way, along the residual
 * stream; dx is the gradient of x and of the residual alike.  In a backward pass h
 * (the layer norm's x) is either rows or what was kept of them in 8 bits, with the
 * forward's statistics in both cases.
 *
 * Statistics and sums are float32; a result is rounded once, when it is stored,
 * and an output in 8 bits comes from the float32 y.  Squares past float32's range make r
 * zero.  A row's sum runs in an order that depends on how the rows are aligned and, where they do not
 * start on 32-byte (16-bit types: 16-byte) boundaries, on whether outputs in 8 bits are wanted; the weights' sums along
 * splits that depend on the sizes, the alignment and the device: with those the same, the same
 * inputs give the same bits.
 *
 * Conventions are those of ss.h; rows and strides those of ss_embed.h.
 */
#ifndef SS_RMS_H
#define SS_RMS_H

#include "ss.h"
#include "ss_dtype.h"
#include "ss_rows8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x, residual, sum, y: device [n][D] of `dtype`.  residual: NULL for none;
 * sum: h, wanted (not NULL) where there is a residual and NULL where there is none.
 * y, *out (y in 8 bits), *kept (h in 8 bits), rstd (device float [n]): each NULL
 * if not wanted.  gamma: device [D] of param_dtype (SS_F32 or `dtype`), NULL for 1.
 * sum and y may be x or residual, row for row, but not one another; the rows in 8
 * bits share no memory with anything.  n = 0 does nothing.
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n < 2^31 and 1 <= D <= 65536;
 * SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an unknown type or
 * format, a stride too small, sum without residual or residual without sum, sum = y,
 * eps negative or not finite. */
ss_status ss_rms_norm_fwd(const void *x, ss_dtype dtype, int64_t x_stride, const void *residual,
                          int64_t residual_stride, int64_t n, int32_t D, const void *gamma,
                          ss_dtype param_dtype, float eps, void *sum, int64_t sum_stride, void *y,
                          int64_t y_stride, const ss_rows8 *out, const ss_rows8 *kept, float *rstd,
                          ss_stream_t stream);

/* Bytes of workspace the two backward calls need; 0 for sizes outside the limits. */
size_t ss_rms_norm_workspace_bytes(int64_t n, int32_t D);
size_t ss_layer_norm_bwd8_workspace_bytes(int64_t n, int32_t D);

/* dy, dsum, dx: device [n][D] of `dtype` (dx may be dy, dsum or h, row for row);
 * dsum: NULL for none; h: device [n][D] of `dtype`, or NULL and *kept what was kept of
 * it; rstd: the forward's; dgamma: device [D] of param_dtype, overwritten (n = 0:
 * with zeros), NULL if not wanted; workspace: device, 256-byte aligned, >=
 * ss_rms_norm_workspace_bytes (not read where dgamma is NULL).  Errors as above,
 * and SS_ERR_INVALID_ARG unless one of h and kept is NULL. */
ss_status ss_rms_norm_bwd(const void *dy, int64_t dy_stride, const void *h, int64_t h_stride,
                          const ss_rows8 *kept, ss_dtype dtype, int64_t n, int32_t D,
                          const void *gamma, ss_dtype param_dtype, const float *rstd,
                          const void *dsum, int64_t dsum_stride, void *dx, int64_t dx_stride,
                          void *dgamma, void *workspace, size_t workspace_bytes,
                          ss_stream_t stream);

/* ss_layer_norm_bwd with x kept in 8 bits: its formulas, arguments and errors;
 * workspace >= ss_layer_norm_bwd8_workspace_bytes. */
ss_status ss_layer_norm_bwd8(const void *dy, int64_t dy_stride, const ss_rows8 *kept,
                             ss_dtype dtype, int64_t n, int32_t D, const void *gamma,
                             ss_dtype param_dtype, const float *mean, const float *rstd, void *dx,
                             int64_t dx_stride, void *dgamma, void *dbeta, void *workspace,
                             size_t workspace_bytes, ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_RMS_H */
