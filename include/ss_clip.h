/*
 * ss_clip.h -- C ABI of libss.so, part 6: the norm of all gradients together,
 * and their scaling so that it stays below a bound.
 *
 *   norm = sqrt(sum over every tensor and element of x^2)
 *   coef = min(1, max_norm / (norm + eps))
 *   out  = coef * x
 *
 * A norm that is not finite (an infinity or a NaN among the gradients, or a
 * norm past float32's 3.4e38) scales nothing: coef is reported as 0, gradients
 * clipped in place keep their values and separate outputs receive copies, so
 * that the caller can see which step to skip.  Where coef is 1, in-place
 * gradients are not written.  Squares that leave float32's range, above or
 * below, are taken of scaled values: a second look at the gradients, which
 * takes half as long again.
 *
 * Squares are summed in float32 over at most a few dozen values and from
 * there on in pairs of float32 that keep the additions' rounding errors,
 * along splits that depend on the sizes, the alignments and the device: with
 * those the same, the same inputs give the same bits.  Conventions are those of
 * ss.h.
 */
#ifndef SS_CLIP_H
#define SS_CLIP_H

#include "ss.h"
#include "ss_dtype.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One gradient tensor; a HOST array of these is read during the call. */
typedef struct {
    const void *in;  /* device, numel contiguous elements, aligned to the type */
    void *out;       /* device, same type and size: `in` itself, or a buffer
                        that overlaps no tensor of the list */
    int64_t numel;   /* >= 0; pointers may be NULL when 0 */
    int32_t dtype;   /* an ss_dtype */
    int32_t reserved;  /* 0 */
} ss_tensor;

/* Bytes of workspace the calls below need; 0 for n_tensors outside the limit. */
size_t ss_clip_workspace_bytes(int32_t n_tensors);

/* result: device float[2], overwritten with (norm, coef).
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n_tensors <= 65536 and the elements
 * in all are < 2^40; SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an
 * unknown type, max_norm or eps negative or NaN, a small or misaligned
 * workspace (256 bytes). */
ss_status ss_grad_clip(const ss_tensor *h_tensors, int32_t n_tensors, float max_norm, float eps,
                       float *result, void *workspace, size_t workspace_bytes,
                       ss_stream_t stream);

/* The norm alone (`out` is not looked at): result[0] = norm, result[1] = 1
 * if it is finite, else 0. */
ss_status ss_grad_norm(const ss_tensor *h_tensors, int32_t n_tensors, float *result,
                       void *workspace, size_t workspace_bytes, ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_CLIP_H */
