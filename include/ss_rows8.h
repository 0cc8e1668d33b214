/*
 * ss_rows8.h -- C ABI of libss.so, part 7: rows held in 8 bits, as the
 * activations that a backward pass will need.
 *
 * Every 32 columns of a row (the last group may be shorter) share a scale, a
 * power of two s = 2^(e - 127) whose biased exponent e is one byte; an element is
 * held as q, and reads as q s:
 *   Q = 127 (SS_INT8) or 448 (SS_E4M3)
 *   s = the least power of two with max |x_j| <= Q s, but at least 2^-111
 *   q = x / s, rounded to nearest even: whole numbers -127 .. 127, or the 8-bit
 *       floats with 4 exponent bits and 3 of mantissa (1 sign; no infinities)
 * A group that holds an infinity or a NaN has e = 255 and q = 0, and reads as
 * NaN throughout.
 * Rows that were not packed are read by the same formula: any q (-128 and the
 * 8-bit floats' NaN, 0x7f and 0xff, too) times 2^(e - 127), NaN where e = 255.
 *
 * A division by a power of two is exact, so an element is rounded once:
 * |q s - x| <= s / 2 (SS_INT8), or the larger of |x| 2^-4 and s 2^-10
 * (SS_E4M3); s < 2 max|x| / Q (or 2^-111).  And q s has at most 7 significant bits and
 * no subnormals, so bfloat16 holds it exactly; only a value within a sixteenth of
 * float32's largest may be rounded past the range, and reads as an infinity then.
 *
 * Conventions are those of ss.h; rows and strides those of ss_embed.h.
 */
#ifndef SS_ROWS8_H
#define SS_ROWS8_H

#include "ss.h"
#include "ss_dtype.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SS_INT8 = 0,
    SS_E4M3 = 1
} ss_format8;

#define SS_ROWS8_GROUP 32

/* Rows of D values in 8 bits; a HOST struct, read during the call.  Row i's
 * values begin at q + i * q_stride and take D bytes, rounded up to whole 8 (the
 * bytes past D are written as zeros, and whoever fills rows without packing writes
 * zeros there, too: the norms' gradients read them); its scales are the bytes
 * scales + i * scale_stride + (0 .. (D + 31) / 32 - 1). */
typedef struct {
    void *q;              /* device, 8-byte aligned */
    int64_t q_stride;     /* bytes, a multiple of 8, at least D rounded up to one */
    uint8_t *scales;      /* device */
    int64_t scale_stride; /* bytes, at least (D + 31) / 32 */
    int32_t format;       /* an ss_format8 */
    int32_t reserved;     /* 0 */
} ss_rows8;

/* x: device [n][D] of `dtype`; *out is written, and shares no memory with x.
 * n = 0 does nothing.
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n < 2^31 and 1 <= D <= 65536;
 * SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an unknown type or
 * format, a stride too small. */
ss_status ss_rows8_pack(const void *x, ss_dtype dtype, int64_t x_stride, int64_t n, int32_t D,
                        const ss_rows8 *out, ss_stream_t stream);

/* x: device [n][D] of `dtype`, overwritten with q s: exactly in SS_F32 and
 * SS_BF16; in SS_F16 rounded, and finite values held to +-65504 (a value near the end of its
 * range may have been rounded past it).  Errors as above. */
ss_status ss_rows8_unpack(const ss_rows8 *in, int64_t n, int32_t D, void *x, ss_dtype dtype,
                          int64_t x_stride, ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_ROWS8_H */
