/*
 * ss_dtype.h -- element types of the training operators (ss_embed.h,
 * ss_norm.h, ss_clip.h).  16-bit values are widened to float32 on load and
 * rounded to nearest even once, on store; sums are held in float32 or more.
 */
#ifndef SS_DTYPE_H
#define SS_DTYPE_H

typedef enum {
    SS_F32 = 0,
    SS_F16 = 1,  /* IEEE binary16 */
    SS_BF16 = 2  /* bfloat16 */
} ss_dtype;

#endif /* SS_DTYPE_H */
