/*
 * ss_embed.h -- C ABI of libss.so, part 4: rows of a learned table looked up
 * by id and scaled, and the table's gradient.
 *
 *   forward   out[i, :] = scale * table[ids[i], :]
 *   backward  dtable[v, :] = scale * sum over { i : ids[i] = v } of dout[i, :]
 *
 * An id outside [0, V) names no row: its output row is zero and it adds
 * nothing to the gradient, whatever its dout row holds (infinities and NaN
 * included).  A table row that no id names gets a zero gradient row.
 *
 * The backward sorts (id, position) pairs by id with a stable radix sort and
 * sums each id's rows in order of position, in float32, along splits that
 * depend on the sizes, on how the rows of dout and dtable are aligned and on the
 * device: with those the same, the same inputs give the same bits.
 *
 * Conventions are those of ss.h.  Rows are contiguous; a row's start is
 * `stride` elements after the one before (stride >= D).  Any alignment that
 * the element type has is accepted; rows that start on 16-byte boundaries
 * (base and stride) take the vector path.
 */
#ifndef SS_EMBED_H
#define SS_EMBED_H

#include "ss.h"
#include "ss_dtype.h"

#ifdef __cplusplus
extern "C" {
#endif

/* table: device [V][D]; out: device [n][D], the table's type, sharing no memory
 * with table or ids; ids: device int32 (id_bytes 4) or int64 (id_bytes 8) [n].
 * n = 0 does nothing.
 * Errors: SS_ERR_UNSUPPORTED unless 0 <= n < 2^30, 1 <= V < 2^31 and
 * 1 <= D <= 65536; SS_ERR_INVALID_ARG for a NULL or misaligned pointer, an
 * unknown type, id_bytes other than 4 or 8, a stride below D. */
ss_status ss_embed_fwd(const void *table, ss_dtype dtype, int64_t V, int32_t D,
                       int64_t table_stride, const void *ids, int32_t id_bytes, int64_t n,
                       float scale, void *out, int64_t out_stride, ss_stream_t stream);

/* Bytes of workspace ss_embed_bwd needs; 0 for sizes outside the limits. */
size_t ss_embed_workspace_bytes(int64_t n, int64_t V, int32_t D);

/* dout: device [n][D] of `dtype`; dtable: device [V][D] of grad_dtype (the
 * same type or SS_F32), overwritten whole (n = 0: with zeros), sharing no memory
 * with dout or ids; workspace: device, 256-byte aligned, >=
 * ss_embed_workspace_bytes.  Errors as above,
 * and SS_ERR_INVALID_ARG for a small or misaligned workspace or another
 * grad_dtype. */
ss_status ss_embed_bwd(const void *dout, ss_dtype dtype, int64_t dout_stride, const void *ids,
                       int32_t id_bytes, int64_t n, int64_t V, int32_t D, float scale,
                       void *dtable, ss_dtype grad_dtype, int64_t dtable_stride, void *workspace,
                       size_t workspace_bytes, ss_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SS_EMBED_H */
