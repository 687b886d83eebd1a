/*
 * lrsort_rows.h -- rows of a matrix moved and summed in the order of small
 * integer keys, on AMD MI355X (gfx950): the row-sized payload that the sorts of
 * lrsort.h (which carry 32 bits with each key) stop short of.
 *
 * Two families of operators, both resting on one stable grouping by key:
 *
 *  - tokens sorted by expert and back.  A router gives each of `tokens` tokens
 *    `slots` expert ids; slot (t, k) has the flat index i = t * slots + k.
 *      lrs_group_tokens       the stable order of the slots by expert
 *      lrs_dispatch_rows      rows[position[t,k]] = x[t]
 *      lrs_combine_rows       y[t] = sum_k w[t,k] * rows[position[t,k]]
 *      lrs_combine_rows_grad  its gradient: grad_rows[position[t,k]] = w[t,k] * grad_y[t],
 *                             grad_w[t,k] = <grad_y[t], rows[position[t,k]]>
 *    The gradient of lrs_dispatch_rows is lrs_combine_rows without weights,
 *    grad_x[t] = sum_k grad_rows[position[t,k]];
 *  - embedding lookup.
 *      lrs_embedding          y[i] = scale * table[ids[i] - first_id]
 *      lrs_embedding_grad     grad[v] = scale * sum of grad_y[i] over ids[i] - first_id = v
 *
 * Conventions shared by every call here:
 *  - Ids are int32 or int64 (lrs_id_type).  A call serves the ids
 *    [first_id, first_id + count): one rank's share of the experts or of the
 *    vocabulary, or all of them.  Every other id (a choice that belongs to another
 *    rank, a dropped choice, a padding token) is valid input and takes no part:
 *    it has position -1, is moved nowhere, adds nothing, and its row of an
 *    embedding is zero.  Nothing that belongs to such a slot is read, so NaN or
 *    infinity there never reaches a result.
 *  - Matrices are row-major, of float32, bfloat16 or float16 (lrs_row_type), with
 *    `ld` elements from one row to the next (ld >= cols when there is more than
 *    one row); any alignment of an element's size will do, and rows that begin at
 *    multiples of 16 bytes are fastest.  Positions, ids and weights are contiguous.
 *  - Sums and products are formed in float32 and rounded once (to nearest even)
 *    when an output is stored.  Every sum has a fixed order that depends on the
 *    arguments alone: results are the same on every run.
 *  - Device pointers, streams, asynchrony and graph capture as in lrsort.h: the
 *    library allocates nothing, each call only enqueues kernels on `stream`.
 *    Calls with d_temp follow the two-phase temp storage convention there (the
 *    query with d_temp == NULL checks the arguments too); the size depends on the
 *    sizes and types alone, not on the pointers' values, and a size of 255 (what
 *    alignment may take) means that nothing is stored there.
 *  - Outputs must not overlap inputs or other outputs, except where a call allows
 *    it: LRS_ERR_INVALID_ARG.  Columns of one buffer do not overlap where their
 *    rows are equally far apart, nor do a single row, ids, positions or weights
 *    that lie between a matrix's rows; matrices of different strides are taken to
 *    overlap if the memory from first to last row does.  Overlap of d_temp with
 *    any array is undefined.
 *  - Sizes may be zero.  tokens * slots and the number of ids are at most
 *    2^31 - 1 (positions are int32), rows and columns likewise, the counts of
 *    groups and of a gradient's ids at most 2^31 - 2; strides are 64-bit.  Negative
 *    sizes, NULL pointers to
 *    arrays that are not empty, misaligned pointers, unknown types and
 *    first_id + count beyond int64 give LRS_ERR_INVALID_ARG.  Every check is
 *    made before any work is enqueued.
 *  - Positions are checked against the number of rows on the device: one outside
 *    [0, num_rows) counts as -1.
 */
#ifndef LRSORT_ROWS_H
#define LRSORT_ROWS_H

#include "lrsort.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lrs_id_type { LRS_ID_I32 = 0, LRS_ID_I64 = 1 } lrs_id_type;

typedef enum lrs_row_type { LRS_ROW_F32 = 0, LRS_ROW_BF16 = 1, LRS_ROW_F16 = 2 } lrs_row_type;

/* Stable grouping of n ids into num_groups groups, group g holding the ids equal
 * to first_id + g.  A counting sort: where lrs_sort_pairs_* would return sorted
 * keys, this returns what moving rows needs.
 *  - d_order[n]: the indices 0..n-1 sorted by group, those of no group last;
 *    equal ones in input order.
 *  - d_position[n]: the inverse: where index i stands in d_order, or -1 if its id
 *    is of no group.
 *  - d_offsets[num_groups + 1]: group g is d_order[d_offsets[g]..d_offsets[g+1]);
 *    d_offsets[num_groups] is the number of indices in any group.
 * Each output may be NULL if it is not wanted. */
lrs_status lrs_group_tokens(void *d_temp, size_t *temp_bytes, lrs_id_type id_type, const void *d_ids, int64_t n,
                            int64_t first_id, int64_t num_groups, int32_t *d_order, int32_t *d_position,
                            int32_t *d_offsets, hipStream_t stream);

/* d_rows[d_position[t * slots + k]] = d_x[t] for every slot with a position:
 * d_x is tokens x cols, d_rows num_rows x cols.  Rows of d_rows that no position
 * names are left as they were.  (With positions that are not distinct, which
 * lrs_group_tokens never gives, a row holds one of its sources' values, element
 * by element.) */
lrs_status lrs_dispatch_rows(lrs_row_type type, const void *d_x, int64_t ld_x, const int32_t *d_position,
                             int64_t tokens, int64_t slots, int64_t cols, void *d_rows, int64_t ld_rows,
                             int64_t num_rows, hipStream_t stream);

/* d_y[t] = sum over k of w[t,k] * d_rows[d_position[t * slots + k]], summed in the
 * order of k; slots without a position add nothing, and a token without any gets
 * zeros.  d_weights: tokens x slots of weight_type, or NULL for ones. */
lrs_status lrs_combine_rows(lrs_row_type type, const void *d_rows, int64_t ld_rows, int64_t num_rows,
                            const int32_t *d_position, lrs_row_type weight_type, const void *d_weights,
                            int64_t tokens, int64_t slots, int64_t cols, void *d_y, int64_t ld_y,
                            hipStream_t stream);

/* The gradient of lrs_combine_rows, given that of its output, d_grad_y (tokens x
 * cols):
 *  - d_grad_rows (num_rows x cols): row d_position[t,k] = w[t,k] * d_grad_y[t];
 *    rows that no position names are left as they were.  May be d_rows itself
 *    (same pointer and stride): each element is read before it is replaced.
 *  - d_grad_weights (tokens x slots of weight_type): the inner product of
 *    d_grad_y[t] and d_rows[d_position[t,k]], zero for a slot without a position.
 *    NULL if it is not wanted; then d_rows is not read and may be NULL too.
 * d_weights NULL means ones.  Positions must be distinct. */
lrs_status lrs_combine_rows_grad(lrs_row_type type, const void *d_grad_y, int64_t ld_grad_y, const void *d_rows,
                                 int64_t ld_rows, int64_t num_rows, const int32_t *d_position,
                                 lrs_row_type weight_type, const void *d_weights, int64_t tokens, int64_t slots,
                                 int64_t cols, void *d_grad_rows, int64_t ld_grad_rows, void *d_grad_weights,
                                 hipStream_t stream);

/* d_y[i] = scale * d_table[d_ids[i] - first_id] for i < n (d_table: num_ids x
 * cols, d_y: n x cols), and zeros where d_ids[i] is outside
 * [first_id, first_id + num_ids).  scale == 1 copies values unchanged. */
lrs_status lrs_embedding(lrs_row_type type, const void *d_table, int64_t ld_table, int64_t num_ids,
                         lrs_id_type id_type, const void *d_ids, int64_t n, int64_t first_id, float scale,
                         int64_t cols, void *d_y, int64_t ld_y, hipStream_t stream);

/* The gradient of lrs_embedding with respect to its table, given that of its
 * output, d_grad_y (n x cols, of `type`):
 *    g[v] = scale * (sum of d_grad_y[i] over the i with d_ids[i] = first_id + v)
 * The ids are sorted (with their indices) and each id's rows summed in the order
 * of their indices, in pieces of a length that depends on n, cols and the type
 * alone; the pieces' sums are kept in float32 until they are added up.
 *  - accumulate == 0: every row of d_grad (num_ids x cols, of grad_type) is
 *    written, zeros where no id names it.
 *  - accumulate != 0: g is added to d_grad, in float32, rounded once; rows that no
 *    id names are neither read nor written.
 *  - grad_type: `type`, or LRS_ROW_F32.  LRS_ERR_INVALID_ARG otherwise. */
lrs_status lrs_embedding_grad(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_grad_y,
                              int64_t ld_grad_y, lrs_id_type id_type, const void *d_ids, int64_t n,
                              int64_t first_id, float scale, lrs_row_type grad_type, void *d_grad, int64_t ld_grad,
                              int64_t num_ids, int64_t cols, int accumulate, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LRSORT_ROWS_H */
