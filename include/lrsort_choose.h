/*
 * lrsort_choose.h -- the best few of a row and what moves by the choice, on AMD
 * MI355X (gfx950): the first places of a sort, whose answer is a small integer key.
 *
 *  - a router's choice of experts (whose ids lrs_group_tokens takes, whose weights
 *    lrs_combine_rows takes):
 *      lrs_route_tokens       ids and weights of the best experts of each token
 *      lrs_route_tokens_grad  the gradient of the weights with respect to the logits
 *  - beam search:
 *      lrs_beam_select        the best continuations over all beams and the vocabulary
 *      lrs_beam_reorder       the beams' states in the order of the chosen parents
 *
 * Conventions, beside those of lrsort_rows.h (matrices and their strides, types,
 * streams, temp storage, overlap, refusals before any work is enqueued):
 *  - What is chosen goes by values as they are where they alone decide, and by sums of
 *    them in float64, not by roundings to float32.  (Between beams the logarithms of sums
 *    count, which are formed from float32 exponentials: see there.)  Equal values, and
 *    sums that float64 holds as one number, go to the lowest id, and a choice is listed
 *    from the best down.
 *  - -infinity takes no part: an expert or a continuation of that value is never
 *    chosen.  A place for which nothing is left gets the id -1 (and the weight 0, or
 *    the score -infinity): an id that lrs_group_tokens and lrs_embedding pass over.
 *    The lowest finite value is a value like others.
 */
#ifndef LRSORT_CHOOSE_H
#define LRSORT_CHOOSE_H

#include "lrsort_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lrs_score_type { LRS_SCORE_SOFTMAX = 0, LRS_SCORE_SIGMOID = 1 } lrs_score_type;

typedef enum lrs_group_score { LRS_GROUP_MAX = 0, LRS_GROUP_TOP2 = 1 } lrs_group_score;

/* Limits of one call. */
#define LRS_MAX_EXPERTS 2048
#define LRS_MAX_SLOTS 64
#define LRS_MAX_GROUPS 64
#define LRS_MAX_BEAMS 1024
#define LRS_MAX_BEAM_COUNT 64

/* Chooses `slots` of `experts` experts for each of `tokens` tokens by its row of
 * d_logits (tokens x experts, l below).
 *   s[t,e] = softmax over e of l[t,e], or 1 / (1 + exp(-l[t,e]))
 *   c[t,e] = s[t,e] + bias[e]          (d_bias float32, NULL: zeros)
 * The experts form num_groups groups of equally many consecutive ones.  A group's
 * score is its largest c, or the sum of its two largest (of one, if it has no
 * more); the kept_groups best groups stay.  The ids are those of the `slots` largest
 * c among their experts, and with s at those ids
 *   w[t,k] = scale * s[t,id] / (sum of s over the chosen ids)   normalize != 0
 *   w[t,k] = scale * s[t,id]                                    normalize == 0
 *  - Without a bias experts are compared by their logits (with the softmax, where groups
 *    are kept by their two best, by s), with one by c.  s, c and the scores of groups are
 *    formed in float64: there a softmax's s is one number from 745 below the token's
 *    largest logit on, a sigmoid 1 above 37 and one number below -709.
 *  - The bias changes the choice only.  An expert whose logit or bias is -infinity
 *    takes no part; a group without any that does is the last.
 *  - NaN is larger than any number, as sorts have it: a NaN logit is chosen, and so
 *    shows in the weights (with the softmax in all of the token's, as +infinity does).
 *  - slots <= 64, experts <= 2048, num_groups <= 64, slots <= kept_groups * (experts / num_groups):
 *    LRS_ERR_INVALID_ARG otherwise, and for groups that do not divide the experts.
 *  - d_ids (tokens x slots of id_type) and d_weights (tokens x slots of weight_type)
 *    are contiguous; d_weights may be NULL. */
lrs_status lrs_route_tokens(lrs_row_type type, const void *d_logits, int64_t ld_logits, int64_t tokens,
                            int64_t experts, int64_t slots, lrs_score_type score, const float *d_bias,
                            int64_t num_groups, int64_t kept_groups, lrs_group_score group_score, int normalize,
                            float scale, lrs_id_type id_type, void *d_ids, lrs_row_type weight_type,
                            void *d_weights, hipStream_t stream);

/* The gradient of lrs_route_tokens' weights with respect to the logits, given that of
 * the weights (d_grad_weights, tokens x slots of weight_type) and the ids it chose;
 * every element of d_grad_logits (tokens x experts of `type`) is written.  With p the
 * normalised weights without `scale`, g = scale * grad_weights, sums over the chosen:
 *   softmax, normalize:  p[k] * (g[k] - sum of g * p)            at ids[k], 0 elsewhere
 *   sigmoid, normalize:  the same times 1 - s[ids[k]]
 *   softmax:             (g[k] at ids[k], 0 elsewhere) * s[e] - s[e] * sum of g * s
 *   sigmoid:             g[k] * s * (1 - s)                      at ids[k], 0 elsewhere
 * The choice itself has no gradient.  Ids outside [0, experts), and those of a logit of
 * -infinity, take no part and their grad_weights are not read into any result; an id
 * that stands twice adds twice, in the order of its places.  d_grad_logits may be
 * d_logits itself (same pointer and stride). */
lrs_status lrs_route_tokens_grad(lrs_row_type type, const void *d_logits, int64_t ld_logits, int64_t tokens,
                                 int64_t experts, int64_t slots, lrs_score_type score, int normalize, float scale,
                                 lrs_id_type id_type, const void *d_ids, lrs_row_type weight_type,
                                 const void *d_grad_weights, void *d_grad_logits, int64_t ld_grad_logits,
                                 hipStream_t stream);

/* The `count` best continuations of each of `batch` searches of `beams` beams.  Row
 * b * beams + i of d_logits (batch * beams x vocab) holds beam i's logits l, d_scores
 * (batch x beams, float32) its score so far:
 *   total[b,i,v] = scores[b,i] + l[b,i,v] - log(sum over v of exp(l[b,i,v]))   normalize != 0
 *   total[b,i,v] = scores[b,i] + l[b,i,v]                                      normalize == 0
 * d_out_scores (batch x count, float32) gets the largest totals, d_parents (int32) their
 * i and d_tokens (id_type) their v; equal totals go to the lowest i, equal logits of one
 * beam to the lowest v.
 *  - Tokens of one beam are compared by their logits (also where a large score, an
 *    infinite one or NaN makes their totals the same), beams by totals in float64.  Sums
 *    of exponentials add up float32 ones in float64: their logarithms are off by less
 *    than 1.2e-7 where that was measured (mostly by 5e-8 alike for all beams), by (2
 *    log(vocab) + 12) * 2^-24 at most, and totals of two beams closer than that may
 *    change places.
 *  - A beam of score -infinity takes no part, and its logits are not read.
 *  - d_finished (batch x beams bytes, NULL: none): a beam whose byte is not 0 offers
 *    end_id at its own score and nothing else; its logits are not read.
 *  - NaN logits are never chosen.  With normalize they, and logits of +infinity, make
 *    all totals of their beam NaN; a NaN score does so too.  NaN totals are larger than
 *    any number.
 *  - batch * beams and beams * vocab are at most 2^31 - 1, beams 1024, count 64; end_id
 *    (where d_finished is given) in [0, vocab).  count may exceed what there is to choose from. */
lrs_status lrs_beam_select(void *d_temp, size_t *temp_bytes, lrs_row_type type, const void *d_logits,
                           int64_t ld_logits, const float *d_scores, const uint8_t *d_finished, int64_t end_id,
                           int64_t batch, int64_t beams, int64_t vocab, int64_t count, int normalize,
                           float *d_out_scores, int32_t *d_parents, lrs_id_type id_type, void *d_tokens,
                           hipStream_t stream);

/* Where the states of beams lie, in bytes: `row_bytes` bytes next to each other at
 *   outer * outer_step + batch * batch_step + beam * beam_step + middle * middle_step
 *   + row * row_step
 * (layers, heads and positions, in any order; a dimension that is not there has size 1). */
typedef struct lrs_beam_layout {
    int64_t outer_step, batch_step, beam_step, middle_step, row_step;
} lrs_beam_layout;

/* out[o,b,j,m,r] = in[o,b,parents[b,j],m,r] for o < outer, b < batch, j < count,
 * m < middle, r < rows: each beam's state is its parent's; zeros where the parent is outside [0, beams).
 * d_parents: batch x count, int32.  Values are moved as bytes, so any type will do.
 *  - d_out may be d_in (same pointer and layout, count <= 64): a beam that is its own
 *    parent is then neither read nor written for itself.  Otherwise they must not
 *    overlap: LRS_ERR_INVALID_ARG if the memory from first to last byte does.
 *  - The rows of d_out must not overlap one another, which is taken from its steps: each
 *    has to pass over all that the smaller ones reach.  Those of d_in may (a step of 0 is
 *    a state that beams share), but not in place, where one search would write what
 *    another reads.  Steps are not negative; outer * batch * middle * rows is at most
 *    2^31 - 1. */
lrs_status lrs_beam_reorder(const void *d_in, const lrs_beam_layout *in_layout, void *d_out,
                            const lrs_beam_layout *out_layout, const int32_t *d_parents, int64_t outer,
                            int64_t batch, int64_t beams, int64_t count, int64_t middle, int64_t rows,
                            int64_t row_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LRSORT_CHOOSE_H */
