/*
 * vrc_model.h -- operators of a tensor-parallel model around its layers, over
 * virtual ranks on one AMD Instinct MI355X (gfx950): layer norm in the
 * collective that comes before it, the cross entropy of an output projection
 * whose vocabulary is split over the ranks, and the gradients of both.
 *
 * They live in libvrc_ops.so beside the operators of vrc_ops.h and share their
 * conventions: arrays of device pointers read during the call only, buffers
 * owned by the caller, no memory allocated or kept, work enqueued on `stream`
 * of the current device, argument errors returned before anything is enqueued,
 * re-entrant and thread-safe, capturable into a graph; VRC_INT32 is not
 * supported.  Where a call takes a workspace, a query beside it tells its size;
 * its contents are the call's own until the work is done, so two calls that may
 * run at once need one each, two graphs that may be replayed at once among them.
 *
 * Arithmetic.  Values are widened to fp32; sums, statistics and products are held
 * in fp32 and rounded once, to nearest even, where they are stored.
 */
#ifndef VRC_MODEL_H
#define VRC_MODEL_H

#include "vrc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm.  Of a row h of `width` values:
 *     mean = sum h / width (0 where not centred: RMS norm),
 *     rstd = (sum (h - mean)^2 / width + eps)^(-1/2),
 *     y = (h - mean) rstd weight + bias.
 * Which rows, by `join`:
 *   VRC_NORM_EACH     rank r's own [rows, width]: h = send[r] + residual[r].
 *   VRC_NORM_SUM      the all-reduced [rows, width]: h = sum over ranks q of send[q]
 *                     + residual[0]; every recv[r] gets all of y.
 *   VRC_NORM_SCATTER  rank c's rows of the sum (vrc_chunk_range of `rows`: the last
 *                     rank takes what the ranks do not divide): h = rows of the sum
 *                     over q of send[q] + residual[c]; recv[c] gets their y.
 * What there is one of per row has `parts` arrays: one for VRC_NORM_SUM, else
 * one for each rank.  The part of a rank without rows may be null.
 */
typedef enum { VRC_NORM_EACH = 0, VRC_NORM_SUM = 1, VRC_NORM_SCATTER = 2 } vrc_norm_join_t;

typedef struct {
    size_t rows, width;    /* of every send[r] */
    vrc_dtype_t dtype;     /* of rows */
    vrc_dtype_t wdtype;    /* of weight, bias and their gradients: dtype or VRC_FP32 */
    vrc_norm_join_t join;
    int center;            /* 0: RMS norm */
    double eps;            /* at least 0 */
} vrc_layer_norm_t;

/*
 *   residual  NULL, or `parts` arrays.
 *   weight    [width]; bias [width] or NULL.
 *   recv      one output per rank.
 *   sum       NULL, or `parts` arrays that receive h, rounded to the type (y is
 *             computed from h before that rounding): the residual stream, and what
 *             the gradient takes.
 *   mean, rstd  NULL, or `parts` arrays of fp32, one value per row.  mean is NULL
 *             where not centred, both where rows have no values (width 0).
 * recv[r] may be send[r] itself (not for VRC_NORM_SCATTER), sum[p] may be
 * residual[p] itself; outputs overlap nothing else.  width < 2^26; rows of up to 16384
 * values are read once, longer ones once for each pass over them.
 */
vrc_status_t vrc_layer_norm(const vrc_layer_norm_t* norm, const void* const* send, const void* const* residual,
                            const void* weight, const void* bias, void* const* recv, void* const* sum,
                            float* const* mean, float* const* rstd, int nranks, vrc_stream_t stream);

/*
 * Its gradient.  With send[r] = dy, joined over the ranks as the rows were, x =
 * (sum - mean) rstd and g = dy weight:
 *     dx = rstd (g - mean of g [where centred] - x mean of (g x)) + residual,
 *     dweight = sum of dy x over all rows of all parts, dbias = sum of dy.
 *   VRC_NORM_EACH     recv[r] = dx of rank r's rows: the gradient of send[r] (and of
 *                     residual[r]) of the forward call.
 *   VRC_NORM_SUM      dy is the sum over ranks (each holds its column-parallel
 *                     products' part of it); every recv[r] = dx.
 *   VRC_NORM_SCATTER  dy of rank c's rows is their sum over ranks; recv[c] = dx of
 *                     rank c's rows: vrc_all_gather of these is the gradient of every
 *                     send of the forward call.
 *   sum, mean, rstd  as the forward call wrote them (mean NULL where not centred).
 *   residual  NULL, or `parts` arrays: what is added to dx, the gradient that
 *             reaches `sum` by the residual stream.
 *   dweight   [width] of wdtype, reduced over all ranks; dbias [width] or NULL.
 * recv[r] may be send[r] itself (not for VRC_NORM_SCATTER); outputs overlap nothing
 * else.  Sums are taken in a fixed order: equal calls give equal bits.
 */
vrc_status_t vrc_layer_norm_grad(const vrc_layer_norm_t* norm, const void* const* send, const void* const* sum,
                                 const float* const* mean, const float* const* rstd, const void* weight,
                                 const void* const* residual, void* const* recv, void* dweight, void* dbias, int nranks,
                                 void* workspace, size_t workspace_bytes, vrc_stream_t stream);

/* The workspace of vrc_layer_norm_grad, in bytes (16-byte aligned). */
vrc_status_t vrc_layer_norm_grad_workspace(const vrc_layer_norm_t* norm, int nranks, size_t* bytes);

/*
 * Cross entropy over a vocabulary split over the ranks.  Rank r holds `vocab[r]`
 * rows of the output projection, weight[r] = [vocab[r], width]; the whole
 * vocabulary is their concatenation.  With z_v = <hidden_t, weight row v>:
 *     lse[t] = log sum over v of exp z_v,      loss[t] = lse[t] - z_target[t].
 * A token whose target is `ignore_index` has loss 0.  One whose target is neither
 * that nor within the vocabulary has loss NaN.  No logits are kept.
 */
typedef struct {
    size_t tokens, width;
    const size_t* vocab;    /* HOST array of nranks: weight rows of each rank, 0 allowed (read during the call) */
    vrc_dtype_t dtype;      /* of hidden, weight and their gradients */
    long long ignore_index;
} vrc_cross_entropy_t;

/*
 *   hidden  [tokens, width], which all ranks share; target [tokens], 64-bit.
 *   loss, lse  [tokens] of fp32; loss may be NULL (and target then too).
 * An empty vocabulary gives lse -infinity.
 * tokens < 2^24, width from 1 to 2^20 - 1, the sum of vocab < 2^23, and tokens and the sum
 * of vocab times width < 2^37 (VRC_ERR_INVALID_ARG otherwise).
 */
vrc_status_t vrc_cross_entropy(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                               const long long* target, float* loss, float* lse, int nranks, void* workspace,
                               size_t workspace_bytes, vrc_stream_t stream);

/* The workspace of vrc_cross_entropy, in bytes (16-byte aligned). */
vrc_status_t vrc_cross_entropy_workspace(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                                         int nranks, size_t* bytes);

/*
 * Its gradient, the logits computed again in pieces of the vocabulary.  With
 * b = dloss[t] (0 where the target is ignore_index) and a = b + dlse[t], the
 * gradient of z_v is
 *     a exp(z_v - lse[t]) - b [v = target[t]],
 * exactly 0 for a token whose a and b are 0, whatever its hidden state, lse and target
 * hold; NaN in all of any other token's whose target is invalid as above.
 *   lse     as the forward call wrote it; dloss [tokens] of fp32; dlse the same, or NULL.
 *   dhidden [tokens, width], summed over the ranks, or NULL;
 *   dweight[r] [vocab[r], width], or dweight NULL.
 * The gradients of the logits are rounded to `dtype` before the two products that
 * are made of them, whose sums are held in fp32 and rounded once; of up to 128 tokens
 * of a 16-bit type they are held as two such values, the rounding and what it left.
 * They are held in units of the largest |a| or |b| of the call's tokens, so that the
 * loss's scale does not matter.  fp16's, in one value as in two, lose bits below 2^-28
 * of it and are 0 below 2^-39 of it: of a token that weighs 2^-k of the largest, those
 * of probabilities below 2^(k - 28) and 2^(k - 39).  Outputs overlap nothing else.  Sums
 * are taken in a fixed order: equal calls on one device give equal bits.
 */
vrc_status_t vrc_cross_entropy_grad(const vrc_cross_entropy_t* ce, const void* hidden, const void* const* weight,
                                    const long long* target, const float* lse, const float* dloss, const float* dlse,
                                    void* dhidden, void* const* dweight, int nranks, void* workspace,
                                    size_t workspace_bytes, vrc_stream_t stream);

/* The workspace of vrc_cross_entropy_grad, in bytes (16-byte aligned); dhidden: whether that is wanted. */
vrc_status_t vrc_cross_entropy_grad_workspace(const vrc_cross_entropy_t* ce, const void* hidden,
                                              const void* const* weight, int dhidden, int nranks, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* VRC_MODEL_H */
