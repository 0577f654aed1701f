/*
 * vrc_ops.h -- the tensor-parallel layer's operators over virtual ranks on
 * one AMD Instinct MI355X (gfx950): dropout inside the collectives, and
 * microscaled 4-bit quantisation with its product.
 *
 * They stand beside the collectives of vrc.h and share its conventions:
 * arrays of `nranks` device pointers read during the call only, buffers owned
 * by the caller, no memory allocated or kept, work enqueued on `stream` (NULL
 * = the null stream) of the current device, argument errors returned before
 * anything is enqueued, re-entrant and thread-safe, capturable into a graph.
 * They live in libvrc_ops.so, apart from libvrc.so, whose kernels only stream
 * through registers; a HIP failure's code is vrc_ops_last_hip_error().
 * VRC_INT32 is not supported by any of them (VRC_ERR_UNSUPPORTED).
 *
 * Dropout.  Element i (its index in the whole tensor that the collective
 * makes, row-major, whatever the split over ranks) is dropped when
 *     w_i < round(p * 2^32),
 * w_i being word i mod 4 of Philox-4x32-10 (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", SC 2011) with the counter
 * (i / 4 as two words, offset as two words) and the key `seed` (two words, low
 * words first).  A dropped element is +0 whatever the sum was (infinities and
 * NaN too); a kept one is multiplied by 1 / (1 - p) rounded to fp32.  Nothing
 * of the mask is stored: a later call with the same p, seed and offset applies
 * the same mask.
 *
 * Arithmetic.  The ranks' values are widened to fp32 and folded in rank order,
 * multiplied by the scale, the residual is added in fp32, and the result is
 * rounded once, to nearest even, into the storage type.
 *
 * Microscaled 4-bit blocks (OCP Microscaling Formats 1.0, MXFP4).  32
 * consecutive values share a scale 2^X, held as the byte X + 127 (E8M0); each
 * value is held as a 4-bit code (E2M1: sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6),
 * two to a byte with the lower-indexed value in the low half.
 *     X = floor(log2 max|v|) - 2, at least -127 (an all-zero block: -127);
 *     code = v / 2^X rounded to nearest, ties to the even code; magnitudes
 *     from 6 up are held as 6 (max|v| / 2^X < 8).
 * A block with an infinity or NaN has the scale byte 255 (NaN) and codes 0: it
 * decodes to NaN, and the products of its row are NaN.  A matrix [rows, cols]
 * has KB = ceil(cols / 32) blocks a row: codes [rows, 16 * KB] bytes and scales
 * [rows, KB] bytes, the codes past `cols` zero.  Codes are 16-byte aligned.
 */
#ifndef VRC_OPS_H
#define VRC_OPS_H

#include "vrc.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VRC_OPS_VERSION 100 /* 1.0.0 */
#define VRC_MX4_BLOCK 32    /* values that share a scale */

typedef struct {
    double p;                  /* probability of dropping an element, in [0, 1]; 1 drops all */
    unsigned long long seed;   /* the generator's key */
    unsigned long long offset; /* the counter's upper half: one value per mask */
    /* NULL, or a DEVICE address (8-byte aligned) of a number that is added to
     * `offset` (modulo 2^64) when the kernel runs: a captured graph draws a new
     * mask at every replay once the caller advances it.  It lies in no output
     * (VRC_ERR_ALIAS). */
    const unsigned long long* offset_dev;
} vrc_dropout_t;

/*
 * All-reduce, dropout, residual:
 *   recv[r] = residual[r] + drop(sum over ranks q of send[q]), every rank r.
 *   residual  NULL for none, or `nranks` device pointers; the same pointer in
 *             every place is one residual for all ranks, read once.
 *   recv[r] may be send[r] or residual[r] itself; any other overlap of an output
 *   with another buffer returns VRC_ERR_ALIAS (so a residual shared by several
 *   ranks cannot be an output).
 * Gradient.  The call is linear and symmetric in the ranks: the gradient of
 * every send[q] is this same call (same dropout, no residual) over the outputs'
 * gradients; a residual's is its output's gradient (a shared one's: their
 * all-reduce).
 */
vrc_status_t vrc_allreduce_dropout(const void* const* send, const void* const* residual, void* const* recv,
                                   int nranks, size_t count, vrc_dtype_t dtype, const vrc_dropout_t* dropout,
                                   vrc_stream_t stream);

/*
 * Reduce-scatter, dropout, residual: the chunks, `count` and `outer` are those
 * of vrc_reduce_scatter; the mask is that of the unsplit tensor.
 *   recv[c] = residual[c] + chunk c of drop(sum over ranks q of send[q]).
 *   residual  NULL, or `nranks` device pointers, residual[c] laid out as recv[c].
 *   recv[c] may be residual[c] itself; no other overlap.
 * Gradient: every send[q]'s is vrc_all_gather_dropout of the outputs' gradients
 * (same dropout); a residual's is its output's gradient.
 */
vrc_status_t vrc_reduce_scatter_dropout(const void* const* send, const void* const* residual, void* const* recv,
                                        int nranks, size_t count, size_t outer, vrc_dtype_t dtype,
                                        const vrc_dropout_t* dropout, vrc_stream_t stream);

/*
 * All-gather, dropout: recv[r] = drop(concatenation of the send buffers), every
 * rank r, laid out as by vrc_all_gather; element indices are those of the gathered
 * tensor, which has `total` elements in `outer` rows.  With outer == 1 input c holds
 * its chunk c (vrc_chunk_range: the last chunk takes what the ranks do not divide);
 * with outer > 1 it holds [outer, total / outer / nranks].  For each element it is
 * one multiplication of an input in fp32, rounded to the type.  Outputs overlap no
 * other buffer.
 * Gradient: each send[c]'s is vrc_reduce_scatter_dropout of the outputs'
 * gradients (same dropout, no residual).
 */
vrc_status_t vrc_all_gather_dropout(const void* const* send, void* const* recv, int nranks, size_t total,
                                    size_t outer, vrc_dtype_t dtype, const vrc_dropout_t* dropout,
                                    vrc_stream_t stream);

/* The axis along which 32 values share a scale. */
typedef enum {
    VRC_MX4_ALONG_COLS = 0, /* blocks along a row: codes [rows, 16 ceil(cols/32)], scales [rows, ceil(cols/32)] */
    VRC_MX4_ALONG_ROWS = 1  /* blocks down a column, stored as the transposed matrix's rows: codes
                               [cols, 16 ceil(rows/32)], scales [cols, ceil(rows/32)] */
} vrc_mx4_axis_t;

/*
 * Quantise x[r], [rows, cols] row-major, for every rank r in one launch.
 * codes and scales overlap no other buffer.  rows == 0 or cols == 0: nothing.
 */
vrc_status_t vrc_mx4_quantize(const void* const* x, void* const* codes, void* const* scales, int nranks, size_t rows,
                              size_t cols, vrc_dtype_t dtype, vrc_mx4_axis_t axis, vrc_stream_t stream);

/*
 * Decode rank r's [rows, cols] matrix (codes laid out by VRC_MX4_ALONG_COLS)
 * into recv[r], for every rank.  Values are exact in fp32, but for magnitudes of
 * 2^128 and more (scale byte 253 with 4 or 6, 254 with 2 to 6; the quantiser
 * makes neither), which are infinite; fp16 and bf16 round to nearest even
 * (overflow to infinity).
 */
vrc_status_t vrc_mx4_dequantize(const void* const* codes, const void* const* scales, void* const* recv, int nranks,
                                size_t rows, size_t cols, vrc_dtype_t dtype, vrc_stream_t stream);

/*
 * All-gather of quantised matrices: recv[r], for every rank r, is the decoded
 * concatenation of all ranks' [rows, cols] matrices, along the rows
 * (by_cols == 0: [nranks * rows, cols]) or along the columns (by_cols != 0:
 * [rows, nranks * cols]).  Every code is read once.
 */
vrc_status_t vrc_mx4_all_gather(const void* const* codes, const void* const* scales, void* const* recv, int nranks,
                                size_t rows, size_t cols, int by_cols, vrc_dtype_t dtype, vrc_stream_t stream);

/* How vrc_mx4_matmul joins the ranks' products. */
typedef enum {
    VRC_MX4_SUM = 0, /* recv[r] = sum over ranks q of A_q B_q^T, every rank r: the all-reduced row-parallel product */
    VRC_MX4_EACH = 1 /* recv[r] = A_r B_r^T */
} vrc_mx4_join_t;

/*
 * Product of quantised matrices.  A_r: [m, 32 kblocks] and B_r: [n, 32 kblocks]
 * as VRC_MX4_ALONG_COLS lays them out (codes past the end of a row zero, as the
 * quantiser leaves them); recv[r]: [m, n] row-major, of type `dtype`.
 *   Each product of two codes is exact; sums are held in fp32 over all of k and,
 *   for VRC_MX4_SUM, over all ranks, and rounded once.  The order of the sum is
 *   fixed by the sizes and by the device's number of CUs, so equal calls on one
 *   device give equal bits.  A partial sum beyond fp32's range leaves its result
 *   undefined.
 *   kblocks == 0 gives zeros.  Outputs overlap no other buffer.
 *   m, n < 2^31, kblocks < 2^20.
 * Gradients of recv = A B^T, with G the output's gradient: A's is G B, the product of
 * G quantised along its columns and B quantised VRC_MX4_ALONG_ROWS; B's is G^T A, of
 * G and A both quantised VRC_MX4_ALONG_ROWS.
 */
vrc_status_t vrc_mx4_matmul(const void* const* a_codes, const void* const* a_scales, const void* const* b_codes,
                            const void* const* b_scales, void* const* recv, int nranks, size_t m, size_t n,
                            size_t kblocks, vrc_dtype_t dtype, vrc_mx4_join_t join, vrc_stream_t stream);

/* HIP error code of the most recent VRC_ERR_HIP of this library on the calling thread (0 if none). */
int vrc_ops_last_hip_error(void);

/* VRC_OPS_VERSION of the loaded library. */
int vrc_ops_version(void);

#ifdef __cplusplus
}
#endif

#endif /* VRC_OPS_H */
