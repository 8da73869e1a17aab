/*
 * iq_layers.h -- C-ABI of libiqcodec.so, second part: the operators that run a
 * layer on decoded weights on AMD Instinct MI355X (gfx950).
 *   - products in 8-bit integers with one scale per token and one per output
 *     channel, dense or with a weight per expert, and the rounding of
 *     activations to 8 bits that they take;
 *   - tokens sorted by expert, copied there and brought back with the router's
 *     weights, with the gradients of both copies.
 *
 * The conventions of iq_codec.h hold: device pointers, buffers owned by the
 * caller, nothing allocated, calls ordered on `stream`, argument errors
 * returned before any launch (shapes first, then pointers, then sizes and
 * alignment), data errors reported into `*status` (NULL: the call waits for
 * its stream and returns the data error itself).  What differs here:
 *   - Values are fp32, bf16 or fp16 (IQ_DTYPE_F64 is IQ_ERR_ARG).
 *   - Rows have a stride of their own, in values (`ld...`); the values of a
 *     row are consecutive.  Pointers need the alignment of their own type
 *     only; rows that start on 16 bytes are read fastest.
 *   - An empty batch (no tokens) is no error: the call writes what is left to
 *     write (the offsets of iq_expert_sort) and returns IQ_OK.
 *   - Outputs and workspaces may not overlap inputs or each other (IQ_ERR_ARG).
 *     Rows may interleave: column slices of one buffer do not overlap.
 */
#ifndef IQ_LAYERS_H
#define IQ_LAYERS_H

#include "iq_codec.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most experts, and the largest depth of an 8-bit product: 131071 products
 * of two 8-bit values (2^14 at most each) stay within 32 bits. */
enum { IQ_MAX_EXPERTS = 512, IQ_MAX_INT8_DEPTH = 131071 };

/* Rows rounded to 8-bit integers with a scale each:
 *   scale[r] = max_i |x[r][i]| * (1/127),   q[r][i] = round(x[r][i] / scale[r]),
 * in fp32 with every operation correctly rounded (1/127 too), halves to the
 * even integer; q is within -127..127.  A row of zeros (or one whose scale underflows to 0)
 * has scale 0 and zero codes.  A row that holds a NaN or an infinity is
 * reported as IQ_ERR_NONFINITE and written as zeros with scale 0. */
iq_status_t iq_quantize_rows(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t rows,
                             int64_t cols, int8_t* q, int64_t ldq, float* scale, int32_t* status,
                             hipStream_t stream);

/* y[t][n] = x_scale[t] * w_scale[n] * sum_i x[t][i] * w[n][i], the sum exact in
 * 32-bit integers, its conversion and the two products in fp32 (x_scale first),
 * rounded once to the type of y.  x is [tokens][depth], w [channels][depth]
 * (a weight as decoded: depth innermost), y [tokens][channels]. */
iq_status_t iq_int8_matmul(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                           int64_t ldw, const float* w_scale, int64_t tokens, int64_t channels,
                           int64_t depth, iq_dtype_t out_dtype, void* y, int64_t ldy,
                           hipStream_t stream);

/* iq_quantize_rows of x followed by iq_int8_matmul: a served layer on
 * activations as they come.  y has the type of x.  `workspace` holds the codes
 * and scales between the two, iq_int8_linear_workspace(tokens, channels, depth)
 * bytes, 16-byte aligned; it may be NULL where that is 0. */
int64_t iq_int8_linear_workspace(int64_t tokens, int64_t channels, int64_t depth);
iq_status_t iq_int8_linear(iq_dtype_t dtype, const void* x, int64_t ldx, const int8_t* w,
                           int64_t ldw, const float* w_scale, int64_t tokens, int64_t channels,
                           int64_t depth, void* y, int64_t ldy, void* workspace,
                           int64_t workspace_bytes, int32_t* status, hipStream_t stream);

/* The product with a weight per expert.  Row p of y, offsets[e] <= p <
 * offsets[e+1], is the product of a token with the weight of expert e,
 * w + e * w_stride, [channels][depth]; rows from offsets[experts] on are written
 * as zeros.  The token of row p is order[p] / top_k (iq_expert_sort's order of
 * the choices), or p itself where order is NULL (x already in that order;
 * tokens >= rows).  w_scale is [experts][channels].  `order` and `offsets` are
 * read on the device: values out of range are clamped into it; a row that no
 * expert's range holds (offsets that begin after 0 or decrease, which
 * iq_expert_sort does not give) is not written. */
iq_status_t iq_int8_expert_matmul(const int8_t* x, int64_t ldx, const float* x_scale,
                                  int64_t tokens, const int32_t* order, int32_t top_k,
                                  const int32_t* offsets, int32_t experts, int64_t rows,
                                  const int8_t* w, int64_t ldw, int64_t w_stride,
                                  const float* w_scale, int64_t channels, int64_t depth,
                                  iq_dtype_t out_dtype, void* y, int64_t ldy, hipStream_t stream);

/* Choices sorted by expert: choice is [tokens][top_k], int32 (choice_bytes 4)
 * or int64 (8), each 0..experts-1, or -1 for a choice that was dropped.  The
 * sort keeps the order of equal choices and puts the dropped ones last:
 *   order[p]    the choice (token * top_k + slot) at place p,   [tokens*top_k]
 *   position[c] the place of choice c,                          [tokens*top_k]
 *   offsets[e]  the first place of expert e; offsets[experts] the first place of
 *               the dropped choices,                            [experts+1]
 * Any other choice is reported as IQ_ERR_INDEX and dropped.
 * `workspace`: iq_expert_sort_workspace(tokens * top_k, experts) bytes, 4-byte
 * aligned (NULL where that is 0); it need not be cleared. */
int64_t iq_expert_sort_workspace(int64_t choices, int32_t experts);
iq_status_t iq_expert_sort(const void* choice, int32_t choice_bytes, int64_t tokens, int32_t top_k,
                           int32_t experts, int32_t* order, int32_t* position, int32_t* offsets,
                           void* workspace, int64_t workspace_bytes, int32_t* status,
                           hipStream_t stream);

/* Tokens copied to the places of their choices: sorted[position[t][j]] = x[t],
 * zeros where the choice was dropped (position >= offsets[experts]).  x is
 * [tokens][width], sorted [tokens*top_k][width].  `position` is read on the
 * device: places outside 0..tokens*top_k-1 are skipped, here and below, and
 * sorted rows that are no choice's place are not written. */
iq_status_t iq_expert_dispatch(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                               int64_t width, const int32_t* position, int32_t top_k,
                               const int32_t* offsets, int32_t experts, void* sorted, int64_t lds,
                               hipStream_t stream);

/* Its gradient: x_grad[t] = sum over the kept choices j of sorted_grad[position[t][j]],
 * summed in fp32 in the order of j, rounded once. */
iq_status_t iq_expert_dispatch_backward(iq_dtype_t dtype, const void* sorted_grad, int64_t lds,
                                        int64_t tokens, int64_t width, const int32_t* position,
                                        int32_t top_k, const int32_t* offsets, int32_t experts,
                                        void* x_grad, int64_t ldx, hipStream_t stream);

/* Brought back with the router's weights: out[t] = sum over the kept choices j
 * of weights[t][j] * y[position[t][j]], in fp32 in the order of j, rounded once.
 * Rows of dropped choices are not read.  y is [tokens*top_k][width]. */
iq_status_t iq_expert_combine(iq_dtype_t dtype, const void* y, int64_t ldy, int64_t tokens,
                              int64_t width, const int32_t* position, int32_t top_k,
                              const int32_t* offsets, int32_t experts, const float* weights,
                              void* out, int64_t ldo, hipStream_t stream);

/* Its gradients, for the gradient out_grad of out:
 *   y_grad[position[t][j]] = weights[t][j] * out_grad[t]     (zeros if dropped)
 *   weights_grad[t][j] = <out_grad[t], y[position[t][j]]>    (0 if dropped; fp32
 *                        sums in an order that depends on the width alone). */
iq_status_t iq_expert_combine_backward(iq_dtype_t dtype, const void* out_grad, int64_t ldo,
                                       const void* y, int64_t ldy, int64_t tokens, int64_t width,
                                       const int32_t* position, int32_t top_k,
                                       const int32_t* offsets, int32_t experts,
                                       const float* weights, void* y_grad, int64_t ldg,
                                       float* weights_grad, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IQ_LAYERS_H */
