/*
 * iq_router.h -- C-ABI of libiqcodec.so, fourth part: the router of an expert layer
 * on AMD Instinct MI355X (gfx950): each token's experts and their weights from its
 * logits, the loss that keeps the experts evenly used, and the gradients of both.
 *
 * The conventions are those of iq_layers.h.
 */
#ifndef IQ_ROUTER_H
#define IQ_ROUTER_H

#include "iq_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The router's choice.  logits is [tokens][experts]; of each token the top_k
 * (<= experts) largest, the largest first and the lowest expert first among equal
 * ones:
 *   choice[t][j]   the expert,                                  [tokens][top_k]
 *   weights[t][j]  its probability, the softmax of the token's logits in fp32, or
 *                  with renormalize != 0 that divided by the sum of the chosen.
 * A logit of -inf is an expert that is never chosen: where fewer than top_k are
 * left, the last choices are -1 with weight 0, as iq_expert_sort takes them.  A
 * token with a NaN or +inf is reported as IQ_ERR_NONFINITE and has no choices. */
iq_status_t iq_expert_gate(iq_dtype_t dtype, const void* logits, int64_t ldl, int64_t tokens,
                           int32_t experts, int32_t top_k, int32_t renormalize, int32_t* choice,
                           float* weights, int32_t* status, hipStream_t stream);

/* Its gradient: of the logits, in their type, for the gradient of the weights.  The
 * logits are read only where renormalize is 0 and may be NULL otherwise.  Choices
 * out of range count as dropped, here and below. */
iq_status_t iq_expert_gate_backward(iq_dtype_t dtype, const float* weights_grad,
                                    const void* logits, int64_t ldl, int64_t tokens,
                                    int32_t experts, const int32_t* choice, const float* weights,
                                    int32_t top_k, int32_t renormalize, void* logits_grad,
                                    int64_t ldg, hipStream_t stream);

/* How evenly the experts are used:
 *   counts[e]  choices of expert e,                             [experts]
 *   live       tokens with a finite logit (and no NaN or +inf),  [1]
 *   loss       experts * sum_e (counts[e] / sum of the counts) * (the mean over the
 *              live tokens of expert e's probability); 0 without choices or tokens. [1]
 * choice is what iq_expert_sort takes ([tokens][top_k], choice_bytes 4 or 8, -1 for
 * dropped); others out of range are reported as IQ_ERR_INDEX and not counted, a
 * token with a NaN or +inf as IQ_ERR_NONFINITE.  `workspace`:
 * iq_expert_balance_workspace(tokens, experts) bytes, 8-byte aligned (NULL where
 * that is 0); it need not be cleared. */
int64_t iq_expert_balance_workspace(int64_t tokens, int32_t experts);
iq_status_t iq_expert_balance(iq_dtype_t dtype, const void* logits, int64_t ldl, int64_t tokens,
                              int32_t experts, const void* choice, int32_t choice_bytes,
                              int32_t top_k, float* loss, int32_t* counts, int32_t* live,
                              void* workspace, int64_t workspace_bytes, int32_t* status,
                              hipStream_t stream);

/* Its gradient: of the logits, in their type, for the gradient of the loss [1]
 * (device memory); the counts are constants. */
iq_status_t iq_expert_balance_backward(iq_dtype_t dtype, const float* loss_grad,
                                       const void* logits, int64_t ldl, int64_t tokens,
                                       int32_t experts, const int32_t* counts, const int32_t* live,
                                       void* logits_grad, int64_t ldg, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* IQ_ROUTER_H */
