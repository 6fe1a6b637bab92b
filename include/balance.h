/*
 * balance.h -- C ABI of the router's balance loss with its per-expert counts
 * and the gradient of the router's logits, on B200 (sm_100a). Same library
 * (libmoe.so), conventions and error codes as moe.h.
 *
 * For logits l[n_tokens][E] and the experts idx[n_tokens][k] that the router
 * selected (moe_route_noalloc), with the sequences b that seq_offsets cuts the
 * tokens into, T_b tokens each:
 *   s_te = sigmoid(l_te),  p_te = s_te / (sum_j s_tj + eps)  (0 where that is 0;
 *     logits below -104, whose scores fp32 rounds to 0, have scores of 0)
 *   counts_be = number of slots of b's tokens that hold expert e
 *   f_be = E counts_be / (k T_b),  prob_be = mean over b's tokens of p_te
 *   loss = coef / B' * sum_b sum_e f_be prob_be,  B' = sequences with tokens
 * (0 without any). counts carry no gradient, so
 *   dloss/dp_te = g_be = coef f_be / (B' T_b)
 *   dloss/dl_te = (g_be - sum_j g_bj p_tj) / (sum_j s_tj + eps) * s_te (1 - s_te)
 * "LFM2.5-24B-A2B: Biased Routing, Short Convolutions and Ten KV Caches"
 * (flozi.net, English page, section "The router has two different scores")
 * has the sigmoid per logit, the normalised scores and the load that follows
 * from the selection; it states no training loss, so the loss's form is this
 * library's own.
 */
#ifndef SIGMOID_BIAS_TOP_BALANCE_H
#define SIGMOID_BIAS_TOP_BALANCE_H

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace of moe_balance_forward (256-byte aligned; scratch
 * of one call: it may be reused once the call's kernels are done); 0 for token
 * and sequence counts that it refuses. */
size_t moe_balance_workspace(int n_tokens, int n_experts, int n_seqs);

/* loss[1] fp32, counts[B][E] int32, prob[B][E] fp32 (0 for a sequence without
 * tokens) and scale[1] fp32 = coef / B' (for the backward pass).
 * logits [n_tokens][E] of dtype MOE_F32 or MOE_BF16, row t at logits + t * ld
 * elements; idx [n_tokens][k] int32, values outside [0, E) (dropped slots)
 * are not counted; seq_offsets [B + 1] int32: sequence b holds tokens
 * seq_offsets[b] .. seq_offsets[b + 1] - 1, NULL with n_seqs == 1 stands for
 * {0, n_tokens}. Tokens of no sequence do not take part. Offsets that do not
 * ascend within [0, n_tokens] give unspecified results, with no access
 * outside the buffers.
 * 1 <= E <= 256, 1 <= k <= min(E, 8), n_seqs >= 1, eps >= 0; n_tokens and
 * n_seqs below 2^30, n_tokens E and n_seqs E below 2^31. All sums run in a fixed
 * order: equal inputs give equal bits. Device pointers, asynchronous on stream, no allocation. */
int moe_balance_forward(const void *logits, int dtype, int64_t ld, const int32_t *idx,
                        const int32_t *seq_offsets, int n_tokens, int n_experts, int top_k,
                        int n_seqs, float coef, float eps, void *workspace, float *loss,
                        int32_t *counts, float *prob, float *scale, void *stream);

/* The same, with the counts stored in kept[B][E] as well: for a backward pass whose
 * caller changes counts meanwhile (a sum over ranks, say). */
int moe_balance_forward_kept(const void *logits, int dtype, int64_t ld, const int32_t *idx,
                             const int32_t *seq_offsets, int n_tokens, int n_experts, int top_k,
                             int n_seqs, float coef, float eps, void *workspace, float *loss,
                             int32_t *counts, float *prob, float *scale, int32_t *kept,
                             void *stream);

/* grad[n_tokens][E] (contiguous, dtype of the logits) = grad_loss[0] (device,
 * fp32) * dloss/dlogits, from the counts (or kept) and scale of the forward call; 0 for
 * tokens of no sequence. */
int moe_balance_backward(const void *logits, int dtype, int64_t ld, const int32_t *counts,
                         const int32_t *seq_offsets, const float *scale, const float *grad_loss,
                         int n_tokens, int n_experts, int top_k, int n_seqs, float eps, void *grad,
                         void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SIGMOID_BIAS_TOP_BALANCE_H */
