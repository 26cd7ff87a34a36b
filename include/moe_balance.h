/*
 * moe_balance.h -- C ABI of the router's balance loss (MI355X, gfx950): the
 * loss with the per-expert counts that go into it, and its gradient.
 *
 * T tokens with S scores each (one an expert) and k chosen experts, in B
 * sequences: sequence b is the tokens [seq_offsets[b], seq_offsets[b + 1]), or
 * all T tokens where seq_offsets is NULL (B = 1). Masked tokens (mask[t] == 0)
 * and tokens in no sequence take no part.
 *
 *   p_t      = softmax(scores_t)
 *   n_b      = tokens of sequence b that take part
 *   c_be     = how many of their ids (t, j) are e; ids outside [0, S) are none
 *   loss     = mean over the sequences with n_b > 0 (0 where there is none) of
 *              S / (k n_b^2) sum_e c_be sum_t p_te
 *   dscores  = dloss S / (B' k n_b^2) p_te (c_be - sum_f c_bf p_tf)
 *              (B' sequences with n_b > 0; the counts are constants; 0 for
 *              tokens that take no part)
 *
 * so that ids spread evenly over the experts have loss 1. A token whose
 * scores are all -inf has p_t = 0 and gradient 0; scores of +inf or NaN give NaN.
 * What a token that takes no part holds is not looked at.
 *
 * Sums over tokens are fp32 over up to 64 tokens and fp64 beyond. Conventions
 * are moe_w4a16.h's: dense row-major device tensors, 16-byte aligned (mask,
 * topk_ids and seq_offsets at their type's alignment); the caller owns every
 * buffer and the workspace; nothing is allocated or kept, the host never waits,
 * launches go to `stream` on the current device and may be captured into a HIP
 * graph; calls that share a workspace must not overlap; argument errors are
 * found on the host and returned as moe_w4a16.h's status codes. The same call
 * gives the same bits: no floating-point atomics. seq_offsets is read on the
 * device: it must not decrease and lie in [0, T]; others give an unspecified
 * loss, counts and gradient, but nothing outside the buffers is touched.
 */
#ifndef MOE_BALANCE_H
#define MOE_BALANCE_H

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_MAX_SEQUENCES 8192

/* Sizes of the balance loss (host struct, read during the call only). */
typedef struct {
  int64_t num_tokens;    /* T >= 0, T * k < 2^31 */
  int32_t num_experts;   /* S, 1 .. MOE_MAX_SCORED */
  int32_t top_k;         /* k, 1 .. S */
  int32_t num_sequences; /* B, 1 .. MOE_MAX_SEQUENCES (1 without seq_offsets) */
  int32_t type;          /* of scores and dscores: MOE_TYPE_* */
} moe_balance_problem;

/* Bytes of workspace of moe_balance_loss (host only). */
int moe_balance_workspace_size(const moe_balance_problem *p, size_t *bytes);

/*
 * loss fp32 [1], counts int32 [B, S], tokens int32 [B] (n_b) from scores
 * [T, S], topk_ids int32 [T, k], mask (one byte a token, or NULL: all take
 * part) and seq_offsets int32 [B + 1] (or NULL).
 */
int moe_balance_loss(const void *scores, const int32_t *topk_ids, const uint8_t *mask,
                     const int32_t *seq_offsets, float *loss, int32_t *counts, int32_t *tokens,
                     const moe_balance_problem *p, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * dscores [T, S], of the scores' type, from dloss fp32 [1] (on the device),
 * the scores, and counts and tokens as moe_balance_loss wrote them for the
 * same scores, mask and seq_offsets. T == 0 is a no-op.
 */
int moe_balance_loss_backward(const float *dloss, const void *scores, const int32_t *counts,
                              const int32_t *tokens, const uint8_t *mask,
                              const int32_t *seq_offsets, void *dscores,
                              const moe_balance_problem *p, void *stream);

#ifdef __cplusplus
}
#endif
#endif
