/*
 * lora_preference.h -- C ABI of the preference loss of a fine-tuning step (paired log ratios), forward and backward.
 *
 * The backward of a fine-tuning step starts from a loss over the fine-tuning rows' logits ("DeltaServe:
 * Host-Agnostic Co-Serving of Inference and Fine-Tuning for LLMs", section 3.2, "Backward subprocess").  For a
 * preference loss each pair holds a chosen and a rejected sequence, scored by the policy (the base model with its
 * adapter) and by a reference.  With the base model as the reference, the same tokens ride in the same mixed batch a
 * second time as segments of adapter -1, and lora_token_logprob of those rows is the reference.
 *
 * With x [T,V] the logits, lse_t = log sum_v e^x[t,v], and label_t the token that row t predicts:
 *     lp_t = x[t,label_t] - lse_t                      (label_t < 0: row t is not counted, lp_t = lse_t = 0)
 *     D_s  = sum over the counted rows t of sequence s of (lp_t - ref_t)
 *     m    = beta (D_chosen - D_rejected)
 *     loss = -(1 - eps) log sig(m) - eps log sig(-m)   per pair; eps: label smoothing, sig(m) = 1 / (1 + e^-m)
 *     dloss/dD_chosen = -dloss/dD_rejected = beta (eps sig(m) - (1 - eps) sig(-m))
 *     dlogits[t,v] = dloss_pair * (dloss/dD_s) * ([v = label_t] - e^(x[t,v] - lse_t))
 *
 * The conventions of lora_mixed.h hold.  Logits are bf16 or float32, row-major, ld in elements (>= V; rows need the
 * alignment of an element only); sums and statistics are float32 or wider, in a fixed order.  A logit of -infinity
 * has probability zero; a row without a finite logit, or with a NaN or +infinity, gives NaN, and so does a label >= V.
 * Rows that are not counted are not read.
 */
#ifndef LORA_PREFERENCE_H
#define LORA_PREFERENCE_H

#include "lora_mixed.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The rows of one pair's sequences in the batch; a length may be zero.  The sequences of a call must not overlap. */
typedef struct lora_pair {
    int32_t chosen_start;
    int32_t chosen_len;
    int32_t rejected_start;
    int32_t rejected_len;
} lora_pair_t;

#define LORA_MAX_PAIRS 256

/* logp [T] and lse [T] of every counted row (zero for the others): the reference's pass. */
int lora_token_logprob(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld, const int64_t* labels,
                       float* logp, float* lse, void* stream);

/* The loss.  ref_logp [T] (read for counted rows of a sequence); pairs: HOST [n_pairs], at most LORA_MAX_PAIRS.
 * Writes loss [n_pairs], rewards [n_pairs, 2] (beta D_chosen, beta D_rejected), logp and lse [T] as
 * lora_token_logprob, and coef [n_pairs, 2] (dloss/dD_chosen, dloss/dD_rejected) for the backward. */
int lora_preference_forward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                            const int64_t* labels, const float* ref_logp, const lora_pair_t* pairs /* HOST */,
                            int32_t n_pairs, float beta, float label_smoothing, float* loss, float* rewards,
                            float* logp, float* lse, float* coef, void* stream);

/* dlogits [T,V] (element type dt, ld_d): every row is written, with zeros where it is not counted or in no sequence.
 *   lse, coef: the forward's.   dloss [n_pairs]: the gradient of each pair's loss; NULL: 1 / n_pairs each (the mean).
 * dlogits may be the logits buffer itself (same ld): the gradient then takes the logits' place.
 * Probabilities are e^(x - lse).  Where |lse| >= 256, so that its rounding to float32 would show in them, the row is
 * summed up again; an lse that differs from that sum by more than 2^-21 of itself (a part of a vocabulary, with the whole
 * one's) is taken as given. */
int lora_preference_backward(int32_t T, int32_t V, lora_dtype_t dt, const void* logits, int64_t ld,
                             const int64_t* labels, const float* lse, const float* coef,
                             const lora_pair_t* pairs /* HOST */, int32_t n_pairs, const float* dloss, void* dlogits,
                             int64_t ld_d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_PREFERENCE_H */
