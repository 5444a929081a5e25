/*
 * dora_posttrain.h - training on preferences and rewards, in the same library
 * (libdora.so): losses on token log probabilities with their gradients, and
 * matrix updates orthogonalised by Newton-Schulz products.
 *
 * The conventions of dora_finetune.h hold: any size, tensor pointers of one
 * element's alignment (workspaces: 16 bytes), every launch on hip_stream,
 * validation before any launch, no allocation, no synchronisation, nothing kept
 * between calls, and the same bits for the same inputs.
 */
#ifndef DORA_POSTTRAIN_H
#define DORA_POSTTRAIN_H

#include "dora.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Tokens of several sequences, one after the other.  Without offsets sequence s
 * has tokens [s length, (s + 1) length) and tokens = sequences length; with them
 * it has [offsets[s], offsets[s + 1]), and tokens before the first and behind
 * the last sequence count nowhere.  Offsets do not decrease (others give wrong
 * results, but nothing outside the arrays is touched).  A token whose mask is 0
 * does not count either, and its values are not looked at (they may be NaN).
 */
typedef struct {
    int64_t        tokens;     /* 0 <= tokens < 2^34                                  */
    int64_t        sequences;  /* 0 <= sequences < 2^31                               */
    int64_t        length;     /* tokens of each sequence; 0 with offsets             */
    const int64_t* offsets;    /* device [sequences + 1], or NULL                     */
    const uint8_t* mask;       /* device [tokens], or NULL: every token counts        */
} dora_token_batch;

typedef enum {
    DORA_PREFERENCE_SIGMOID = 0,
    DORA_PREFERENCE_HINGE   = 1,
    DORA_PREFERENCE_SQUARE  = 2
} dora_preference_kind;

typedef struct {
    int32_t  kind;       /* dora_preference_kind                                      */
    int32_t  normalize;  /* 1: means over a sequence's counted tokens, 0: sums         */
    double   beta;       /* finite, > 0                                               */
    double   margin;     /* finite                                                    */
    double   smoothing;  /* sigmoid: how often a label is wrong, 0 <= smoothing <= 1   */
} dora_preference_options;

/* Bytes of workspace the preference loss and its gradient need (0: invalid, or nothing to do). */
DORA_API size_t dora_preference_workspace_bytes(const dora_token_batch* batch);

/*
 * Loss of `pairs` pairs of sequences, of which chosen[p] is preferred to
 * rejected[p] (device int64; a sequence may be in any number of pairs):
 *   score_s = beta sum_t (logp_t - ref_logp_t)     over the counted tokens of s,
 *             divided by their number (at least 1) with `normalize`
 *   h       = score_chosen - score_rejected - margin
 *   loss    = sigmoid: (1 - smoothing) log(1 + exp(-h)) + smoothing log(1 + exp(h))
 *             hinge:   max(0, 1 - h)
 *             square:  ((h - 1/2) / beta)^2
 *   logp, ref_logp       float32 [tokens]; ref_logp may be NULL (taken as 0)
 *   loss, logit          float32 [pairs]; logit is h
 *   score, count         float32 [sequences]; count: the counted tokens
 * Sums are float64.  A pair with an index outside [0, sequences) has loss and
 * logit 0 and no gradient.
 */
DORA_API int dora_preference_forward(const dora_token_batch* batch,
                                     const dora_preference_options* options, int64_t pairs,
                                     const float* logp, const float* ref_logp,
                                     const int64_t* chosen, const int64_t* rejected, float* loss,
                                     float* score, float* logit, float* count, void* ws,
                                     size_t ws_bytes, void* hip_stream);

/*
 * grad_logp [tokens] for grad_loss [pairs]: beta sum over the pairs of a token's
 * sequence of +- grad_loss dloss/dh (divided by the sequence's count with
 * `normalize`); 0 for tokens that do not count.  The hinge's slope at h = 1 is 0.
 * logit and count as the forward wrote them.
 */
DORA_API int dora_preference_backward(const dora_token_batch* batch,
                                      const dora_preference_options* options, int64_t pairs,
                                      const float* grad_loss, const float* logit,
                                      const float* count, const int64_t* chosen,
                                      const int64_t* rejected, float* grad_logp, void* ws,
                                      size_t ws_bytes, void* hip_stream);

typedef enum { DORA_REDUCE_TOKEN = 0, DORA_REDUCE_SEQUENCE = 1 } dora_policy_reduce;

typedef struct {
    double   clip_low;      /* 0 <= clip_low <= 1                                      */
    double   clip_high;     /* >= 0, may be infinite                                   */
    double   dual_clip;     /* >= 1, infinite for none                                 */
    double   kl_coef;       /* finite, >= 0                                            */
    double   denominator;   /* divides the sum; 0: the number of what is summed         */
    int32_t  reduce;        /* dora_policy_reduce                                      */
    int32_t  per_sequence;  /* 1: advantages [sequences], 0: [tokens]                  */
} dora_policy_options;

DORA_API size_t dora_policy_workspace_bytes(const dora_token_batch* batch,
                                            const dora_policy_options* options);

/*
 * Clipped policy loss with a divergence from a reference.  Per counted token,
 * with rho = exp(logp - old_logp), A its advantage and d = ref_logp - logp:
 *   gain = A min(rho, 1 + clip_high)                       for A >= 0
 *          A min(max(rho, 1 - clip_low), dual_clip)        for A < 0
 *   kl   = exp(d) - 1 - d
 *   l    = -gain + kl_coef kl
 *   loss = sum of l over the counted tokens / denominator             (token), or
 *          sum over sequences of the mean of l / denominator          (sequence),
 * where a denominator of 0 stands for the number of counted tokens, or of the
 * sequences that have any.  With nothing counted the loss is 0.
 *   logp, old_logp, ref_logp  float32 [tokens]; ref_logp may be NULL (kl = 0)
 *   loss    float32 [1]
 *   stats   float32 [4]: over the counted tokens the mean of kl, the share whose
 *           gain a bound holds (its slope is 0), the mean of rho; their number
 *   weight  float32: what a token's l is multiplied by in the loss, [1] for
 *           `token`, [sequences] for `sequence`
 * Terms and sums are float64.
 */
DORA_API int dora_policy_forward(const dora_token_batch* batch, const dora_policy_options* options,
                                 const float* logp, const float* old_logp, const float* ref_logp,
                                 const float* advantages, float* loss, float* stats, float* weight,
                                 void* ws, size_t ws_bytes, void* hip_stream);

/*
 * grad_logp [tokens] = grad_loss weight dl/dlogp, 0 for tokens that do not count;
 * grad_loss is a device float32 [1], weight as the forward wrote it.  rho exactly
 * at a bound still has its slope.
 */
DORA_API int dora_policy_backward(const dora_token_batch* batch, const dora_policy_options* options,
                                  const float* grad_loss, const float* weight, const float* logp,
                                  const float* old_logp, const float* ref_logp,
                                  const float* advantages, float* grad_logp, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* DORA_POSTTRAIN_H */
