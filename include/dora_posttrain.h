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
 *   kl   = exp(d) - 1 - d, infinite for an infinite d
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

/*
 * Newton-Schulz iteration towards the nearest (semi-)orthogonal matrix:
 *   X <- X / (|X|_F + eps), then for each step k
 *   X <- a_k X + (b_k S + c_k S^2) X,  S = X X^T (X^T X for a tall X: the same X)
 * Singular values s of X become those of the composed polynomials
 * s (a + b s^2 + c s^4); (3.4445, -4.7750, 2.0315) five times takes nearly all of
 * them to between 0.7 and 1.2.
 */
typedef struct {
    const double* coefficients;  /* host [steps][3]: a, b, c; finite, and such that singular
                                    values, Q and S stay below 2^30 (else DORA_ERR_FLAGS)    */
    int32_t       steps;         /* 1 <= steps <= 16                                          */
    uint32_t      reserved;      /* must be 0                                                 */
    double        eps;           /* 2^-100 <= eps, finite as a float32                        */
} dora_newton_schulz;

typedef struct {
    const void* x;     /* [rows, cols] contiguous                                             */
    void*       out;   /* [rows, cols] contiguous; may be its own x, must overlap no other array
                          of the call                                                        */
    int64_t     rows;  /* >= 0; the longer of both at most 2^20, the shorter at most 16384    */
    int64_t     cols;
} dora_matrix;

typedef struct {
    dora_newton_schulz iteration;
    int32_t  dtype;      /* dora_dtype of x and out                                           */
    uint32_t reserved;   /* must be 0                                                         */
} dora_orthogonalize_options;

/*
 * out = the iteration's last X for each of `count` matrices (`matrices` and the
 * coefficients are host arrays, read during the call only).  Matrices of any sizes
 * share launches.  Sums are float32, and float32 results have float32's precision.  A
 * matrix of zeros stays zero; one with a NaN or an infinity becomes NaN throughout, the
 * others of the call do not.
 *
 * The workspace holds 2 to 8 bytes an element, 20 n^2 (n the shorter side) and partial
 * sums, with sides padded to 128 (n <= 64: to 64, the longer one to 128).  Ask for it:
 * how many bytes an element depends on how often the coefficients make the precision
 * ask for a new S on the way.  bf16 matrices take 2 where never, 6 where once, 8 where
 * more often; float32 ones 4 where never, or up to twice with n <= 64, else 8.  The
 * usual five steps ask for none for bf16 and for two for float32, ten for one and for
 * four.
 */
DORA_API size_t dora_orthogonalize_workspace_bytes(const dora_matrix* matrices, int64_t count,
                                                   const dora_orthogonalize_options* options);
DORA_API int dora_orthogonalize(const dora_matrix* matrices, int64_t count,
                                const dora_orthogonalize_options* options, void* ws,
                                size_t ws_bytes, void* hip_stream);

typedef struct {
    void*       param;     /* [rows, cols], param_dtype: read and written                     */
    const void* grad;      /* [rows, cols], grad_dtype                                        */
    float*      momentum;  /* [rows, cols]                                                    */
    float*      master;    /* float32 [rows, cols] copy of a bf16 param, or NULL; where given
                              it is the value that is updated and param becomes its rounding.
                              All tensors of a call have one or none does.                    */
    int64_t     rows, cols;
    double      scale;     /* of this tensor's update, finite                                 */
} dora_muon_tensor;

typedef struct {
    dora_newton_schulz iteration;
    int32_t  param_dtype;   /* dora_dtype of every param                                      */
    int32_t  grad_dtype;    /* dora_dtype of every grad                                       */
    int32_t  nesterov;      /* 0 or 1                                                         */
    uint32_t reserved;      /* must be 0                                                      */
    double   lr, momentum, weight_decay;   /* finite; 0 <= momentum < 1                       */
} dora_muon_options;

/*
 * A step on `count` matrices with orthogonalised updates (no array that is written
 * may overlap another one of the call):
 *   m = momentum m + (1 - momentum) grad
 *   u = momentum m + (1 - momentum) grad with nesterov, else m
 *   p = p (1 - lr weight_decay) - lr scale X(u),  X(u) the iteration's last X from u
 * m and the update are float32; p is rounded once.  u is taken to 22 bits, down to 2^-38 of its
 * largest element, whatever that is.  A NaN or an infinity in a gradient makes its own element of
 * m NaN or infinite, and its own matrix NaN.  The workspace is a float32 dora_orthogonalize's, with
 * a new S less often: the usual five steps ask for none for bf16 parameters without masters (4 bytes
 * an element) and for one for the others (4 with n <= 64, else 8).
 */
DORA_API size_t dora_muon_workspace_bytes(const dora_muon_tensor* tensors, int64_t count,
                                          const dora_muon_options* options);
DORA_API int dora_muon_step(const dora_muon_tensor* tensors, int64_t count,
                            const dora_muon_options* options, void* ws, size_t ws_bytes,
                            void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* DORA_POSTTRAIN_H */
