/*
 * dora_finetune.h - the rest of a fine-tuning step around the adapted layers, in
 * the same library (libdora.so): layer norm, log probabilities of given tokens
 * and the AdamW step, for training and serving code.
 *
 * The conventions of dora.h hold (types, memory, streams, errors: validation
 * first, no allocation, no synchronisation, nothing kept between calls), with
 * these differences:
 *   - any size >= 1 is taken, not only multiples of 8;
 *   - tensor pointers need the alignment of one element only (workspaces:
 *     16 bytes; else DORA_ERR_ALIGN);
 *   - every launch goes on hip_stream itself.
 * All sums, statistics and states are float32 or wider, and every reduction has
 * a fixed order: two calls on the same inputs return the same bits.
 */
#ifndef DORA_FINETUNE_H
#define DORA_FINETUNE_H

#include "dora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm over rows of `width` elements. */
typedef struct {
    int64_t  rows;      /* 0 <= rows < 2^31                                         */
    int64_t  width;     /* 1 <= width < 2^22                                        */
    int64_t  ld_x;      /* row stride of x in elements, width <= ld_x < 2^31        */
    int64_t  ld_gy;     /* backward: row stride of grad_y (the forward ignores it)  */
    int32_t  dtype;     /* dora_dtype of x, y, weight, bias and their gradients     */
    float    eps;       /* added to the variance; finite and >= 0                   */
    uint32_t flags;     /* must be 0                                                */
    uint32_t reserved;  /* must be 0                                                */
} dora_layernorm_shape;

/* The widest rows whose grad_x alone dora_layernorm_backward forms without a workspace. */
#define DORA_LAYERNORM_NO_WS_WIDTH(dtype) ((dtype) == DORA_BF16 ? 16384 : 8192)

/* Bytes of workspace dora_layernorm_backward needs (0: invalid shape or nothing to reduce). */
DORA_API size_t dora_layernorm_workspace_bytes(const dora_layernorm_shape* shape);

/*
 * y = weight (x - mean) rstd + bias per row, with mean and the (biased) variance
 * of the row taken in two passes over its values and rstd = 1 / sqrt(var + eps).
 *   x            [rows, width], row stride ld_x
 *   weight, bias [width], each may be NULL (taken as 1 and 0)
 *   y            [rows, width] contiguous; must not overlap x
 *   mean, rstd   float32 [rows], each may be NULL when not wanted
 */
DORA_API int dora_layernorm_forward(const dora_layernorm_shape* shape, const void* x,
                                    const void* weight, const void* bias, void* y, float* mean,
                                    float* rstd, void* hip_stream);

/*
 * Backward of dora_layernorm_forward for L with dL/dy = grad_y:
 *   h = grad_y weight, xhat = (x - mean) rstd
 *   grad_x = rstd (h - mean_j h - xhat mean_j (h xhat))
 *   grad_weight = sum_t grad_y xhat,  grad_bias = sum_t grad_y
 *   grad_x [rows, width] contiguous, grad_weight, grad_bias [width], layer
 *   dtype; each may be NULL to skip it.
 *   ws  workspace of dora_layernorm_workspace_bytes(shape); may be NULL for
 *       grad_x alone where width <= DORA_LAYERNORM_NO_WS_WIDTH(dtype)
 */
DORA_API int dora_layernorm_backward(const dora_layernorm_shape* shape, const void* grad_y,
                                     const void* x, const void* weight, const float* mean,
                                     const float* rstd, void* grad_x, void* grad_weight,
                                     void* grad_bias, void* ws, size_t ws_bytes, void* hip_stream);

/* Log probabilities of given tokens under rows of logits. */
#define DORA_LOGPROB_MAX_TOP 64
typedef struct {
    int64_t  rows;      /* 0 <= rows < 2^31                                          */
    int64_t  vocab;     /* 1 <= vocab <= 2^23                                        */
    int64_t  ld;        /* row stride of the logits in elements, vocab <= ld < 2^31  */
    int32_t  dtype;     /* dora_dtype of logits and grad_logits                      */
    int32_t  top;       /* alternatives per row, 0 <= top <= min(vocab, 64)          */
    float    scale;     /* multiplies the logits (1 / temperature), 0 < scale < 2^127 */
    uint32_t reserved;  /* must be 0                                                 */
} dora_logprob_shape;

/* Bytes of workspace dora_token_logprob_forward needs (0: none, or an invalid shape). */
DORA_API size_t dora_token_logprob_workspace_bytes(const dora_logprob_shape* shape);

/*
 * With l = scale * logits[t] and lse = log(sum_j exp(l_j)):
 *   logp[t]      = l_target - lse
 *   entropy[t]   = - sum_j p_j log p_j,  p_j = exp(l_j - lse)
 *   top_*[t, i]  = the i-th largest logit's index and l - lse; equal logits in
 *                  order of their index
 *   logits   [rows, vocab], row stride ld; targets int64 [rows]
 *   logp     float32 [rows]; entropy, lse float32 [rows], may be NULL
 *   top_logp float32 [rows, top], top_index int64 [rows, top]; needed when top > 0
 * A target outside [0, vocab) (-100, say) marks a row without one: the row is
 * skipped, its logp, entropy, lse and top_logp are 0 and its top_index -1.
 * Masked logits are -inf (p = 0) or the type's lowest value.  A row with
 * nothing left (all -inf) has lse = logp = top_logp = -inf and entropy 0; a NaN
 * or +inf in a row makes its logp, entropy and lse NaN (a NaN orders above
 * every number among the alternatives).
 */
DORA_API int dora_token_logprob_forward(const dora_logprob_shape* shape, const void* logits,
                                        const int64_t* targets, float* logp, float* entropy,
                                        float* lse, float* top_logp, int64_t* top_index, void* ws,
                                        size_t ws_bytes, void* hip_stream);

/*
 * Gradient of dora_token_logprob_forward's logp and entropy:
 *   grad_logits_j = scale (grad_logp (1[j = target] - p_j)
 *                          - grad_entropy p_j (log p_j + entropy))
 *   grad_logp, grad_entropy  float32 [rows], each may be NULL (taken as 0)
 *   lse, entropy             as written by the forward (entropy may be NULL
 *                            when grad_entropy is)
 *   grad_logits              [rows, vocab] contiguous, layer dtype; must not
 *                            overlap logits (a row may be read again)
 * Rows without a target and rows with nothing left get zeros.  shape->top is
 * not used.
 */
DORA_API int dora_token_logprob_backward(const dora_logprob_shape* shape, const float* grad_logp,
                                         const float* grad_entropy, const void* logits,
                                         const int64_t* targets, const float* lse,
                                         const float* entropy, void* grad_logits,
                                         void* hip_stream);

/*
 * One tensor of an AdamW step.  States are float32 [n] (state_bits 32), or
 * 8-bit codes with a float32 scale per block of DORA_STATE_BLOCK elements
 * (state_bits 8):
 *   exp_avg     int8 c,  value = exp_avg_scale c |c| / 127^2
 *   exp_avg_sq  uint8 u, its square root = exp_avg_sq_scale (u / 255)^2
 * with the block's largest magnitude as scale and codes rounded to nearest
 * even; a second moment of 2^-126 or more keeps u >= 1.  Squared codes spend their steps
 * on the small values: a step is 1.6% of a value at the block's largest and 16%
 * at a hundredth of it.
 */
#define DORA_STATE_BLOCK 128
typedef struct {
    void*       param;             /* [n], param_dtype: read and written               */
    const void* grad;              /* [n], grad_dtype                                  */
    void*       exp_avg;           /* [n]                                              */
    void*       exp_avg_sq;        /* [n]                                              */
    float*      exp_avg_scale;     /* [ceil(n / 128)] with 8-bit states, else NULL     */
    float*      exp_avg_sq_scale;  /* [ceil(n / 128)] with 8-bit states, else NULL     */
    float*      master;            /* float32 [n] copy of a bf16 param, or NULL; where
                                      given it is the value that is updated and param
                                      becomes its rounding.  All tensors of a call
                                      have one or none does.                           */
    int64_t     n;                 /* 0 <= n < 2^34                                    */
} dora_adamw_tensor;

typedef struct {
    int32_t  param_dtype;      /* dora_dtype of every param                            */
    int32_t  grad_dtype;       /* dora_dtype of every grad                             */
    int32_t  state_bits;       /* 32 or 8                                              */
    uint32_t reserved;         /* must be 0                                            */
    int64_t  step;             /* 1 for the first step                                 */
    double   lr, beta1, beta2, eps, weight_decay;   /* finite; betas in [0, 1); eps >= 0 */
    const float* grad_scale;   /* device: factor on every gradient (a clip
                                  coefficient), or NULL                                */
} dora_adamw_options;

/*
 * AdamW on `count` tensors (`tensors` is a host array of device pointers, read
 * during the call only; no two of the arrays that are written may overlap):
 *   g = grad_scale grad
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in float32 from the stored states; param and states are rounded once (so a
 * decay below float32's spacing at 1 still counts beside an update), the
 * parameter from the moments before their rounding.  A NaN or infinite gradient
 * makes its own element NaN (with 8-bit states: the moments of its block).  With
 * eps = 0 an element whose second moment float32 cannot hold (under 2^-149) is
 * infinite, or NaN where the first moment is 0 too.
 * Pointers and hyperparameters are kernel arguments: a captured graph replays
 * the values of the call that was captured.
 */
DORA_API int dora_adamw_step(const dora_adamw_tensor* tensors, int64_t count,
                             const dora_adamw_options* options, void* hip_stream);

/*
 * Global norm of the gradients (grad and n of each tensor; the rest is not
 * looked at), summed in float64:
 *   norm  = sqrt(sum over all tensors of grad^2)         float32 [1]
 *   scale = min(1, max_norm / (norm + 1e-6))             float32 [1], may be NULL
 * `scale` is what dora_adamw_step takes as grad_scale.  max_norm is finite and
 * >= 0.  ws: dora_grad_norm_workspace_bytes(tensors, count) bytes.
 */
DORA_API size_t dora_grad_norm_workspace_bytes(const dora_adamw_tensor* tensors, int64_t count);
DORA_API int dora_grad_norm(const dora_adamw_tensor* tensors, int64_t count, int32_t grad_dtype,
                            double max_norm, float* norm, float* scale, void* ws, size_t ws_bytes,
                            void* hip_stream);

/*
 * Between 8-bit states and their values (for checkpoints, or to look at them):
 *   (0 <= n < 2^34)
 *   dequantize  out[i] = the value of codes[i] (exp_avg, or exp_avg_sq itself,
 *               not its root, with second_moment), float32 or bf16
 *   quantize    codes and scales of float32 values (values of exp_avg_sq >= 0)
 */
DORA_API int dora_adamw_dequantize(const void* codes, const float* scales, int64_t n,
                                   int second_moment, void* out, int32_t out_dtype,
                                   void* hip_stream);
DORA_API int dora_adamw_quantize(const float* values, int64_t n, int second_moment, void* codes,
                                 float* scales, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* DORA_FINETUNE_H */
