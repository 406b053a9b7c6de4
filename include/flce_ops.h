/*
 * flce_ops.h — C ABI of the operators around the language-model head that
 * libflce.so provides next to the fused linear cross-entropy of flce.h:
 *
 *   - log probabilities of given tokens with the entropy and the most likely
 *     alternatives of each row, over given logits or straight from hidden states
 *     (the [N, V] logits are never stored), and their gradients;
 *   - layer norm (the norm whose output is the head's H), forward and backward;
 *   - the global norm of many gradients, and clipping by it.
 *
 * flce.h's conventions hold unless a function says otherwise: dense row-major
 * device memory, bf16 as uint16_t bit patterns, caller-owned outputs and
 * workspaces, stream-ordered calls that allocate nothing, host-side errors
 * returned before anything is enqueued, FLCE_ERR_* codes, FLCE_DTYPE_* types.
 * A call with no rows (N = 0) or no gradients is valid.
 */
#ifndef FLCE_OPS_H_
#define FLCE_OPS_H_

#include <stddef.h>
#include <stdint.h>

#include "flce.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FLCE_MAX_TOP_K = 32 };

typedef struct flce_logprob_options {
  int32_t ignore_index; /* token id that marks a row without a token; default -100 */
  int32_t top_k;        /* alternatives per row, 0 (default) to min(FLCE_MAX_TOP_K, V) */
  float temperature;    /* the logits are divided by it: 1e-6 to 1e6, default 1 */
  int32_t dw_dtype;     /* linear form: dW element type, FLCE_DTYPE_F32 (default) or _BF16 */
  int64_t timeout_ns;   /* limit of every device-side wait; 0 = 2 s */
} flce_logprob_options;

/* Fill *opt with the defaults listed above. */
void flce_default_logprob_options(flce_logprob_options* opt);

/*
 * Log probabilities of given tokens over given logits. Per row, with
 * x_v = z_v / temperature, M = max_v x_v and S = sum_v exp(x_v - M):
 *
 *   lse      = M + log S
 *   logprob  = x_y - lse          (as -log1p(sum of the others / the token's term):
 *                                  exact to fp32 however close to 0)
 *   entropy  = log S - sum_v exp(x_v - M) (x_v - M) / S
 *   top      = the top_k largest logits in descending order, the lowest id first
 *              among equal ones: their ids and their x_v - lse
 *
 *   logits   [N, V] of dtype (FLCE_DTYPE_F32 / _BF16), row stride ld >= V elements;
 *            aligned to its element size (16-byte aligned rows are fastest)
 *   tokens   int32 [N], 4-byte aligned: ids in [0, V) or ignore_index; NULL = no row
 *            has a token
 *   logprob, entropy, lse   fp32 [N], 4-byte aligned (any may be NULL)
 *   top_logprob, top_id     fp32 / int32 [N, top_k] (both required if top_k > 0)
 *   status   int32 [1] or NULL. It is only written when the device finds an error
 *            (unlike flce.h's calls, which also reset it): the caller zeroes it once.
 *
 * A row without a token has logprob 0; its other outputs are as usual. A logit of
 * -inf is an id that cannot come: it is never an alternative, and where fewer than
 * top_k ids are left the remaining slots hold id -1 and -inf. A row whose logits
 * are all -inf has lse = logprob = -inf and entropy 0. A row with a NaN or +inf has
 * NaN for logprob, entropy, lse and its top log probabilities. A token outside
 * [0, V) that is not ignore_index gives logprob NaN and FLCE_ERR_LABEL_RANGE; a wait
 * that ran out of time gives FLCE_ERR_TIMEOUT and NaN for its row and for those still to
 * come in the same CTAs (the linear form's calls below: for what they did not compute).
 * Sums and maxima are fp32; results do not change from run to run.
 */
int flce_token_logprobs(const void* logits, int32_t dtype, int64_t ld, const int32_t* tokens,
                        int64_t N, int64_t V, const flce_logprob_options* opt, float* logprob,
                        float* entropy, float* lse, float* top_logprob, int32_t* top_id,
                        int32_t* status, void* stream);

/*
 * Gradient of flce_token_logprobs in the logits. With a = dL/dlogprob, b =
 * dL/dentropy and c = dL/dlse per row (fp32 [N]; each may be NULL for 0, not all):
 *
 *   dL/dz_v = (p_v (c - a - b (log p_v + entropy)) + a [v = y]) / temperature
 *
 * with p_v = exp(x_v - lse), and at the token a (1 - p_y) with 1 - p_y =
 * -expm1(logprob), so that a confident token's entry keeps its precision. lse,
 * entropy and logprob are what flce_token_logprobs wrote (fp32 [N]; entropy may be
 * NULL when b is, logprob when tokens is). a counts for no row
 * without a token. Every -inf logit has gradient 0, and so has a row with lse below
 * -1e30 (every id masked, with -inf or with the type's lowest value). p carries the
 * fp32 rounding of lse, 2^-24 |lse|. Options as in the forward call (top_k is not read).
 *   dlogits  [N, V] of the logits' dtype, row stride dld >= V; may be the logits
 *            themselves with dld == ld, must not otherwise overlap them
 */
int flce_token_logprobs_backward(const void* logits, int32_t dtype, int64_t ld,
                                 const int32_t* tokens, int64_t N, int64_t V,
                                 const flce_logprob_options* opt, const float* logprob,
                                 const float* entropy, const float* lse, const float* dlogprob,
                                 const float* dentropy, const float* dlse, void* dlogits,
                                 int64_t dld, void* stream);

/*
 * The same from hidden states: z = H W^T with H bf16 [N, D] and W bf16 [V, D]
 * (16-byte aligned, D % 8 == 0), products accumulated in fp32, and no [N, V] array
 * but for up to 128 rows, whose fp32 logits pass through the workspace. Outputs and
 * rules as in flce_token_logprobs. The workspace (16-byte aligned,
 * flce_linear_logprobs_workspace_size() bytes with backward = 0) holds the partial
 * results of each vocabulary range.
 */
int flce_linear_logprobs_workspace_size(int64_t N, int64_t D, int64_t V,
                                        const flce_logprob_options* opt, int32_t backward,
                                        size_t* bytes);
int flce_linear_token_logprobs(const uint16_t* H, const uint16_t* W, const int32_t* tokens,
                               int64_t N, int64_t D, int64_t V, const flce_logprob_options* opt,
                               float* logprob, float* entropy, float* lse, float* top_logprob,
                               int32_t* top_id, void* workspace, size_t ws_bytes,
                               int32_t* status, void* stream);

/*
 * Gradients of flce_linear_token_logprobs: G = dL/dz as in
 * flce_token_logprobs_backward, recomputed chunk by chunk and rounded once to bf16
 * (the operand type of the tensor cores), dH = G W and dW = G^T H accumulated in
 * fp32.
 *   dH  bf16 [N, D], or NULL      dW  [V, D] fp32 or bf16 (opt->dw_dtype), or NULL
 *   (not both NULL; 16-byte aligned)
 * workspace: flce_linear_logprobs_workspace_size() with backward = 1.
 */
int flce_linear_token_logprobs_backward(const uint16_t* H, const uint16_t* W,
                                        const int32_t* tokens, int64_t N, int64_t D, int64_t V,
                                        const flce_logprob_options* opt, const float* logprob,
                                        const float* entropy, const float* lse,
                                        const float* dlogprob, const float* dentropy,
                                        const float* dlse, uint16_t* dH, void* dW,
                                        void* workspace, size_t ws_bytes, int32_t* status,
                                        void* stream);

/*
 * Layer norm over the rows of x [N, D]:
 *
 *   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
 *   y = (x - mean) rstd weight + bias
 *
 *   x, y          of dtype, row strides ldx, ldy >= D elements (y may be x)
 *   weight, bias  [D] of wdtype; either may be NULL (1 and 0)
 *   mean, rstd    fp32 [N], or NULL
 * Statistics and products are fp32 (the variance from centred values); y is rounded
 * once. Every pointer is aligned to its element size.
 */
int flce_layer_norm(const void* x, int32_t dtype, int64_t ldx, const void* weight,
                    const void* bias, int32_t wdtype, int64_t N, int64_t D, float eps, void* y,
                    int64_t ldy, float* mean, float* rstd, void* stream);

/*
 * Its gradients, with h = (x - mean) rstd and g = dy weight:
 *
 *   dx = rstd (g - mean_D(g) - h mean_D(g h)),  dweight = sum_rows dy h,
 *   dbias = sum_rows dy
 *
 * dy and dx have x's dtype and their own row strides; dx (which may be dy), dweight
 * and dbias ([D], wdtype) may be NULL. The sums over rows are formed in fp32 in a
 * fixed order and rounded once. workspace (16-byte aligned):
 * flce_layer_norm_workspace_size() bytes; not needed (may be NULL) when dweight and
 * dbias are both NULL.
 */
int flce_layer_norm_workspace_size(int64_t N, int64_t D, size_t* bytes);
int flce_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int32_t dtype,
                             int64_t ldx, const void* weight, int32_t wdtype, const float* mean,
                             const float* rstd, int64_t N, int64_t D, void* dx, int64_t lddx,
                             void* dweight, void* dbias, void* workspace, size_t ws_bytes,
                             void* stream);

/*
 * The global 2-norm of `count` gradients and their clipping by it:
 *
 *   norm = sqrt(sum over all elements of g^2),  c = min(1, max_norm / (norm + 1e-6)),
 *   out = c g
 *
 *   grads[i]  device pointer of dtypes[i] (FLCE_DTYPE_*) with numel[i] >= 0 elements,
 *             aligned to its element size (the three arrays are host memory, read
 *             before the call returns)
 *   outs      NULL: norm only. Else outs[i] receives the clipped grads[i] (same type
 *             and size); outs[i] may be grads[i], and then, when c = 1, nothing is
 *             written. Other overlaps are not allowed.
 *   norm      fp32 [1] device, the norm before clipping (required)
 *   workspace 16-byte aligned, flce_clip_grads_workspace_size() bytes
 * Squares and their sums are formed in fp32 and joined in fp64 in a fixed order. A
 * norm that is not finite clips as the formula says: infinite gives c = 0 (and NaN
 * where a gradient is infinite), NaN gives NaN everywhere. max_norm >= 0.
 */
int flce_clip_grads_workspace_size(int64_t count, size_t* bytes);
int flce_clip_grads(const void* const* grads, void* const* outs, const int64_t* numel,
                    const int32_t* dtypes, int64_t count, float max_norm, float* norm,
                    void* workspace, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FLCE_OPS_H_ */
