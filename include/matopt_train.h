/*
 * matopt_train.h -- C ABI of the training-pass operators: what produces the
 * gradients that opt_group_step (matopt.h) consumes.
 *
 *   attention        O = softmax(scale Q K^T) V with its backward pass, which
 *                    recomputes the probabilities from the saved log-sums
 *   layer norm       with the residual sum and dropout in the same pass, and
 *                    the backward pass with the weight's and bias's gradients
 *   rotary           position rotation of queries and keys, and its gradient
 *   qk norm          norms of queries and keys per head with the rotation in
 *                    the same pass, and the backward pass with the weights'
 *                    gradients
 *   dropout          from a counter-based generator; no mask is stored
 *   policy loss      clipped policy-gradient loss with a KL term on logits,
 *                    forward, backward, or both in one pass over the logits
 *
 * Conventions, besides those of matopt.h (errors, streams, no allocation, no
 * host synchronisation):
 *  - Tensors are device memory of the current device; strides are in elements
 *    and may not be negative. Outputs overlap no other tensor unless a call
 *    says so.
 *  - Nothing is accumulated with atomics: equal inputs give bitwise equal
 *    outputs.
 *  - Sums, statistics and probabilities are held in fp32; a value is rounded
 *    to 16 bits where it is stored and where it enters a matrix instruction
 *    (the probabilities and the score gradients).
 *  - Every call can be captured into a graph: kernels only, no memset or copy.
 */
#ifndef MATOPT_TRAIN_H_
#define MATOPT_TRAIN_H_

#include "matopt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* IEEE half precision, next to OPT_F32 and OPT_BF16, for these operators only. */
enum { OPT_F16 = 2 };

/* ------------------------------------------------------------ attention ----
 *
 * Per sequence b and head h (key head h / (heads / kv_heads)):
 *   S = scale Q K^T,   L_i = log sum_j exp(S_ij) over the keys query i sees
 *   P = exp(S - L),    O = P V
 * and backward, from O, L and dO:
 *   D_i = sum_d dO_id O_id,   dP = dO V^T,   dS = P (dP - D)
 *   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
 * dK and dV sum over the heads that share a key head.
 *
 * Query i of n_q sees key j of n_k where j < n_k, with causal also
 * j <= i + n_k - n_q (the last query sees the last key), and with window > 0,
 * which needs causal, also j > i + n_k - n_q - window or, with sinks > 0, j <
 * sinks: a sequence's first keys stay in sight of all later queries. A query that sees no
 * key has O = 0, L = -inf, dQ = 0. Keys and queries past a sequence's length
 * are not read, whatever they hold; a non-finite key or value inside the
 * length may reach a query whose causal bound or window hides it, and a
 * non-finite query or dO a key it does not see (0 times infinity).
 *
 * P and dS enter matrix instructions in dtype. OPT_F16 holds dS in steps of
 * 2^-24 below 2^-14 and up to 65504, as it does dQ, dK and dV: scale the loss
 * so that they lie between. (P is kept clear of both.) Scores S are fp32, which
 * tells them apart up to 2^24.
 */
typedef struct {
    int32_t dtype;            /* OPT_BF16 or OPT_F16: every tensor but lse */
    int32_t batch, heads, kv_heads;   /* heads a multiple of kv_heads */
    int32_t head_dim;         /* a multiple of 8, at most 128 */
    int32_t q_len, k_len;     /* tokens per sequence; packed: the longest sequence; at most 2^29 */
    int32_t causal, window;   /* window: 0 for none */
    float scale;
    /* Packed sequences: batch + 1 ascending device offsets into the token
     * axis (then batch strides are unused). Both or neither. Tokens outside
     * every sequence, and past the first q_len or k_len of a longer one, are
     * not read; outputs and gradients are written there as zeros (L: -inf). */
    const int32_t* q_start;
    const int32_t* k_start;
    int64_t q_tokens, k_tokens;       /* packed: rows of the token axes */
    /* Padded batches: device lengths per sequence, at most q_len and k_len
     * (NULL: full). Outputs past a length are written as zeros (L: -inf).
     * Not together with q_start. */
    const int32_t* q_lens;
    const int32_t* k_lens;
    int32_t sinks;            /* 0 for none; needs a window */
} opt_attention_desc;

/* A tensor (batch, tokens, heads, head_dim), the last axis contiguous;
 * strides are multiples of 8 and data is 16-byte aligned. */
typedef struct {
    const void* data;
    int64_t batch_stride, token_stride, head_stride;
} opt_attention_tensor;

/* Scratch of one call (backward: 0 or 1), 256-byte aligned device memory. */
opt_status opt_attention_workspace_size(const opt_attention_desc* a, int32_t backward, uint64_t* bytes);
/* lse: fp32, heads x (batch * q_len), packed: heads x q_tokens. */
opt_status opt_attention_forward(const opt_attention_desc* a, const opt_attention_tensor* q,
                                 const opt_attention_tensor* k, const opt_attention_tensor* v,
                                 const opt_attention_tensor* out, float* lse, void* workspace,
                                 uint64_t workspace_bytes, void* stream);
opt_status opt_attention_backward(const opt_attention_desc* a, const opt_attention_tensor* dout,
                                  const opt_attention_tensor* q, const opt_attention_tensor* k,
                                  const opt_attention_tensor* v, const opt_attention_tensor* out, const float* lse,
                                  const opt_attention_tensor* dq, const opt_attention_tensor* dk,
                                  const opt_attention_tensor* dv, void* workspace, uint64_t workspace_bytes,
                                  void* stream);

/* --------------------------------------------------------------- rotary ----
 *
 * Pair i of a head at position p turns by the angle p f_i:
 *   (a, b) -> scale (a cos - b sin, b cos + a sin)
 * Layout HALF pairs element i with i + rot / 2, PAIRS 2 i with 2 i + 1; the
 * elements from rot on stay as they are (unscaled). The gradient is the same call
 * with inverse set: it turns by -p f_i.
 *
 * Frequencies are given as turns[i] = round(2^64 f_i / (2 pi)) mod 2^64, so that
 * p turns[i] mod 2^64 is the angle in 2^-64 turns, exact but for that rounding
 * (|p| 2^-65 turns). Angles, sines and the rotation are fp32 (the fraction of a
 * turn is cut at 2^-32); y is rounded once.
 */
enum { OPT_ROTARY_HALF = 0, OPT_ROTARY_PAIRS = 1 };
typedef struct {
    const uint64_t* turns;     /* rot / 2, device */
    int32_t rot, layout;       /* rot even, 2 <= rot <= head_dim */
    float scale;               /* > 0: of cosine and sine */
    int32_t positions_i64;     /* positions are int64_t (else int32_t); any value */
    const void* positions;     /* device, (batch, tokens) by strides >= 0; NULL: first + index along the tokens */
    int64_t position_batch_stride, position_token_stride, first;
} opt_rotary;

/* Queries (batch, tokens, heads, head_dim) and keys (kv_heads; 0: no keys, and
 * what belongs to them is ignored). Tensors have strides in elements, a contiguous
 * last axis and one element's alignment; opt_attention_tensor describes them. */
typedef struct {
    int32_t dtype;             /* OPT_F32, OPT_BF16 or OPT_F16, of all but weights and statistics */
    int32_t heads, kv_heads, head_dim;   /* heads, kv_heads <= 65536, head_dim <= 512 */
    int64_t batch, tokens;     /* batch * tokens < 2^31 */
} opt_heads_desc;

/* yq may be q and yk may be k (same strides); results that overlap these tensors or each
 * other otherwise are refused. */
opt_status opt_rotary_apply(const opt_heads_desc* d, const opt_rotary* r, int32_t inverse, const opt_attention_tensor* q,
                            const opt_attention_tensor* k, const opt_attention_tensor* yq,
                            const opt_attention_tensor* yk, void* stream);

/* -------------------------------------------------------------- qk norm ----
 *
 *   y = R(x rstd w),  rstd = 1 / sqrt(mean(x^2) + eps) over a head's elements
 * backward, with R the rotation of opt_rotary_apply (r NULL: none):
 *   g = R^T dy,  z = g w,  xh = x rstd,  dx = rstd (z - xh mean(z xh)),  dw = sum g xh
 * Weights (head_dim) and their gradients are fp32, one for all heads of q and one
 * for those of k; rstd is fp32, (batch, tokens, heads) contiguous. yq may be q, dq
 * may be dyq or q (same strides), and so for k; results of the tensors' type that
 * overlap them or each other otherwise are refused. The fp32 results and the workspace
 * overlap nothing.
 */
opt_status opt_qk_norm_forward(const opt_heads_desc* d, const opt_rotary* r, const opt_attention_tensor* q,
                               const opt_attention_tensor* k, const float* q_weight, const float* k_weight, float eps,
                               const opt_attention_tensor* yq, const opt_attention_tensor* yk, float* q_rstd,
                               float* k_rstd, void* stream);
opt_status opt_qk_norm_workspace_size(const opt_heads_desc* d, uint64_t* bytes);   /* backward; 256-byte aligned */
opt_status opt_qk_norm_backward(const opt_heads_desc* d, const opt_rotary* r, const opt_attention_tensor* dyq,
                                const opt_attention_tensor* dyk, const opt_attention_tensor* q,
                                const opt_attention_tensor* k, const float* q_weight, const float* k_weight,
                                const float* q_rstd, const float* k_rstd, const opt_attention_tensor* dq,
                                const opt_attention_tensor* dk, float* dq_weight, float* dk_weight, void* workspace,
                                uint64_t workspace_bytes, void* stream);

/* -------------------------------------------------------------- dropout ----
 *
 * Element (r, c) of a rows x cols tensor takes 16 bits of Philox4x32-10
 * (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2,
 * 3", SC 2011) with counter (c / 8, r, offset low, offset high) and key
 * (seed low, seed high): word (c % 8) / 2, its low half for even c. With
 * t = round(65536 p) the element is dropped where the bits are below t and
 * multiplied by 65536 / (65536 - t) otherwise, so its mean is kept exactly.
 * The mask depends on position, seed and offset only, not on strides or
 * types: the backward pass is the same call on the gradient.
 */
typedef struct {
    uint64_t seed, offset;
    const uint64_t* device_offset;   /* added to offset when not NULL: a step counter that a replayed graph reads */
} opt_rng;

/* y = residual + dropout(x) (residual NULL: none; y may be x or residual);
 * dtype OPT_F32, OPT_BF16 or OPT_F16 for all three; 0 <= p < 1; row strides
 * ld*; rows < 2^32, cols < 2^34. rng may be NULL where p is 0. */
opt_status opt_dropout(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, void* y, int64_t ldy, float p, const opt_rng* rng, void* stream);

/* ----------------------------------------------------------- layer norm ----
 *
 *   h = residual + dropout(x)     product and sum rounded to fp32, then to h's type
 *   y = (h - mean) rstd weight + bias,   rstd = 1 / sqrt(var + eps), of the stored h
 * backward:
 *   z = dy weight,  xh = (h - mean) rstd
 *   g = rstd (z - mean(z) - xh mean(z xh)) + dh     dh: what reaches h past the norm
 *   dx = dropout'(g),  dres = g,  dweight = sum dy xh,  dbias = sum dy
 *
 * cols <= OPT_MAX_DIM. weight, bias, mean, rstd and their gradients are fp32;
 * x, y, dy, dx have dtype; residual, h, dh, dres have h_dtype, which is dtype
 * or OPT_F32. Without residual and dropout h is x itself: pass h = NULL (and
 * x as h to the backward call). bias, dbias, dh and dres may be NULL. h may
 * be residual, y may be x, dx may be dy and dres may be dh.
 */
opt_status opt_layer_norm_forward(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx,
                                  int32_t h_dtype, const void* residual, int64_t ldr, const float* weight,
                                  const float* bias, float eps, float p, const opt_rng* rng, void* y, int64_t ldy,
                                  void* h, int64_t ldh, float* mean, float* rstd, void* stream);
opt_status opt_layer_norm_workspace_size(int64_t rows, int64_t cols, uint64_t* bytes);   /* backward; 256-byte aligned */
opt_status opt_layer_norm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t lddy,
                                   int32_t h_dtype, const void* h, int64_t ldh, const void* dh, int64_t lddh,
                                   const float* weight, const float* mean, const float* rstd, float p,
                                   const opt_rng* rng, void* dx, int64_t lddx, void* dres, int64_t lddres,
                                   float* dweight, float* dbias, void* workspace, uint64_t workspace_bytes,
                                   void* stream);

/* ---------------------------------------------------------- policy loss ----
 *
 * Per row i of logits, with z = logit_scale * logits and target t:
 *   lse = log sum_j exp(z_j),  logp = z_t - lse
 *   r = exp(logp - old_logp),  d = ref_logp - logp
 *   loss = sum_i weight_i (max(-A r, -A clip(r, 1 - clip_low, 1 + clip_high)) + kl_coef (exp(d) - d - 1))
 *   slope_i = weight_i ([the unclipped term is the larger or equal] (-A r) + kl_coef (1 - exp(d)))
 *   dlogits_ij = grad logit_scale slope_i ([j = t] - exp(z_j - lse))
 * The weights hold the normalisation (mask / tokens, for a mean over tokens).
 * A row of weight 0 is not read: logp = lse = slope = 0 and its dlogits are
 * zeros, whatever its logits and target hold. Elsewhere a target outside
 * [0, vocab) makes the row's results and the loss NaN, and a NaN among the
 * row's other inputs its slope, its dlogits and the loss.
 */
typedef struct {
    int32_t dtype;             /* of logits and dlogits: OPT_F32, OPT_BF16 or OPT_F16 */
    int32_t target_i64;        /* targets are int64_t (else int32_t) */
    int64_t rows, vocab;       /* rows < 2^31, vocab < 2^31 - 2^16; backward: vocab <= 2^29 - 2^13 */
    int64_t ld;                /* row stride of logits */
    float logit_scale, clip_low, clip_high, kl_coef;
    /* rows floats (may be NULL): lse is rounded to fp32, off by up to
     * 2^-24 |lse|, and this is what the rounding left out. The forward call
     * writes it; the backward call, given the same, forms exp(z_j - lse)
     * without that error, which an offset common to the logits enlarges. */
    float* lse_rest;
} opt_policy_desc;

/* Per-row inputs: target, old_logp, advantage, weight and, unless kl_coef is
 * 0, ref_logp (else it may be NULL). */
typedef struct {
    const void* target;
    const float *old_logp, *ref_logp, *advantage, *weight;
} opt_policy_rows;

opt_status opt_policy_loss_workspace_size(const opt_policy_desc* a, uint64_t* bytes);   /* 256-byte aligned */
/* Writes loss (one float), logp, lse and slope (rows each). */
opt_status opt_policy_loss_forward(const opt_policy_desc* a, const void* logits, const opt_policy_rows* in,
                                   float* loss, float* logp, float* lse, float* slope, void* workspace,
                                   uint64_t workspace_bytes, void* stream);
/* dlogits (row stride ldd, may be logits) from what the forward call wrote;
 * grad: device scalar, the loss's own gradient (NULL: 1). */
opt_status opt_policy_loss_backward(const opt_policy_desc* a, const void* logits, const void* target,
                                    const float* lse, const float* slope, const float* grad, void* dlogits,
                                    int64_t ldd, void* stream);
/* Both in one pass over the logits, for a loss that is the last operator:
 * grad is known on the host. logp as in the forward call (may be NULL). */
opt_status opt_policy_loss_step(const opt_policy_desc* a, const void* logits, const opt_policy_rows* in, float grad,
                                float* loss, float* logp, void* dlogits, int64_t ldd, void* workspace,
                                uint64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MATOPT_TRAIN_H_ */
