/*
 * matopt_adamw.h -- C ABI of the AdamW step over many tensors at once: for the
 * parameters that are no matrix for opt_group_step (matopt.h) to rotate, such as
 * embeddings, norm weights and biases.
 *
 * Per tensor with gradient G, at step t (counted from 1):
 *   g = scale G                               scale: a device scalar, or 1
 *   m <- beta1 m + (1 - beta1) g
 *   v <- beta2 v + (1 - beta2) g^2            each product and sum rounded to fp32
 *   u  = m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps)
 *   W <- W - lr lr_scale (u + weight_decay W)
 * and the tensor's 16-bit copy, where it has one, is W rounded to nearest even.
 * (Loshchilov, Hutter: "Decoupled weight decay regularization", ICLR 2019.)
 *
 * States of 8 bits. Blocks of 256 consecutive elements of a tensor (the last one
 * may be shorter) share a scale, a power of two: with M the block's largest finite
 * magnitude, 2^(floor(log2 M) - 7) for m and 2^(floor(log2 M) - 14) for v, the
 * exponents held to [-120, 120]. An element is its value over the scale as an OCP
 * 8-bit float, E4M3 for m and E5M2 for v, rounded up in magnitude where the
 * discarded fraction of a step plus r / 65536 reaches 1, down otherwise: at beta2 =
 * 0.999 an average moves by less than half a step of 8 bits, so rounding to nearest
 * would leave it where it is, while the mean of this rounding is the value itself.
 * A v above 0 takes the smallest code above 0 at least: where it became 0 beside an
 * m that does not, the steps after it would divide m by next to nothing. So sqrt(v)
 * counts as 2^-15.5 to 2^-15 of the block's largest at least, and elements whose gradients
 * stay below that move less than with 32 bits.
 * Element i of tensor n takes for r 16 bits of Philox4x32-10 (see opt_dropout) with
 * counter (i / 8, n, offset low, offset high) and key (seed low, seed high): word
 * (i % 8) / 2, its low half for even i; m takes them with their two bytes exchanged.
 * W is updated from m and v before they are rounded. Values that are not finite
 * become NaN.
 *
 * Conventions as in matopt.h: the library allocates no device memory, the tensors
 * and the workspace are the caller's and outlive the group, calls only enqueue
 * kernels on `stream` (they can be captured into a graph), a group is not
 * thread-safe, and calls on one group that overlap on the GPU are the caller's to
 * order (they share the workspace). Nothing is accumulated with atomics.
 */
#ifndef MATOPT_ADAMW_H_
#define MATOPT_ADAMW_H_

#include "matopt_train.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct opt_adamw_s* opt_adamw_t;

#define OPT_ADAMW_BLOCK 256   /* elements to a scale of an 8-bit state */

/* One tensor of n elements, contiguous, with any alignment that its elements have. */
typedef struct {
    int64_t n;                 /* 0 <= n <= 2^35 */
    float* W;                  /* fp32 weights, updated in place */
    const void* G;             /* gradient, read by every step */
    int32_t G_dtype;           /* OPT_F32, OPT_BF16 or OPT_F16 */
    int32_t state_bits;        /* 32: m and v are fp32; 8: as above */
    void *m, *v;               /* start at 0 */
    float *m_scale, *v_scale;  /* 8 bits: ceil(n / 256) each, any finite value at the start (else NULL) */
    void* W16;                 /* 16-bit copy of W, written by every step (NULL: none) */
    int32_t W16_dtype;         /* OPT_BF16 or OPT_F16 */
    float lr_scale, weight_decay;   /* >= 0 */
} opt_adamw_desc;

typedef struct {
    double lr, beta1, beta2, eps;   /* lr >= 0, 0 <= beta < 1, eps > 0 */
} opt_adamw_hparams;

/* Device bytes: the tensors' table and the gradient norm's partial sums. */
opt_status opt_adamw_workspace_size(const opt_adamw_desc* descs, int32_t count, uint64_t* bytes);

/* Checks the tensors (none may overlap, but for gradients with each other) and
 * uploads the table; returns when it is on the device (so the stream may not be
 * captured). t starts at 0. */
opt_status opt_adamw_create(const opt_adamw_desc* descs, int32_t count, const opt_adamw_hparams* hp, void* workspace,
                            uint64_t workspace_bytes, void* stream, opt_adamw_t* out);

/* norm: the 2-norm of all gradients together, its squares summed in 64 bits.
 * scale: what clips it, min(1, max_norm / (norm + 1e-6)); NaN where the norm is
 * not finite. Both are device floats. max_norm > 0 (infinite: scale is 1). */
opt_status opt_adamw_grad_norm(opt_adamw_t g, float max_norm, float* norm, float* scale, void* stream);

/* One step of all tensors. grad_scale: device float (NULL: 1); where it is NaN the
 * step writes nothing, so that a gradient that is not finite can be skipped. rng:
 * for 8-bit states (NULL allowed without any); give each step another offset.
 * device_step: t is read there (one int64 on the device, values below 1 count as 1),
 * for a replayed graph; NULL: the group's counter. The counter is incremented
 * either way. */
opt_status opt_adamw_step(opt_adamw_t g, const float* grad_scale, const opt_rng* rng, const int64_t* device_step,
                          void* stream);
opt_status opt_adamw_get_step(opt_adamw_t g, int64_t* t);
opt_status opt_adamw_set_step(opt_adamw_t g, int64_t t);   /* t >= 0: steps taken so far */
opt_status opt_adamw_set_lr(opt_adamw_t g, double lr);
void opt_adamw_destroy(opt_adamw_t g);

#ifdef __cplusplus
}
#endif

#endif /* MATOPT_ADAMW_H_ */
