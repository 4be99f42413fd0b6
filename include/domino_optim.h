/*
 * domino_optim.h - C ABI of the weights' update on GB300 (sm_103a), beside the
 * training operators of domino_train.h (same library, same status codes and
 * dtypes).
 *
 *   adamw_step       one AdamW step over many tensors at once, with moments in
 *                    32 bits or in 8;
 *   adamw_grad_norm  the norm of all their gradients and the factor that clips it.
 *
 * Conventions.  All tensors are DEVICE pointers to contiguous elements, owned by
 * the caller, aligned to their element; tensors whose elements start on 32-byte
 * boundaries run fastest.  No two of them may overlap.  Calls are asynchronous on
 * `cuda_stream` (NULL = legacy default stream), make no host synchronisation and
 * allocate nothing, so they can be captured into a CUDA graph after one ordinary
 * call: the step's number is counted on the device.  A context may be used from
 * one host thread at a time, on any streams; its calls run one after another on
 * the device (each waits for an event of the last one; inside a graph capture, of
 * the last one of that capture).  A replayed graph does not take part in this:
 * the caller orders replays with the context's other calls and replays.  Results
 * do not depend on the launch: repeated calls on equal inputs give equal bits.
 *
 * Flat layout.  The moments (and the master copy) of all tensors lie in one
 * buffer each: tensor i begins at position at_i = sum over j < i of n_j rounded
 * up to DOMINO_ADAMW_BLOCK, and the buffers hold the total of that.  What lies
 * between two tensors is neither read nor written.
 */
#ifndef DOMINO_OPTIM_H
#define DOMINO_OPTIM_H

#include "domino_rollout.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct domino_adamw_ctx domino_adamw_ctx;

#define DOMINO_ADAMW_BLOCK 128            /* elements that share a scale */
#define DOMINO_ADAMW_MAX_TENSORS 65536    /* of one context              */

/* A tensor to update: n >= 0 elements of dtype DOMINO_DTYPE_*.  master = 1 (bf16
 * only): its exact value is held in the flat fp32 buffer `master`, and the tensor
 * gets that value rounded to nearest. */
typedef struct {
    void* param;
    long long n;
    int dtype;
    int master;
} domino_adamw_tensor;

/* state_bits 32: m and v are flat fp32 buffers.  state_bits 8: flat buffers of
 * e4m3 codes, with one fp32 scale per block of DOMINO_ADAMW_BLOCK positions in
 * m_scale and v_scale: a moment is its code's value times its block's scale.  m, v
 * and master are aligned to 32 bytes.  All
 * zero at the start.  count: the steps taken so far, device, 8-byte aligned.
 * 0 <= beta1, beta2 < 1; 1e-16 <= eps <= 1; 0 <= weight_decay <= 1. */
typedef struct {
    int n_tensors;
    const domino_adamw_tensor* tensors;
    int state_bits;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    float* master;
    long long* count;
    double beta1, beta2, eps, weight_decay;
    unsigned seed;
} domino_adamw_config;

/* Create a context on CUDA device `device` over these tensors and buffers, which
 * are used as they are from then on.  *out receives the context (NULL on failure).
 * Errors: INVALID_ARG (null or misaligned pointer, a number out of range, tensors
 * that overlap), UNSUPPORTED (state_bits, dtype), CUDA, OOM. */
DOMINO_API int domino_adamw_init(domino_adamw_ctx** out, const domino_adamw_config* cfg, int device);

/* One step.  grads [n_tensors] host array of device pointers to the tensors'
 * gradients, of grad_dtypes [n_tensors] (host); NULL (or n = 0): the tensor is left as it
 * is.  With t = *count + 1, g' = *scale g (scale NULL: 1) and
 * rate = lr * *lr_factor (lr_factor NULL: 1), scale and lr_factor on the device:
 *   m = beta1 m + (1 - beta1) g'
 *   v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - rate weight_decay)
 *       - rate / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32, every product and sum of m and v rounded by itself (so that their codes
 * can be reproduced), p from m and v before they are narrowed (the root of a v below
 * 2^-126 counts as 0); then *count = t.  What is taken from p, decay and update together,
 * is formed by itself and subtracted with one rounding to fp32: it is as good as fp32
 * holds it at its own size, and lost only where it is below 2^-25 |p|.  An infinite p stays
 * as it is.  Where *scale is not finite the whole step is left out, count included.
 * Gradients that are not finite spoil their elements (with 8 bits: their blocks) for good.
 *
 * What is held in fewer than 32 bits, and has no exact copy, is rounded
 * stochastically, so that changes below a rounding step add up over the steps:
 * bf16 parameters without master, and 8-bit moments.  A block's scale is
 * max(largest |a| * (1 / 448), 2^-120); |a| / scale, at most 448, goes to one of
 * its two neighbours in e4m3, up with the probability of its place between them;
 * a v that is not 0 is never rounded to 0.  The random bits of position i in step
 * t are a function of (seed, t, i) alone, modulo 2^32:
 *   mix(h): h ^= h >> 15, h *= 0x6A09E667, h ^= h >> 13, h *= 0xBB67AE85, h ^ h >> 16
 *   key = mix(mix(t + 0x9E3779B9) + seed)
 *   h = mix(i * 0x9E3779B9 + (i >> 32) * 0x3C6EF373 + key)
 * of which m takes the lowest 20 bits, v the highest 20, the parameter bits 4 to
 * 19.  0 <= lr <= 1e3.  Errors: INVALID_ARG, UNSUPPORTED (dtype), CUDA. */
DOMINO_API int domino_adamw_step(domino_adamw_ctx* ctx, const void* const* grads, const int* grad_dtypes, double lr,
                                 const float* lr_factor, const float* scale, void* cuda_stream);

/* *norm = sqrt(sum of g^2 over the elements of all gradients), squares and sums of up to
 * four of them in fp32 (an element past 1.8e19 makes the norm infinite, one below 2e-23
 * adds nothing), sums of those in twice its precision, in an order that the sizes fix:
 * off by at most 2^-23 of itself where elements above 1.1e-19, whose squares are normal
 * numbers, make it up;
 * *scale = min(1, max_norm / (*norm + 1e-6)), NaN where the norm is not finite (so
 * that a step with this scale is left out).  Both on the device; scale may be
 * NULL.  grads and grad_dtypes as in domino_adamw_step; max_norm > 0.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype), CUDA. */
DOMINO_API int domino_adamw_grad_norm(domino_adamw_ctx* ctx, const void* const* grads, const int* grad_dtypes,
                                      float max_norm, float* norm, float* scale, void* cuda_stream);

/* Kernel launches the last successful call enqueued. */
DOMINO_API int domino_adamw_last_launch_count(const domino_adamw_ctx* ctx);

/* Free the context and its workspace (NULL is ignored), after a device sync. */
DOMINO_API void domino_adamw_destroy(domino_adamw_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* DOMINO_OPTIM_H */
