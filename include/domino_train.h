/*
 * domino_train.h - C ABI of the draft-head training operators on GB300
 * (sm_103a), beside the rollout of domino_rollout.h (same library, same
 * status codes and dtypes).
 *
 * A draft head is trained on the target model's logits.  Four operators:
 *
 *   top_logits   boils each row of the teacher's logits down to a record: the
 *                K largest logits, their ids, and the log-sum-exp of the rest;
 *   distill_*    the divergence of the student's distribution from that
 *                record, and its gradient by the student's logits;
 *   logprobs_*   the log probability of each row's token, the row's entropy and
 *                its most likely alternatives, and the gradient of the first two;
 *   embed*       the scaled embedding lookup (the GRU's input) and the
 *                gradient of its table.
 *
 * The weights' update and the gradients' norm are in domino_optim.h.
 *
 * Conventions.  All tensors are DEVICE pointers, row-major, owned by the
 * caller; `ld` arguments are row strides in elements.  Any pointer aligned to
 * its element and any ld >= the row's length is accepted; rows that start on
 * 16-byte boundaries run fastest.  Outputs must not overlap inputs.  Calls are
 * asynchronous on `cuda_stream` (a cudaStream_t, NULL = legacy default
 * stream), make no host synchronisation and allocate nothing, so they can be
 * captured into a CUDA graph after one ordinary call.  A context may be used
 * from one host thread at a time, on any streams.  embed_grad uses the
 * context's workspace: its calls on one context run one after another on the
 * device, whatever their streams (each waits for an event of the last one;
 * inside a graph capture, of the last one of that capture).  A replayed graph
 * does not take part in this: the caller orders the replay of a graph that
 * holds embed_grad with the context's other embed_grad calls and replays.
 * Results do not depend on the launch: repeated calls on equal inputs give
 * equal bits.  Sums and softmax statistics are held in fp32.
 *
 * Ids and tokens are int32.  -1 is padding: it takes no part.  Any other value
 * outside [0, V) is treated as padding too and raises DOMINO_ERR_BAD_TOKEN at
 * the next domino_train_status().
 */
#ifndef DOMINO_TRAIN_H
#define DOMINO_TRAIN_H

#include "domino_rollout.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct domino_train_ctx domino_train_ctx;

#define DOMINO_TRAIN_MAX_V 524288 /* largest vocabulary                      */
#define DOMINO_TRAIN_MAX_K 8192   /* largest record                          */
#define DOMINO_TRAIN_MAX_TOKENS 4194304 /* tokens of one embed_grad call   */
#define DOMINO_TRAIN_STATS 8      /* floats per row of distill_forward's stats */
#define DOMINO_TRAIN_MAX_ALTERNATIVES 32 /* of logprobs_forward              */
#define DOMINO_TRAIN_LOGPROB_STATS 4     /* floats per row of its stats      */

/* V vocabulary (2 .. DOMINO_TRAIN_MAX_V); E embedding width (0: the embedding
 * entry points are not used); max_tokens (0 .. DOMINO_TRAIN_MAX_TOKENS) sizes the workspace of embed_grad
 * (0: not used); dtype (DOMINO_DTYPE_*) of the student's logits and their
 * gradient, of the embedding table and of embedding rows. */
typedef struct {
    int V, E;
    int max_tokens;
    int dtype;
} domino_train_config;

/* Create a context on CUDA device `device`, with its workspace.  *out receives
 * the context (NULL on failure).  Errors: INVALID_ARG (null pointer, a size out
 * of range), UNSUPPORTED (V > DOMINO_TRAIN_MAX_V, unknown dtype), CUDA, OOM. */
DOMINO_API int domino_train_init(domino_train_ctx** out, const domino_train_config* cfg, int device);

/* Teacher's record.  logits [n_rows, V] of dtype `dtype` (the teacher's own,
 * whatever the context's).  Per row:
 *   ids  [n_rows, K]  the K ids with the largest logits, ascending; ties to
 *                     the lower id; -0.0 equals +0.0; NaN counts as largest
 *   top  [n_rows, K]  their logits, fp32 (unscaled)
 *   rest [n_rows]     log sum exp(logit / temperature) over all other ids,
 *                     fp32; -inf when they hold no mass (all -inf, or K = V)
 * 1 <= K <= min(V, DOMINO_TRAIN_MAX_K); 1e-3 <= temperature <= 1e3.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype), CUDA. */
DOMINO_API int domino_train_top_logits(domino_train_ctx* ctx, const void* logits, int dtype, long long ld, int n_rows,
                                       int K, float temperature, int32_t* ids, float* top, float* rest,
                                       void* cuda_stream);

/* Distillation loss of the rows of student logits x [n_rows, V] (context
 * dtype) from a teacher's record (ids, top [n_rows, K] contiguous, any order;
 * rest [n_rows], or NULL for -inf: the record is the whole distribution).
 * With S the record's ids (-1 left out, a repeated id counted once, at its first place):
 *   L   = log(sum_S exp(top_k / T) + exp(rest)),  p_k = exp(top_k / T - L),
 *   p_r = exp(rest - L),  z = log sum_v exp(x_v / T),  q_v = exp(x_v / T - z),
 *   q_r = sum_{v not in S} q_v,
 *   loss = sum_S p_k (log p_k - log q_k) + p_r (log p_r - log q_r)
 * (0 log 0 = 0).  A row whose record holds no mass (L = -inf) has loss 0.  A row
 * with a target whose own logits are all -inf has no q: its loss is NaN.  What
 * all logits of a row share cancels, up to the type's lowest value.  With K = 1
 * and no rest the loss is the cross entropy with the label ids[n] (any finite
 * top), and -1 is an ignored position.
 * stats [n_rows, DOMINO_TRAIN_STATS] fp32 is what distill_backward needs.
 * 1 <= K <= DOMINO_TRAIN_MAX_K; 1e-3 <= temperature <= 1e3.
 * Errors: INVALID_ARG, CUDA. */
DOMINO_API int domino_train_distill_forward(domino_train_ctx* ctx, const void* logits, long long ld, int n_rows,
                                            const int32_t* ids, const float* top, const float* rest, int K,
                                            float temperature, float* loss, float* stats, void* cuda_stream);

/* Gradient: dlogits [n_rows, V] (context dtype, row stride ld_d), written whole,
 *   dlogits_v = dloss / T * (q_v - p_v)            v in S
 *             = dloss / T * q_v (1 - p_r / q_r)    otherwise
 * with dloss [n_rows] fp32 the gradient by each row's loss and stats from
 * distill_forward on the same inputs.  A row with dloss 0, or whose record
 * holds no mass, gets zeros whatever its logits.  Where the loss is +inf
 * because q_r = 0 < p_r, the ids outside the record get 0.
 * Errors: INVALID_ARG, CUDA. */
DOMINO_API int domino_train_distill_backward(domino_train_ctx* ctx, const void* logits, long long ld, int n_rows,
                                             const int32_t* ids, const float* top, const float* rest, int K,
                                             float temperature, const float* stats, const float* dloss, void* dlogits,
                                             long long ld_d, void* cuda_stream);

/* Loss and gradient in one call, for a training step that knows its rows'
 * weights: loss as distill_forward writes it (not multiplied by the weight; 0
 * for a row of weight 0, which is skipped), dlogits as distill_backward with
 * dloss = weight.  Errors: INVALID_ARG, CUDA. */
DOMINO_API int domino_train_distill_step(domino_train_ctx* ctx, const void* logits, long long ld, int n_rows,
                                         const int32_t* ids, const float* top, const float* rest, int K,
                                         float temperature, const float* weight, float* loss, void* dlogits,
                                         long long ld_d, void* cuda_stream);

/* Scores of the rows of logits x [n_rows, V] of dtype `dtype` (whatever the
 * context's), one token each.  With T = temperature, q_v = exp(x_v / T - z) and
 * z = log sum_v exp(x_v / T):
 *   logprob [n_rows]  log q_t of t = tokens[n]
 *   entropy [n_rows]  -sum_v q_v log q_v (NULL: not written)
 *   alt_ids, alt_logprobs [n_rows, n_alternatives]  the ids with the largest
 *       logits, largest first, ties to the lower id, -0.0 equal to +0.0, NaN
 *       largest, and their log q.  Ids whose logit is -inf are no alternatives:
 *       places that remain hold -1 and -inf
 *   stats [n_rows, DOMINO_TRAIN_LOGPROB_STATS]  what logprobs_backward needs
 *       (NULL: not written)
 * 0 <= n_alternatives <= min(V, DOMINO_TRAIN_MAX_ALTERNATIVES); at 0 the two
 * arrays may be NULL.  1e-3 <= temperature <= 1e3.
 * A row whose token is -1 takes no part, whatever its logits: 0, 0 and
 * no alternatives.  A row without a logit above -inf has no distribution: -inf,
 * 0 and no alternatives.  A row with a NaN or +inf logit gets NaN for all its
 * floats.  What all logits of a row share cancels, up to the type's lowest value.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype), CUDA. */
DOMINO_API int domino_train_logprobs_forward(domino_train_ctx* ctx, const void* logits, int dtype, long long ld,
                                             int n_rows, const int32_t* tokens, float temperature, float* logprob,
                                             float* entropy, int n_alternatives, int32_t* alt_ids, float* alt_logprobs,
                                             float* stats, void* cuda_stream);

/* Gradient: dlogits [n_rows, V] (context dtype, row stride ld_d), written whole,
 *   dlogits_v = 1 / T * (dlogprob ([v = t] - q_v) - dentropy q_v (log q_v + entropy))
 * with dlogprob and dentropy [n_rows] fp32 the gradients by each row's two values
 * (NULL: zeros; one of them at least is given) and stats from logprobs_forward on
 * the same inputs in the context's dtype.  A row with both 0, without
 * distribution, or whose token is -1 gets zeros whatever its logits.
 * Errors: INVALID_ARG, CUDA. */
DOMINO_API int domino_train_logprobs_backward(domino_train_ctx* ctx, const void* logits, long long ld, int n_rows,
                                              const int32_t* tokens, float temperature, const float* stats,
                                              const float* dlogprob, const float* dentropy, void* dlogits,
                                              long long ld_d, void* cuda_stream);

/* Scores and gradient in one call, for a training step that knows its rows'
 * weights: logprob and entropy as logprobs_forward writes them (not multiplied;
 * 0 for a row whose weights are both 0, which is skipped), dlogits as
 * logprobs_backward with dlogprob = weight and dentropy = entropy_weight (either
 * may be NULL: zeros, but not both).  Errors: INVALID_ARG, CUDA. */
DOMINO_API int domino_train_logprobs_step(domino_train_ctx* ctx, const void* logits, long long ld, int n_rows,
                                          const int32_t* tokens, float temperature, const float* weight,
                                          const float* entropy_weight, float* logprob, float* entropy, void* dlogits,
                                          long long ld_d, void* cuda_stream);

/* out[i, :] = scale * table[tokens[i], :] in the context dtype (the product is
 * formed in fp32 and rounded once); zeros for padding.  table [V, E]
 * contiguous, out [n_tokens, E] with row stride ld_out.  Any n_tokens.
 * Errors: INVALID_ARG (E = 0 in the config too), CUDA. */
DOMINO_API int domino_train_embed(domino_train_ctx* ctx, const void* table, const int32_t* tokens, int n_tokens,
                                  float scale, void* out, long long ld_out, void* cuda_stream);

/* Gradient of the table: dtable[v, :] = scale * sum of dout[i, :] over the i
 * with tokens[i] = v, summed in fp32, in an order fixed by the sorted tokens.
 * dout [n_tokens, E] in the context dtype with row stride ld; dtable [V, E]
 * contiguous, fp32 or bf16 (grad_dtype).  accumulate = 0 writes every row of
 * dtable (zeros for tokens that do not occur); accumulate = 1 adds to the rows
 * of the tokens that occur and leaves the others alone.
 * 0 <= n_tokens <= max_tokens.  Errors: INVALID_ARG, UNSUPPORTED (grad_dtype), CUDA. */
DOMINO_API int domino_train_embed_grad(domino_train_ctx* ctx, const void* dout, long long ld, const int32_t* tokens,
                                       int n_tokens, float scale, void* dtable, int grad_dtype, int accumulate,
                                       void* cuda_stream);

/* Take the device error word in the order of `cuda_stream`, leave 0 in its
 * place, synchronise that stream (no other) and return the word's status
 * (DOMINO_OK, DOMINO_ERR_BAD_TOKEN, or DOMINO_ERR_TIMEOUT after a device-side
 * wait of a distillation or scoring call ran out of time: all outputs of that call are
 * undefined, rows unwritten among them, and it has to be made again), or
 * DOMINO_ERR_CUDA. */
DOMINO_API int domino_train_status(domino_train_ctx* ctx, void* cuda_stream);

/* Kernel launches the last successful operator call enqueued. */
DOMINO_API int domino_train_last_launch_count(const domino_train_ctx* ctx);

/* Free the workspace and the context (NULL is ignored), after a device sync. */
DOMINO_API void domino_train_destroy(domino_train_ctx* ctx);

#ifdef __cplusplus
}
#endif
#endif /* DOMINO_TRAIN_H */
