// Host-side launch interface of the draft-head training operators.
#pragma once

#include "internal.h"
#include "workspace_order.h"

#include "domino_train.h"

struct domino_train_ctx {
    domino_train_config cfg;
    int device;
    int num_sms;
    int last_launches;
    int* err;             // device error word, and behind it the word that domino_train_status took
    // clusters of each size that the GPU holds at once in distill_step and in logprobs_step (0: not asked yet)
    int step_clusters[17], score_clusters[17];
    // embed_grad workspace (max_tokens > 0)
    uint32_t* keys[2];    // [max_tokens] tokens between the passes of the sort
    int32_t* pos[2];      // [max_tokens] their positions
    unsigned* hist;       // [tiles][kSortMaxBins] digit counts of the sort's tiles (more tokens than a cluster sorts)
    unsigned* named;      // [ceil(V/32)] a bit per row of the table that a token of the call names
    unsigned* claim;      // rows of zeros claimed so far
    float* part;          // [units][2][E] partial sums of the runs that cross a unit's edge
    void* ws_base;
    domino::WorkspaceUse use;  // of embed_grad's workspace
};

namespace domino {
namespace train {

// Lets a kernel be launched with all the shared memory an SM gives one block
// and in clusters of 16, once for all launches.
template <typename K>
cudaError_t allow_all(K kern) {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kern);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(227 * 1024 - a.sharedSizeBytes));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

constexpr int kSortTile = 8192;      // most tokens per tile of the sort
constexpr int kSortMaxCluster = 16;  // tiles that one cluster sorts
constexpr int kSortMaxBins = 1024;   // two digits cover tokens up to DOMINO_TRAIN_MAX_V

struct DistillArgs {
    const void* x;          // [n, V] student logits
    long long ld;
    int n, V;
    const int32_t* ids;     // [n, K]
    const float* top;       // [n, K]
    const float* rest;      // [n] or null
    int K;
    float temperature;
    const float* weight;    // [n] gradient by each row's loss (null: forward only)
    float* loss;            // [n] or null
    float* stats;           // [n, DOMINO_TRAIN_STATS], written by the forward, read by the backward
    void* dx;               // [n, V]
    long long ld_d;
    int* err;
};

struct LogprobArgs {
    const void* x;           // [n, V] logits
    long long ld;
    int n, V;
    const int32_t* tokens;   // [n]
    float temperature;
    float* logprob;          // [n]
    float* entropy;          // [n] or null
    int k;                   // alternatives
    int32_t* alt_ids;        // [n, k]
    float* alt_logprobs;
    float* stats;            // [n, DOMINO_TRAIN_LOGPROB_STATS] or null, written by the forward, read by the backward
    const float* dlogprob;   // [n] or null
    const float* dentropy;   // [n] or null
    void* dx;                // [n, V]
    long long ld_d;
    int* err;
};

cudaError_t prepare_logprob_kernels();
cudaError_t launch_logprobs_forward(domino_train_ctx* c, int dtype, const LogprobArgs& a, cudaStream_t st);
cudaError_t launch_logprobs_backward(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st);
cudaError_t launch_logprobs_step(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st);
cudaError_t prepare_top_kernels();
cudaError_t launch_top(domino_train_ctx* c, const void* x, int dtype, long long ld, int n, int K, float temperature,
                       int32_t* ids, float* top, float* rest, cudaStream_t st);
cudaError_t prepare_distill_kernels();
cudaError_t launch_distill_forward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st);
cudaError_t launch_distill_backward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st);
cudaError_t launch_distill_step(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st);
cudaError_t prepare_embed_kernels();
int max_sum_units(int max_tokens, int num_sms);  // most groups of threads that sum runs in any call
cudaError_t launch_embed(domino_train_ctx* c, const void* table, const int32_t* tokens, int n, float scale, void* out,
                         long long ld, cudaStream_t st);
cudaError_t launch_embed_grad(domino_train_ctx* c, const void* dout, long long ld, const int32_t* tokens, int n,
                              float scale, void* dtable, int grad_dtype, bool accumulate, cudaStream_t st);

}  // namespace train
}  // namespace domino
