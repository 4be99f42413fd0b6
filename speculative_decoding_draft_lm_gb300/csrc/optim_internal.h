// Host-side launch interface of the weights' update.
#pragma once

#include "internal.h"
#include "workspace_order.h"

#include "domino_optim.h"

namespace domino {
namespace optim {

// elements that a CTA takes at once, in each kernel
constexpr int kTile8 = 4096, kTile32 = 2048, kNormTile = 4096;
constexpr int kMaxPerLaunch = 1000;  // tensors

// A tensor of one launch, as the kernels' parameters hold it.
struct alignas(16) Entry {
    void* p;
    const void* g;
    unsigned long long n;  // elements, and what they are in the top bits
    unsigned tile;         // its first tile in the launch
    unsigned block;        // its first block of DOMINO_ADAMW_BLOCK positions
};
constexpr unsigned long long kElements = (1ull << 48) - 1;
constexpr unsigned long long kParamBf16 = 1ull << 48, kMaster = 1ull << 49, kGradBf16 = 1ull << 50;
constexpr long long kMaxElements = 1ll << 38;  // of one context: tiles and blocks in 32 bits

struct Work {
    int tensors;
    unsigned tiles;
    unsigned long long kind;  // of all its tensors, as in Entry::n (0 for the norm)
    Entry* entry;  // host, [tensors]
};

struct AdamArgs {
    void *m, *v;
    float *m_scale, *v_scale, *master;
    long long* count;
    const float* scale;
    const float* lr_factor;
    unsigned* ticket;
    // twice each, as the packed operations take them; rest: 1 - beta; one: 1
    float2 beta1, beta2, rest1, rest2, eps, one;
    float lr, decay, log_beta1, log_beta2;
    unsigned seed;
    unsigned golden, up12;  // factors that the compiler does not know
    int last;  // the step's last launch: the one that counts it
};

struct NormArgs {
    float2* part;      // a partial sum per CTA of the call
    unsigned* ticket;
    unsigned first, ctas;  // of this launch, and of the call
    double max_norm;
    float *norm, *scale;
};

}  // namespace optim
}  // namespace domino

struct domino_adamw_ctx {
    domino_adamw_config cfg;  // its tensors: this context's copy
    int device, num_sms;
    int last_launches;
    domino_adamw_tensor* tensors;
    unsigned* block;               // [n_tensors] first block of each
    domino::optim::Entry* entry;   // [kMaxPerLaunch] of the launch that is being put together
    unsigned* ticket;              // device: CTAs of a call that are done
    float2* part;                  // device
    void* ws_base;
    domino::WorkspaceUse use;
};

namespace domino {
namespace optim {

unsigned norm_ctas(const domino_adamw_ctx* c, unsigned tiles);  // of a launch over so many tiles
cudaError_t launch_adamw8(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st);
cudaError_t launch_adamw32(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st);
cudaError_t launch_norm(const Work& w, const NormArgs& a, unsigned ctas, cudaStream_t st);

}  // namespace optim
}  // namespace domino
