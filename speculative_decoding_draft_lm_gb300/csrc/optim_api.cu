// C ABI of the weights' update: argument checks, workspace and launches.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "optim_internal.h"

using namespace domino;
using namespace domino::optim;

namespace {

inline bool known(int dtype) { return dtype == DOMINO_DTYPE_FP32 || dtype == DOMINO_DTYPE_BF16; }
inline int esize(int dtype) { return dtype == DOMINO_DTYPE_BF16 ? 2 : 4; }
inline bool aligned(const void* p, int a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }
inline bool between(double x, double lo, double hi) { return x >= lo && x <= hi; }  // false for NaN

struct Range {
    uintptr_t from, to;
};

// whether two of the ranges overlap; sorts them
bool overlap(Range* r, int n) {
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.from < b.from; });
    for (int i = 1; i < n; ++i)
        if (r[i].from < r[i - 1].to) return true;
    return false;
}

// DOMINO_OK, or what is wrong with the config; *blocks: of its flat buffers
int check(const domino_adamw_config* g, long long* blocks) {
    if (g->state_bits != 8 && g->state_bits != 32) return DOMINO_ERR_UNSUPPORTED;
    if (g->n_tensors < 1 || g->n_tensors > DOMINO_ADAMW_MAX_TENSORS || !g->tensors) return DOMINO_ERR_INVALID_ARG;
    bool master = false;
    *blocks = 0;
    for (int i = 0; i < g->n_tensors; ++i) {
        const domino_adamw_tensor& t = g->tensors[i];
        if (!known(t.dtype)) return DOMINO_ERR_UNSUPPORTED;
        if (t.n < 0 || t.n > kMaxElements || (t.n > 0 && !t.param) || !aligned(t.param, esize(t.dtype)) ||
            (t.master != 0 && t.dtype != DOMINO_DTYPE_BF16))
            return DOMINO_ERR_INVALID_ARG;
        master = master || t.master != 0;
        *blocks += (t.n + DOMINO_ADAMW_BLOCK - 1) / DOMINO_ADAMW_BLOCK;
        if (*blocks > kMaxElements / DOMINO_ADAMW_BLOCK) return DOMINO_ERR_INVALID_ARG;
    }
    const bool narrow = g->state_bits == 8, empty = *blocks == 0;
    const int align = 32;
    if (!g->count || !aligned(g->count, 8) || !aligned(g->m, align) || !aligned(g->v, align) ||
        !aligned(g->m_scale, 4) || !aligned(g->v_scale, 4) || !aligned(g->master, align))
        return DOMINO_ERR_INVALID_ARG;
    if (!empty && (!g->m || !g->v || (narrow && (!g->m_scale || !g->v_scale)) || (master && !g->master)))
        return DOMINO_ERR_INVALID_ARG;
    if (!between(g->beta1, 0, 1) || g->beta1 == 1 || !between(g->beta2, 0, 1) || g->beta2 == 1 ||
        !between(g->eps, 1e-16, 1) || !between(g->weight_decay, 0, 1))
        return DOMINO_ERR_INVALID_ARG;
    const int n = g->n_tensors;
    Range* r = (Range*)malloc((n + 6) * sizeof(Range));
    if (!r) return DOMINO_ERR_OOM;
    int k = 0;
    const auto add = [&](const void* p, long long bytes) {
        if (bytes > 0) r[k++] = {(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes};
    };
    for (int i = 0; i < n; ++i) add(g->tensors[i].param, g->tensors[i].n * esize(g->tensors[i].dtype));
    const long long positions = *blocks * DOMINO_ADAMW_BLOCK;
    add(g->m, positions * (narrow ? 1 : 4));
    add(g->v, positions * (narrow ? 1 : 4));
    add(g->m_scale, narrow ? *blocks * 4 : 0);
    add(g->v_scale, narrow ? *blocks * 4 : 0);
    add(g->master, master ? positions * 4 : 0);
    add(g->count, 8);
    const bool bad = overlap(r, k);
    free(r);
    return bad ? DOMINO_ERR_INVALID_ARG : DOMINO_OK;
}

// checks the gradients of a call
int check_gradients(const domino_adamw_ctx* c, const void* const* grads, const int* dtypes) {
    if (!grads || !dtypes) return DOMINO_ERR_INVALID_ARG;
    for (int i = 0; i < c->cfg.n_tensors; ++i) {
        if (!grads[i] || c->tensors[i].n == 0) continue;
        if (!known(dtypes[i])) return DOMINO_ERR_UNSUPPORTED;
        if (!aligned(grads[i], esize(dtypes[i])) || grads[i] == c->tensors[i].param) return DOMINO_ERR_INVALID_ARG;
    }
    return DOMINO_OK;
}

// what a tensor and its gradient are, as in Entry::n
unsigned long long kind_of(const domino_adamw_tensor& t, int grad_dtype) {
    return (t.dtype == DOMINO_DTYPE_BF16 ? kParamBf16 : 0) | (t.master ? kMaster : 0) |
           (grad_dtype == DOMINO_DTYPE_BF16 ? kGradBf16 : 0);
}

// The tensors from *next on that one launch takes, of one kind or (kAnyKind) of any; *next becomes the one behind them.
constexpr unsigned long long kAnyKind = ~0ull;
Work gather(domino_adamw_ctx* c, const void* const* grads, const int* dtypes, unsigned long long kind, int tile,
            int* next) {
    Work w = {0, 0, kind == kAnyKind ? 0 : kind, c->entry};
    int i = *next;
    for (; i < c->cfg.n_tensors && w.tensors < kMaxPerLaunch; ++i) {
        const domino_adamw_tensor& t = c->tensors[i];
        if (!grads[i] || t.n == 0) continue;
        const unsigned long long its = kind_of(t, dtypes[i]);
        if (kind != kAnyKind && its != kind) continue;
        Entry& e = w.entry[w.tensors++];
        e.p = t.param;
        e.g = grads[i];
        e.n = (unsigned long long)t.n | its;
        e.tile = w.tiles;
        e.block = c->block[i];
        w.tiles += (unsigned)((t.n + tile - 1) / tile);
    }
    *next = i;
    return w;
}

void release(domino_adamw_ctx* c) {  // on the context's device
    c->use.release();
    cudaFree(c->ws_base);
    free(c->tensors);
    free(c->block);
    free(c->entry);
    free(c);
}

}  // namespace

extern "C" {

int domino_adamw_init(domino_adamw_ctx** out, const domino_adamw_config* cfg, int device) {
    if (!out) return DOMINO_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg) return DOMINO_ERR_INVALID_ARG;
    long long blocks = 0;
    const int status = check(cfg, &blocks);
    if (status != DOMINO_OK) return status;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) return DOMINO_ERR_CUDA;
    DeviceGuard guard(device);
    domino_adamw_ctx* c = (domino_adamw_ctx*)calloc(1, sizeof(domino_adamw_ctx));
    if (!c) return DOMINO_ERR_OOM;
    const int n = cfg->n_tensors;
    c->cfg = *cfg;
    c->device = device;
    c->tensors = (domino_adamw_tensor*)malloc(n * sizeof(domino_adamw_tensor));
    c->block = (unsigned*)malloc(n * sizeof(unsigned));
    c->entry = (Entry*)aligned_alloc(16, kMaxPerLaunch * sizeof(Entry));
    if (!c->tensors || !c->block || !c->entry) {
        release(c);
        return DOMINO_ERR_OOM;
    }
    memcpy(c->tensors, cfg->tensors, n * sizeof(domino_adamw_tensor));
    c->cfg.tensors = c->tensors;
    blocks = 0;
    for (int i = 0; i < n; ++i) {
        c->block[i] = (unsigned)blocks;
        blocks += (c->tensors[i].n + DOMINO_ADAMW_BLOCK - 1) / DOMINO_ADAMW_BLOCK;
    }
    if (cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        release(c);
        return DOMINO_ERR_CUDA;
    }
    const size_t parts = (size_t)norm_ctas(c, ~0u) * ((n + kMaxPerLaunch - 1) / kMaxPerLaunch);
    if (cudaMalloc(&c->ws_base, 256 + parts * sizeof(float2)) != cudaSuccess) {
        cudaGetLastError();
        release(c);
        return DOMINO_ERR_OOM;
    }
    c->ticket = (unsigned*)c->ws_base;
    c->part = (float2*)((char*)c->ws_base + 256);
    if (c->use.create() != cudaSuccess || cudaMemset(c->ws_base, 0, 256) != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        release(c);
        return DOMINO_ERR_CUDA;
    }
    *out = c;
    return DOMINO_OK;
}

int domino_adamw_step(domino_adamw_ctx* c, const void* const* grads, const int* grad_dtypes, double lr,
                      const float* lr_factor, const float* scale, void* stream) {
    if (!c || !between(lr, 0, 1e3) || !aligned(lr_factor, 4) || !aligned(scale, 4)) return DOMINO_ERR_INVALID_ARG;
    const int status = check_gradients(c, grads, grad_dtypes);
    if (status != DOMINO_OK) return status;
    const domino_adamw_config& g = c->cfg;
    AdamArgs a = {};
    a.m = g.m;
    a.v = g.v;
    a.m_scale = g.m_scale;
    a.v_scale = g.v_scale;
    a.master = g.master;
    a.count = g.count;
    a.scale = scale;
    a.lr_factor = lr_factor;
    a.ticket = c->ticket;
    a.lr = (float)lr;
    const auto twice = [](double x) { return make_float2((float)x, (float)x); };
    a.beta1 = twice(g.beta1);
    a.beta2 = twice(g.beta2);
    a.rest1 = twice(1 - g.beta1);
    a.rest2 = twice(1 - g.beta2);
    a.eps = twice(g.eps);
    a.one = twice(1);
    a.log_beta1 = (float)log(g.beta1);
    a.log_beta2 = (float)log(g.beta2);
    a.decay = (float)g.weight_decay;
    a.seed = g.seed;
    a.golden = 0x9E3779B9u;
    a.up12 = 1u << 12;
    DeviceGuard guard(c->device);
    const cudaStream_t st = (cudaStream_t)stream;
    WorkspaceOrder order(&c->use, st);
    if (order.error != cudaSuccess) return DOMINO_ERR_CUDA;
    // a launch for every kind of tensors (mostly one), and for every kMaxPerLaunch of a kind
    bool seen[8] = {};
    int kinds = 0, launches = 0;
    unsigned long long kind[8];
    for (int i = 0; i < g.n_tensors; ++i) {
        if (!grads[i] || c->tensors[i].n == 0) continue;
        const unsigned long long its = kind_of(c->tensors[i], grad_dtypes[i]);
        bool& known_kind = seen[its / kParamBf16];
        if (!known_kind) kind[kinds++] = its;
        known_kind = true;
    }
    if (kinds == 0) kind[kinds++] = 0;  // also without a gradient: the step counts
    cudaError_t launched = cudaSuccess;
    for (int k = 0; launched == cudaSuccess && k < kinds; ++k) {
        int next = 0;
        do {
            const Work w = gather(c, grads, grad_dtypes, kind[k], g.state_bits == 8 ? kTile8 : kTile32, &next);
            for (; next < g.n_tensors; ++next)  // to the next one of this kind
                if (grads[next] && c->tensors[next].n > 0 &&
                    kind_of(c->tensors[next], grad_dtypes[next]) == kind[k])
                    break;
            a.last = k == kinds - 1 && next == g.n_tensors;
            launched = g.state_bits == 8 ? launch_adamw8(c, w, a, st) : launch_adamw32(c, w, a, st);
            ++launches;
        } while (launched == cudaSuccess && next < g.n_tensors);
    }
    // a call cut short has not counted its CTAs out
    if (launched != cudaSuccess) cudaMemsetAsync(c->ws_base, 0, 256, st);
    const cudaError_t recorded = order.done();
    if (launched != cudaSuccess || recorded != cudaSuccess) return DOMINO_ERR_CUDA;
    c->last_launches = launches;
    return DOMINO_OK;
}

int domino_adamw_grad_norm(domino_adamw_ctx* c, const void* const* grads, const int* grad_dtypes, float max_norm,
                           float* norm, float* scale, void* stream) {
    if (!c || !(max_norm > 0.f) || !norm || !aligned(norm, 4) || !aligned(scale, 4) || norm == scale)
        return DOMINO_ERR_INVALID_ARG;
    const int status = check_gradients(c, grads, grad_dtypes);
    if (status != DOMINO_OK) return status;
    NormArgs a = {};
    a.part = c->part;
    a.ticket = c->ticket + 1;
    a.max_norm = max_norm;
    a.norm = norm;
    a.scale = scale;
    for (int next = 0; next < c->cfg.n_tensors;)
        a.ctas += norm_ctas(c, gather(c, grads, grad_dtypes, kAnyKind, kNormTile, &next).tiles);
    DeviceGuard guard(c->device);
    const cudaStream_t st = (cudaStream_t)stream;
    WorkspaceOrder order(&c->use, st);
    if (order.error != cudaSuccess) return DOMINO_ERR_CUDA;
    cudaError_t launched = cudaSuccess;
    int launches = 0;
    const bool none = a.ctas == 0;
    if (none) a.ctas = 1;
    for (int next = 0; launched == cudaSuccess && next < c->cfg.n_tensors;) {
        const Work w = gather(c, grads, grad_dtypes, kAnyKind, kNormTile, &next);
        const unsigned ctas = none ? 1 : norm_ctas(c, w.tiles);
        if (ctas == 0) continue;
        launched = launch_norm(w, a, ctas, st);
        a.first += ctas;
        ++launches;
        if (none) break;
    }
    // a call cut short has not counted its CTAs out
    if (launched != cudaSuccess) cudaMemsetAsync(c->ws_base, 0, 256, st);
    const cudaError_t recorded = order.done();
    if (launched != cudaSuccess || recorded != cudaSuccess) return DOMINO_ERR_CUDA;
    c->last_launches = launches;
    return DOMINO_OK;
}

int domino_adamw_last_launch_count(const domino_adamw_ctx* c) { return c ? c->last_launches : 0; }

void domino_adamw_destroy(domino_adamw_ctx* c) {
    if (!c) return;
    DeviceGuard guard(c->device);
    cudaDeviceSynchronize();
    release(c);
}

}  // extern "C"
