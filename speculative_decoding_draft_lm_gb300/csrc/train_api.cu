// C ABI of the draft-head training operators: argument checks, workspace,
// status and teardown.
#include <math.h>
#include <stdlib.h>

#include "train_internal.h"

using namespace domino;

namespace {

inline int esize(int dtype) { return dtype == DOMINO_DTYPE_BF16 ? 2 : 4; }
inline bool known(int dtype) { return dtype == DOMINO_DTYPE_FP32 || dtype == DOMINO_DTYPE_BF16; }
inline bool aligned(const void* p, int a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }
inline bool good_temperature(float t) { return t >= 1e-3f && t <= 1e3f; }  // false for NaN

int nothing_to_do(domino_train_ctx* c) {
    c->last_launches = 0;
    return DOMINO_OK;
}

// what the three distillation calls share; n = 0 is checked by the caller
bool good_record(const domino_train_ctx* c, const void* x, long long ld, const int32_t* ids, const float* top,
                 const float* rest, int K, float temperature) {
    return x && ids && top && ld >= c->cfg.V && K >= 1 && K <= DOMINO_TRAIN_MAX_K && good_temperature(temperature) &&
           aligned(x, esize(c->cfg.dtype)) && aligned(ids, 4) && aligned(top, 4) && aligned(rest, 4);
}

train::DistillArgs distill_args(const domino_train_ctx* c, const void* x, long long ld, int n, const int32_t* ids,
                                const float* top, const float* rest, int K, float temperature) {
    train::DistillArgs a = {};
    a.x = x;
    a.ld = ld;
    a.n = n;
    a.V = c->cfg.V;
    a.ids = ids;
    a.top = top;
    a.rest = rest;
    a.K = K;
    a.temperature = temperature;
    a.err = c->err;
    return a;
}

void release(domino_train_ctx* c) {  // on the context's device
    if (c->used) cudaEventDestroy(c->used);
    if (c->captured) cudaEventDestroy(c->captured);
    cudaFree(c->ws_base);
    free(c);
}

// Orders the calls that use the workspace among each other, whatever their
// streams: a call waits for the event that the last one recorded.  Always, even
// on what looks like the same stream: a handle's value may be another stream's by
// now.  An event recorded outside of a capture cannot be waited for inside it, nor
// the other way round, so a capture has an event of its own for its calls.
struct WorkspaceOrder {
    domino_train_ctx* c;
    cudaStream_t st;
    bool capturing = false;
    cudaError_t error;

    WorkspaceOrder(domino_train_ctx* c_, cudaStream_t st_) : c(c_), st(st_) {
        cudaStreamCaptureStatus status;
        unsigned long long id = 0;
        error = cudaStreamGetCaptureInfo(st, &status, &id);
        if (error != cudaSuccess) return;
        capturing = status == cudaStreamCaptureStatusActive;
        if (capturing) {
            if (c->captured_id == id) error = cudaStreamWaitEvent(st, c->captured, 0);
            c->captured_id = id;
        } else if (c->was_used) {
            error = cudaStreamWaitEvent(st, c->used, 0);
        }
    }
    // after the launches, also where one of them failed
    cudaError_t done() {
        if (!capturing) c->was_used = true;
        return cudaEventRecord(capturing ? c->captured : c->used, st);
    }
};

// The error word to `taken`, and 0 in its place: in one step, so that what
// another stream raises meanwhile is in this answer or in the next.
__global__ void k_take_error(int* err, int* taken) { *taken = atomicExch(err, 0); }

}  // namespace

extern "C" {

int domino_train_init(domino_train_ctx** out, const domino_train_config* cfg, int device) {
    if (!out) return DOMINO_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg) return DOMINO_ERR_INVALID_ARG;
    if (!known(cfg->dtype) || cfg->V > DOMINO_TRAIN_MAX_V) return DOMINO_ERR_UNSUPPORTED;
    if (cfg->V < 2 || cfg->E < 0 || cfg->E > (1 << 20) || cfg->max_tokens < 0 ||
        cfg->max_tokens > DOMINO_TRAIN_MAX_TOKENS)
        return DOMINO_ERR_INVALID_ARG;
    int ndev = 0;
    if (cudaGetDeviceCount(&ndev) != cudaSuccess || device < 0 || device >= ndev) return DOMINO_ERR_CUDA;
    DeviceGuard guard(device);
    domino_train_ctx* c = (domino_train_ctx*)calloc(1, sizeof(domino_train_ctx));
    if (!c) return DOMINO_ERR_OOM;
    c->cfg = *cfg;
    c->device = device;
    if (cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        free(c);
        return DOMINO_ERR_CUDA;
    }
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align_up(off + bytes, 256);
        return o;
    };
    const size_t n = (size_t)cfg->max_tokens, tiles = (n + train::kSortTile - 1) / train::kSortTile;
    const size_t o_err = take(2 * sizeof(int));
    size_t o_keys[2], o_pos[2];
    for (int i = 0; i < 2; ++i) {
        o_keys[i] = take(n * 4);
        o_pos[i] = take(n * 4);
    }
    const size_t o_hist = take(tiles > train::kSortMaxCluster ? tiles * train::kSortMaxBins * 4 : 0);
    const size_t units = n > 0 ? train::max_sum_units((int)n, c->num_sms) : 0;
    const size_t o_part = take(units * 2 * cfg->E * sizeof(float));
    const size_t o_named = take(cfg->E > 0 ? ((size_t)cfg->V + 31) / 32 * 4 : 0), o_claim = take(sizeof(unsigned));
    if (cudaMalloc(&c->ws_base, off) != cudaSuccess) {
        cudaGetLastError();
        free(c);
        return DOMINO_ERR_OOM;
    }
    char* base = (char*)c->ws_base;
    c->err = (int*)(base + o_err);
    for (int i = 0; i < 2; ++i) {
        c->keys[i] = (uint32_t*)(base + o_keys[i]);
        c->pos[i] = (int32_t*)(base + o_pos[i]);
    }
    c->hist = (unsigned*)(base + o_hist);
    c->part = (float*)(base + o_part);
    c->named = (unsigned*)(base + o_named);
    c->claim = (unsigned*)(base + o_claim);
    if (cudaEventCreateWithFlags(&c->used, cudaEventDisableTiming) != cudaSuccess ||
        cudaEventCreateWithFlags(&c->captured, cudaEventDisableTiming) != cudaSuccess ||
        cudaMemset(c->err, 0, sizeof(int)) != cudaSuccess || train::prepare_embed_kernels() != cudaSuccess ||
        train::prepare_distill_kernels() != cudaSuccess || train::prepare_top_kernels() != cudaSuccess ||
        cudaDeviceSynchronize() != cudaSuccess) {
        release(c);
        return DOMINO_ERR_CUDA;
    }
    *out = c;
    return DOMINO_OK;
}

int domino_train_top_logits(domino_train_ctx* c, const void* logits, int dtype, long long ld, int n_rows, int K,
                            float temperature, int32_t* ids, float* top, float* rest, void* stream) {
    if (!c || n_rows < 0) return DOMINO_ERR_INVALID_ARG;
    if (!known(dtype)) return DOMINO_ERR_UNSUPPORTED;
    if (K < 1 || K > c->cfg.V || K > DOMINO_TRAIN_MAX_K || !good_temperature(temperature)) return DOMINO_ERR_INVALID_ARG;
    if (n_rows == 0) return nothing_to_do(c);
    if (!logits || !ids || !top || !rest || ld < c->cfg.V || !aligned(logits, esize(dtype)) || !aligned(ids, 4) ||
        !aligned(top, 4) || !aligned(rest, 4))
        return DOMINO_ERR_INVALID_ARG;
    DeviceGuard guard(c->device);
    const cudaError_t e =
        train::launch_top(c, logits, dtype, ld, n_rows, K, temperature, ids, top, rest, (cudaStream_t)stream);
    return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

int domino_train_distill_forward(domino_train_ctx* c, const void* logits, long long ld, int n_rows, const int32_t* ids,
                                 const float* top, const float* rest, int K, float temperature, float* loss,
                                 float* stats, void* stream) {
    if (!c || n_rows < 0) return DOMINO_ERR_INVALID_ARG;
    if (n_rows == 0) return nothing_to_do(c);
    if (!good_record(c, logits, ld, ids, top, rest, K, temperature) || !loss || !stats || !aligned(loss, 4) ||
        !aligned(stats, 4))
        return DOMINO_ERR_INVALID_ARG;
    train::DistillArgs a = distill_args(c, logits, ld, n_rows, ids, top, rest, K, temperature);
    a.loss = loss;
    a.stats = stats;
    DeviceGuard guard(c->device);
    return train::launch_distill_forward(c, a, (cudaStream_t)stream) == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

int domino_train_distill_backward(domino_train_ctx* c, const void* logits, long long ld, int n_rows,
                                  const int32_t* ids, const float* top, const float* rest, int K, float temperature,
                                  const float* stats, const float* dloss, void* dlogits, long long ld_d,
                                  void* stream) {
    if (!c || n_rows < 0) return DOMINO_ERR_INVALID_ARG;
    if (n_rows == 0) return nothing_to_do(c);
    if (!good_record(c, logits, ld, ids, top, rest, K, temperature) || !stats || !dloss || !dlogits ||
        dlogits == logits || ld_d < c->cfg.V || !aligned(dlogits, esize(c->cfg.dtype)) || !aligned(stats, 4) ||
        !aligned(dloss, 4))
        return DOMINO_ERR_INVALID_ARG;
    train::DistillArgs a = distill_args(c, logits, ld, n_rows, ids, top, rest, K, temperature);
    a.stats = const_cast<float*>(stats);
    a.weight = dloss;
    a.dx = dlogits;
    a.ld_d = ld_d;
    DeviceGuard guard(c->device);
    return train::launch_distill_backward(c, a, (cudaStream_t)stream) == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

int domino_train_distill_step(domino_train_ctx* c, const void* logits, long long ld, int n_rows, const int32_t* ids,
                              const float* top, const float* rest, int K, float temperature, const float* weight,
                              float* loss, void* dlogits, long long ld_d, void* stream) {
    if (!c || n_rows < 0) return DOMINO_ERR_INVALID_ARG;
    if (n_rows == 0) return nothing_to_do(c);
    if (!good_record(c, logits, ld, ids, top, rest, K, temperature) || !weight || !loss || !dlogits ||
        dlogits == logits || ld_d < c->cfg.V || !aligned(dlogits, esize(c->cfg.dtype)) || !aligned(weight, 4) ||
        !aligned(loss, 4))
        return DOMINO_ERR_INVALID_ARG;
    train::DistillArgs a = distill_args(c, logits, ld, n_rows, ids, top, rest, K, temperature);
    a.weight = weight;
    a.loss = loss;
    a.dx = dlogits;
    a.ld_d = ld_d;
    DeviceGuard guard(c->device);
    return train::launch_distill_step(c, a, (cudaStream_t)stream) == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

int domino_train_embed(domino_train_ctx* c, const void* table, const int32_t* tokens, int n_tokens, float scale,
                       void* out, long long ld_out, void* stream) {
    if (!c || n_tokens < 0 || c->cfg.E < 1) return DOMINO_ERR_INVALID_ARG;
    if (n_tokens == 0) return nothing_to_do(c);
    const int es = esize(c->cfg.dtype);
    if (!table || !tokens || !out || ld_out < c->cfg.E || !aligned(table, es) || !aligned(out, es) ||
        !aligned(tokens, 4) || table == out)
        return DOMINO_ERR_INVALID_ARG;
    DeviceGuard guard(c->device);
    return train::launch_embed(c, table, tokens, n_tokens, scale, out, ld_out, (cudaStream_t)stream) == cudaSuccess
               ? DOMINO_OK
               : DOMINO_ERR_CUDA;
}

int domino_train_embed_grad(domino_train_ctx* c, const void* dout, long long ld, const int32_t* tokens, int n_tokens,
                            float scale, void* dtable, int grad_dtype, int accumulate, void* stream) {
    if (!c || n_tokens < 0 || c->cfg.E < 1 || n_tokens > c->cfg.max_tokens) return DOMINO_ERR_INVALID_ARG;
    if (!known(grad_dtype)) return DOMINO_ERR_UNSUPPORTED;
    if (!dtable || !aligned(dtable, esize(grad_dtype))) return DOMINO_ERR_INVALID_ARG;
    if (n_tokens == 0 && accumulate) return nothing_to_do(c);
    if (n_tokens > 0 && (!dout || !tokens || ld < c->cfg.E || !aligned(dout, esize(c->cfg.dtype)) ||
                         !aligned(tokens, 4) || dout == dtable))
        return DOMINO_ERR_INVALID_ARG;
    DeviceGuard guard(c->device);
    const cudaStream_t st = (cudaStream_t)stream;
    WorkspaceOrder order(c, st);
    if (order.error != cudaSuccess) return DOMINO_ERR_CUDA;
    c->last_launches = 0;
    const cudaError_t launched =
        train::launch_embed_grad(c, dout, ld, tokens, n_tokens, scale, dtable, grad_dtype, accumulate != 0, st);
    const cudaError_t recorded = order.done();
    return launched == cudaSuccess && recorded == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

int domino_train_status(domino_train_ctx* c, void* stream) {
    if (!c) return DOMINO_ERR_INVALID_ARG;
    DeviceGuard guard(c->device);
    // all in the stream's order: another stream, the default one too, is not ordered with it
    const cudaStream_t st = (cudaStream_t)stream;
    int word = 0;
    const auto read = [&](const int* from) {
        return cudaMemcpyAsync(&word, from, sizeof(int), cudaMemcpyDeviceToHost, st) == cudaSuccess &&
               cudaStreamSynchronize(st) == cudaSuccess;
    };
    if (!read(c->err)) return DOMINO_ERR_CUDA;
    if (word) {
        cudaLaunchConfig_t one = {};
        one.gridDim = one.blockDim = dim3(1);
        one.stream = st;
        if (cudaLaunchKernelEx(&one, k_take_error, c->err, c->err + 1) != cudaSuccess || !read(c->err + 1))
            return DOMINO_ERR_CUDA;
    }
    if (word & kErrTimeout) return DOMINO_ERR_TIMEOUT;
    return word & kErrBadToken ? DOMINO_ERR_BAD_TOKEN : DOMINO_OK;
}

int domino_train_last_launch_count(const domino_train_ctx* c) { return c ? c->last_launches : 0; }

void domino_train_destroy(domino_train_ctx* c) {
    if (!c) return;
    DeviceGuard guard(c->device);
    cudaDeviceSynchronize();
    release(c);
}

}  // extern "C"
