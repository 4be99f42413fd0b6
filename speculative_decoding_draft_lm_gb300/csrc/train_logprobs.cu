// Scores of rows of logits: the log probability of each row's token, the row's
// entropy and its most likely alternatives, and the gradient of the first two.
//
// With m the largest logit of a row, d_v = (x_v - m) / T, s = sum e^(d_v) and
// t = sum e^(d_v) d_v,
//   log q_v = d_v - log s,   H = log s - t / s,
//   T dx_v = g ([v = tok] - q_v) - h q_v (log q_v + H).
// What all logits of a row share cancels in d, which is exact where it is small.
#include "train_internal.h"
#include "train_stream.cuh"

namespace domino {
namespace train {

namespace {

constexpr int kThreads = 256;

// What a row's gradient goes by; row layout of `stats`.
struct LogprobStats {
    float m, inv_s;       // q = inv_s 2^((x - m) c); inv_s = 0: the row takes no part
    float log_s, entropy;
};
static_assert(sizeof(LogprobStats) == DOMINO_TRAIN_LOGPROB_STATS * sizeof(float), "stats row");

// A set of logits through its largest one, s and t (t on the scale of base-2 exponents).
struct Scores {
    float m, s, t;
};
__device__ __forceinline__ Scores no_scores() { return {-FLT_MAX, 0.f, 0.f}; }
// a + b where a is moved to the maximum m
__device__ __forceinline__ Scores moved(Scores a, float m, float c) {
    const float d = (a.m - m) * c, f = ex2(d);
    return {m, a.s * f, f == 0.f ? 0.f : f * fmaf(d, a.s, a.t)};
}
__device__ __forceinline__ void add(Scores& a, float v, float c) {
    if (v > a.m) a = moved(a, clamp_max(a.m, v), c);
    const float d = (v - a.m) * c, e = ex2(d);
    a.s += e;
    if (e != 0.f) a.t = fmaf(e, d, a.t);
}
__device__ __forceinline__ Scores join(Scores a, Scores b, float c) {
    const float m = fmaxf(a.m, b.m);
    a = moved(a, m, c);
    b = moved(b, m, c);
    return {m, a.s + b.s, a.t + b.t};
}

struct RowScore {
    LogprobStats st;
    bool some;  // the row has a distribution
};
__device__ __forceinline__ RowScore finish(const Scores& a) {
    RowScore r;
    r.some = a.s != 0.f;
    if (!r.some) {
        r.st = {0.f, 0.f, 0.f, 0.f};
    } else if (!(a.s < INFINITY)) {
        const float nan = __uint_as_float(0x7FC00000u);
        r.st = {nan, nan, nan, nan};
    } else {
        r.st.m = a.m;
        r.st.inv_s = 1.f / a.s;
        r.st.log_s = logf(a.s);
        r.st.entropy = r.st.log_s - a.t / a.s * 0.69314718055994531f;
    }
    return r;
}
__device__ __forceinline__ float log_q(const LogprobStats& st, float x, float T) {
    return (x - st.m) / T - st.log_s;
}

template <typename T>
__device__ __forceinline__ Scores block_scores(const T* x, int V, float c, Scores* part) {
    Scores a = no_scores();
    for (int i = threadIdx.x; i < V; i += kThreads) add(a, to_f32(x[i]), c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Scores b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o),
                          __shfl_xor_sync(0xffffffffu, a.t, o)};
        a = join(a, b, c);
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = a;
    __syncthreads();
    a = part[0];
    for (int i = 1; i < kThreads / 32; ++i) a = join(a, part[i], c);
    return a;
}

// key of a logit and its id: larger is earlier among the alternatives
__device__ __forceinline__ unsigned long long word_of(float x, int id) {
    return (unsigned long long)(x != x ? 0xFFFFFFFFu : ord_f32(x)) << 32 | (unsigned)~id;
}

// The gradient of the elements first, first + stride, ... < last of a row.
template <typename T>
__device__ __forceinline__ void gradient_row(const LogprobArgs& p, const T* x, T* dx, const LogprobStats& st, int tok,
                                             float g, float h, int first, int last, int stride) {
    const float c = kLog2e / p.temperature;
    if (st.inv_s == 0.f || (g == 0.f && h == 0.f)) {
        for (int i = first; i < last; i += stride) dx[i] = from_f32<T>(0.f);
        return;
    }
    for (int i = first; i < last; i += stride) {
        const float d = (to_f32(x[i]) - st.m) * c, q = st.inv_s * ex2(d);
        const float l = fmaf(fmaxf(d, -200.f), 0.69314718055994531f, st.entropy - st.log_s);
        dx[i] = from_f32<T>((g * ((i == tok ? 1.f : 0.f) - q) - h * q * l) / p.temperature);
    }
}

template <typename T, bool kStep>
__global__ void __launch_bounds__(kThreads) k_scores(LogprobArgs p) {
    __shared__ Scores part[kThreads / 32];
    __shared__ unsigned long long best[kThreads / 32];
    const int n = blockIdx.x, t = threadIdx.x;
    const T* x = static_cast<const T*>(p.x) + (size_t)n * p.ld;
    const int tok = p.tokens[n];
    const bool in = (unsigned)tok < (unsigned)p.V;
    const float g = kStep && p.dlogprob ? p.dlogprob[n] : 0.f, h = kStep && p.dentropy ? p.dentropy[n] : 0.f;
    const float c = kLog2e / p.temperature;
    if (t == 0 && !in && tok != -1) atomicOr(p.err, kErrBadToken);
    if (!in || (kStep && g == 0.f && h == 0.f)) {
        if (t == 0) {
            p.logprob[n] = 0.f;
            if (p.entropy) p.entropy[n] = 0.f;
            if (p.stats) reinterpret_cast<LogprobStats*>(p.stats)[n] = {0.f, 0.f, 0.f, 0.f};
        }
        for (int k = t; k < p.k; k += kThreads) {
            p.alt_ids[(size_t)n * p.k + k] = -1;
            p.alt_logprobs[(size_t)n * p.k + k] = -INFINITY;
        }
        if (kStep)
            for (int i = t; i < p.V; i += kThreads) static_cast<T*>(p.dx)[(size_t)n * p.ld_d + i] = from_f32<T>(0.f);
        return;
    }
    const RowScore r = finish(block_scores(x, p.V, c, part));
    if (t == 0) {
        p.logprob[n] = r.some ? log_q(r.st, to_f32(x[tok]), p.temperature) : -INFINITY;
        if (p.entropy) p.entropy[n] = r.st.entropy;
        if (p.stats) reinterpret_cast<LogprobStats*>(p.stats)[n] = r.st;
    }
    if (kStep) {
        gradient_row(p, x, static_cast<T*>(p.dx) + (size_t)n * p.ld_d, r.st, tok, g, h, t, p.V, kThreads);
        return;
    }
    unsigned long long last = ~0ull;
    for (int k = 0; k < p.k; ++k) {
        unsigned long long w = 0;
        for (int i = t; i < p.V; i += kThreads) {
            const float v = to_f32(x[i]);
            const unsigned long long u = v == -INFINITY ? 0ull : word_of(v, i);
            if ((k == 0 || u < last) && u > w) w = u;
        }
        w = warp_max_u64(w);
        __syncthreads();
        if (t % 32 == 0) best[t / 32] = w;
        __syncthreads();
        for (int i = 0; i < kThreads / 32; ++i) w = best[i] > w ? best[i] : w;
        last = w;
        if (t == 0) {
            const int id = w ? (int)~(unsigned)w : -1;
            p.alt_ids[(size_t)n * p.k + k] = id;
            p.alt_logprobs[(size_t)n * p.k + k] = w ? log_q(r.st, to_f32(x[id]), p.temperature) : -INFINITY;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scores_backward(LogprobArgs p) {
    const int n = blockIdx.x, tok = p.tokens[n];
    const T* x = static_cast<const T*>(p.x) + (size_t)n * p.ld;
    const float g = p.dlogprob ? p.dlogprob[n] : 0.f, h = p.dentropy ? p.dentropy[n] : 0.f;
    gradient_row(p, x, static_cast<T*>(p.dx) + (size_t)n * p.ld_d, reinterpret_cast<const LogprobStats*>(p.stats)[n], tok,
                 g, h, (int)threadIdx.x, p.V, kThreads);
}

template <bool kStep>
cudaError_t launch(domino_train_ctx* c, int dtype, const LogprobArgs& a, cudaStream_t st) {
    if (dtype == DOMINO_DTYPE_BF16) k_scores<__nv_bfloat16, kStep><<<a.n, kThreads, 0, st>>>(a);
    else k_scores<float, kStep><<<a.n, kThreads, 0, st>>>(a);
    c->last_launches = 1;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs_forward(domino_train_ctx* c, int dtype, const LogprobArgs& a, cudaStream_t st) {
    return launch<false>(c, dtype, a, st);
}
cudaError_t launch_logprobs_step(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st) {
    return launch<true>(c, c->cfg.dtype, a, st);
}
cudaError_t launch_logprobs_backward(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st) {
    if (c->cfg.dtype == DOMINO_DTYPE_BF16) k_scores_backward<__nv_bfloat16><<<a.n, kThreads, 0, st>>>(a);
    else k_scores_backward<float><<<a.n, kThreads, 0, st>>>(a);
    c->last_launches = 1;
    return cudaGetLastError();
}

}  // namespace train
}  // namespace domino
