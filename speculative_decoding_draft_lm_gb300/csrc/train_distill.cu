// Distillation of a draft head from a record of its teacher's logits: the loss
// of each row and its gradient by the student's logits.
//
// With S the record's ids, u = x / T the student's scaled logits and t / T the
// teacher's, write
//   Z_S = sum_S e^u,  Z_o = sum_{v not in S} e^u,  W = sum_S e^(t/T) + e^rest,
//   p_k = e^(t_k/T) / W,  p_r = e^rest / W,  q_v = e^(u_v) / (Z_S + Z_o).
// Since sum p + p_r = 1,
//   loss = sum_S p_k (t_k - x_k) / T + p_r (rest - log Z_o) + log((Z_S + Z_o) / W),
// in which the two normalisers meet as one ratio (their logarithms, near log V,
// never appear alone), and, dividing the outside by its own sum,
//   T dloss/dx_v = q_v - p_v                                  v in S
//                = e^(u_v) (1 / (Z_S + Z_o) - p_r / Z_o)      otherwise.
// Z_o is summed over the ids outside the record and not taken as a difference:
// near convergence the record holds almost all of the mass.
#include "train_internal.h"
#include "train_math.cuh"

namespace domino {
namespace train {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// What a row's loss and gradient go by; row layout of `stats`.
struct Stats {
    float mo, co;   // outside: T dloss/dx = co 2^((x - mo) c)
    float mx, qx;   // record:  q = qx 2^((x - mx) c)
    float mt, pt;   //          p = pt 2^((t - mt) c)
    float has;      // 0: the record holds no mass
    float pad;
};
static_assert(sizeof(Stats) == DOMINO_TRAIN_STATS * sizeof(float), "stats row");

struct Sums {
    MaxSum t, s, o;  // teacher's record, student's record, student's outside
    float a;         // sum 2^((t - mt) c) (t - x) / T
};

// a sum scaled to a new maximum; an infinite term whose weight vanished is 0
__device__ __forceinline__ float rescaled(float a, float f) { return f == 0.f ? 0.f : a * f; }

__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float c) {
    Sums r;
    r.t = join(x.t, y.t, c);
    r.s = join(x.s, y.s, c);
    r.o = join(x.o, y.o, c);
    r.a = rescaled(x.a, ex2((x.t.m - r.t.m) * c)) + rescaled(y.a, ex2((y.t.m - r.t.m) * c));
    return r;
}

__device__ __forceinline__ Sums shuffled(const Sums& x, int mask) {
    Sums r;
    r.t.m = __shfl_xor_sync(0xffffffffu, x.t.m, mask);
    r.t.s = __shfl_xor_sync(0xffffffffu, x.t.s, mask);
    r.s.m = __shfl_xor_sync(0xffffffffu, x.s.m, mask);
    r.s.s = __shfl_xor_sync(0xffffffffu, x.s.s, mask);
    r.o.m = __shfl_xor_sync(0xffffffffu, x.o.m, mask);
    r.o.s = __shfl_xor_sync(0xffffffffu, x.o.s, mask);
    r.a = __shfl_xor_sync(0xffffffffu, x.a, mask);
    return r;
}

// The row's statistics and loss from its sums; rest = -inf where there is none.
__device__ Stats finish(const Sums& u, float rest, float inv_t, float c, float* loss) {
    Stats st = {};
    *loss = 0.f;
    if (u.t.s == 0.f && rest == -INFINITY) return st;  // no target
    // the teacher's two parts on the larger one's scale
    float part = 1.f, part_r = 0.f, top = 0.f;  // top: the scale, kept apart where it is mt / T
    bool top_is_t = true;
    if (rest != -INFINITY) {
        const float d = u.t.s == 0.f ? -INFINITY : fmaf(u.t.m, inv_t, -rest);
        if (d >= 0.f) {
            part_r = expf(-d);
        } else {
            part = expf(d);  // NaN stays NaN
            part_r = 1.f;
            top = rest;
            top_is_t = false;
        }
    }
    const float w = u.t.s * part + part_r;
    const float pr = part_r / w;
    const MaxSum x = join(u.s, u.o, c);
    st.has = 1.f;
    st.mt = u.t.m;
    st.pt = part / w;
    st.mx = x.m;
    st.qx = 1.f / x.s;
    st.mo = u.o.m;
    float l = rescaled(u.a, st.pt) + (top_is_t ? (x.m - u.t.m) * inv_t : fmaf(x.m, inv_t, -top)) + logf(x.s / w);
    st.co = ex2((u.o.m - x.m) * c) / x.s;
    if (pr != 0.f) {
        l -= pr * (fmaf(u.o.m, inv_t, -rest) + logf(u.o.s));
        st.co = u.o.s == 0.f ? 0.f : st.co - pr / u.o.s;
    }
    *loss = l;
    return st;
}

// Marks the row's record in `bits` (one bit per id) and returns whether an id
// occurs twice.  All threads.
__device__ bool mark_record(const int32_t* ids, int K, int V, unsigned* bits, int* flag, int* err) {
    if (threadIdx.x == 0) *flag = 0;
    for (int i = threadIdx.x; i < (V + 31) / 32; i += kThreads) bits[i] = 0;
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += kThreads) {
        const int id = ids[k];
        if ((unsigned)id < (unsigned)V) {
            const unsigned bit = 1u << (id & 31);
            if (atomicOr(&bits[id >> 5], bit) & bit) *flag = 1;
        } else if (id != -1) {
            atomicOr(err, kErrBadToken);
        }
    }
    __syncthreads();
    return *flag != 0;
}

// Whether entry k of the record takes part: a valid id, and its first place.
__device__ __forceinline__ bool takes_part(const int32_t* ids, int k, int id, int V, bool twice) {
    if ((unsigned)id >= (unsigned)V) return false;
    if (twice)
        for (int j = 0; j < k; ++j)
            if (ids[j] == id) return false;
    return true;
}

template <typename T, bool kForward, bool kBackward>
__global__ void __launch_bounds__(kThreads) k_distill(DistillArgs p) {
    extern __shared__ unsigned bits[];
    __shared__ Sums part[kWarps];
    __shared__ Stats row;
    __shared__ int flag;
    const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float inv_t = 1.f / p.temperature, c = kLog2e / p.temperature;
    const T* x = static_cast<const T*>(p.x) + (size_t)n * p.ld;
    T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d;
    const int32_t* ids = p.ids + (size_t)n * p.K;
    const float* top = p.top + (size_t)n * p.K;
    Stats st = {};
    if (!kForward) st = reinterpret_cast<const Stats*>(p.stats)[n];
    if (kBackward) {
        if (p.weight[n] == 0.f || (!kForward && st.has == 0.f)) {
            for (int v = threadIdx.x; v < p.V; v += kThreads) dx[v] = from_f32<T>(0.f);
            if (kForward && threadIdx.x == 0) p.loss[n] = 0.f;
            return;
        }
    }
    const bool twice = mark_record(ids, p.K, p.V, bits, &flag, p.err);
    if (kForward) {
        Sums u = {empty_set(), empty_set(), empty_set(), 0.f};
        for (int k = threadIdx.x; k < p.K; k += kThreads) {
            const int id = ids[k];
            if (!takes_part(ids, k, id, p.V, twice)) continue;
            const float t = top[k], v = to_f32(x[id]);
            if (t > u.t.m) {
                const float m = clamp_max(u.t.m, t), f = ex2((u.t.m - m) * c);
                u.t.s *= f;
                u.a = rescaled(u.a, f);
                u.t.m = m;
            }
            const float e = ex2((t - u.t.m) * c);
            u.t.s += e;
            if (e != 0.f) u.a += e * (t - v) * inv_t;
            add(u.s, v, c);
        }
        for (int v = threadIdx.x; v < p.V; v += kThreads)
            if (!(bits[v >> 5] >> (v & 31) & 1u)) add(u.o, to_f32(x[v]), c);
        for (int o = 16; o > 0; o >>= 1) u = join(u, shuffled(u, o), c);
        if (lane == 0) part[warp] = u;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) u = join(u, part[w], c);
            float loss;
            row = finish(u, p.rest ? p.rest[n] : -INFINITY, inv_t, c, &loss);
            p.loss[n] = loss;
            if (p.stats) reinterpret_cast<Stats*>(p.stats)[n] = row;
        }
        __syncthreads();
        st = row;
    }
    if (kBackward) {
        // a row without mass takes this path too: its factors are 0, but its
        // logits may be infinite
        const float w = st.has == 0.f ? 0.f : p.weight[n] * inv_t;
        for (int v = threadIdx.x; v < p.V; v += kThreads)
            if (!(bits[v >> 5] >> (v & 31) & 1u))
                dx[v] = from_f32<T>(w == 0.f ? 0.f : w * st.co * ex2((to_f32(x[v]) - st.mo) * c));
        for (int k = threadIdx.x; k < p.K; k += kThreads) {
            const int id = ids[k];
            if (!takes_part(ids, k, id, p.V, twice)) continue;
            const float q = st.qx * ex2((to_f32(x[id]) - st.mx) * c), pk = st.pt * ex2((top[k] - st.mt) * c);
            dx[id] = from_f32<T>(w == 0.f ? 0.f : w * (q - pk));
        }
    }
}

template <bool kForward, bool kBackward>
cudaError_t launch(domino_train_ctx* ctx, const DistillArgs& a, cudaStream_t st) {
    const size_t smem = (size_t)(a.V + 31) / 32 * 4;
    auto kern = ctx->cfg.dtype == DOMINO_DTYPE_BF16 ? k_distill<__nv_bfloat16, kForward, kBackward>
                                                    : k_distill<float, kForward, kBackward>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<a.n, kThreads, smem, st>>>(a);
    ctx->last_launches = 1;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_distill_forward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return launch<true, false>(c, a, st);
}
cudaError_t launch_distill_backward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return launch<false, true>(c, a, st);
}
cudaError_t launch_distill_step(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return launch<true, true>(c, a, st);
}

}  // namespace train
}  // namespace domino
