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
#include <cooperative_groups.h>

#include "tc_common.cuh"
#include "train_internal.h"
#include "train_math.cuh"

namespace cg = cooperative_groups;

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

// Whether entry k of the record takes part: a valid id, and its first place.
__device__ __forceinline__ bool takes_part(const int32_t* ids, int k, int id, int V, bool twice) {
    if ((unsigned)id >= (unsigned)V) return false;
    if (twice)
        for (int j = 0; j < k; ++j)
            if (ids[j] == id) return false;
    return true;
}

// ---- loss and gradient at once ---------------------------------------------------
//
// A cluster of CTAs holds one row in shared memory, a slice each: bulk copies
// bring it in, the sums and the gradient are two passes over shared memory, and
// bulk copies take the gradient, written in place, out.  So the logits are read
// once and the gradient written once, which is all the traffic there is.  A
// slice is at most kSliceBytes, so that five CTAs share an SM and one's copies
// run under another's arithmetic; with few rows the slices are smaller and the
// row is spread over up to 16 SMs.
//
// Entries of the record are taken out of the slice (set to -inf) once their
// logits are read, so that the first pass is a plain sum over the outside.

constexpr int kStepThreads = 256;
constexpr int kStepWarps = kStepThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kSliceBytes = 40 * 1024;
constexpr int kHeld = 4;  // record entries whose logits a thread keeps; later ones are read again

struct StepShared {
    Sums warp[kStepWarps];
    Sums cta[kMaxCluster];
    Stats row;
    unsigned long long bar;
    int twice, abort;
};

// The slice of a row that a CTA holds: element i of the row is at data + i - v0,
// at the same place modulo 16 bytes as in memory.
template <typename T>
struct Slice {
    const T* src;   // element v0 of the row
    T* data;        // shared
    uint4* vec;     // the 16-byte vectors that cover it
    int v0, n, nvec;
    int head, body;  // elements before the first whole vector; elements of whole vectors

    __device__ Slice(const T* row, int V, int chunk, int rank, uint8_t* smem) {
        v0 = min(V, rank * chunk);
        n = min(V, v0 + chunk) - v0;
        src = row + v0;
        const int phase = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        vec = reinterpret_cast<uint4*>(smem);
        data = reinterpret_cast<T*>(smem + phase);
        nvec = (phase + n * (int)sizeof(T) + 15) / 16;
        head = min(n, ((16 - phase) & 15) / (int)sizeof(T));
        body = (n - head) / (16 / (int)sizeof(T)) * (16 / (int)sizeof(T));
    }
    // fills what the copies leave of the first and last vectors: the row's own
    // elements, and -inf where there are none
    __device__ void load_edges() {
        const int first = (int)(data - reinterpret_cast<T*>(vec)), per = 16 / (int)sizeof(T);
        const int t = threadIdx.x;
        if (t < first) reinterpret_cast<T*>(vec)[t] = from_f32<T>(-INFINITY);
        if (t < head) data[t] = src[t];
        const int tail = n - head - body;
        if (t < tail) data[head + body + t] = src[head + body + t];
        const int end = first + n, pad = nvec * per - end;
        if (t < pad) reinterpret_cast<T*>(vec)[end + t] = from_f32<T>(-INFINITY);
    }
};

__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() {
    asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Adds the values of shared vectors to a set, four vectors of a thread at once:
// one look at their maximum, then the exponentials.
template <typename T>
__device__ __forceinline__ MaxSum sum_vectors(const uint4* vec, int nvec, float c) {
    constexpr int U = 4, P = Vec16<T>::kElems / 2;
    const F2 cc = f2(c, c);
    MaxSum r = empty_set();
    F2 s = f2(0.f, 0.f);
    for (int i0 = threadIdx.x; i0 < nvec; i0 += U * kStepThreads) {
        Vec16<T> v[U];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + j * kStepThreads;
            if (i < nvec) {
                v[j].q = vec[i];
                top = fmaxf(top, v[j].top());
            }
        }
        if (top > r.m) {
            const float m = clamp_max(r.m, top), f = ex2((r.m - m) * c);
            s = mul2(s, f2(f, f));
            r.m = m;
        }
        const F2 minus = f2(-r.m, -r.m);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i0 + j * kStepThreads < nvec)
#pragma unroll
                for (int k = 0; k < P; ++k) s = add2(s, ex2x2(mul2(add2(v[j].pair(k), minus), cc)));
    }
    const float2 h = halves(s);
    r.s = h.x + h.y;
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kStepThreads) k_step(DistillArgs p, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ StepShared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int n = blockIdx.x / size, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const float inv_t = 1.f / p.temperature, c = kLog2e / p.temperature;
    const float weight = p.weight[n];
    Slice<T> x(static_cast<const T*>(p.x) + (size_t)n * p.ld, p.V, chunk, rank, smem);
    T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d + x.v0;
    unsigned* bits = reinterpret_cast<unsigned*>(smem + (size_t)chunk * sizeof(T) + 32);
    const int32_t* ids = p.ids + (size_t)n * p.K;
    const float* top = p.top + (size_t)n * p.K;
    float w = 0.f;

    if (weight != 0.f) {
        const uint32_t bar = tc::smem_u32(&S.bar);
        if (t == 0) {
            tc::mbar_init(bar, 1);
            S.twice = S.abort = 0;
            tc::fence_barrier_init();
            const uint32_t bytes = (uint32_t)x.body * sizeof(T);
            tc::mbar_arrive_expect_tx(bar, bytes);
            if (bytes) tc::bulk_load(tc::smem_u32(x.data + x.head), x.src + x.head, bytes, bar, tc::policy_evict_first());
        }
        cluster.sync();  // the barrier is up here, and every CTA of the row is running
        for (int i = t; i < (x.n + 31) / 32; i += kStepThreads) bits[i] = 0;
        x.load_edges();
        __syncthreads();
        for (int k = t; k < p.K; k += kStepThreads) {
            const int id = ids[k];
            const unsigned at = (unsigned)id - (unsigned)x.v0;
            if (id >= 0 && at < (unsigned)x.n) {
                const unsigned bit = 1u << (at & 31);
                if (atomicOr(&bits[at >> 5], bit) & bit) S.twice = 1;
            } else if (rank == 0 && id != -1 && (unsigned)id >= (unsigned)p.V) {
                atomicOr(p.err, kErrBadToken);
            }
        }
        __syncthreads();
        const bool twice = S.twice != 0;
        tc::mbar_wait(bar, 0, &S.abort, p.err);

        Sums u = {empty_set(), empty_set(), empty_set(), 0.f};
        float held[kHeld];
        int j = 0;
        for (int k = t; k < p.K; k += kStepThreads, ++j) {
            const int id = ids[k];
            if ((unsigned)id - (unsigned)x.v0 >= (unsigned)x.n || !takes_part(ids, k, id, p.V, twice)) continue;
            const float tk = top[k], v = to_f32(x.data[id - x.v0]);
            x.data[id - x.v0] = from_f32<T>(-INFINITY);
#pragma unroll
            for (int h = 0; h < kHeld; ++h)
                if (h == j) held[h] = v;
            if (tk > u.t.m) {
                const float m = clamp_max(u.t.m, tk), f = ex2((u.t.m - m) * c);
                u.t.s *= f;
                u.a = rescaled(u.a, f);
                u.t.m = m;
            }
            const float e = ex2((tk - u.t.m) * c);
            u.t.s += e;
            if (e != 0.f) u.a += e * (tk - v) * inv_t;
            add(u.s, v, c);
        }
        __syncthreads();
        u.o = sum_vectors<T>(x.vec, x.nvec, c);
        for (int o = 16; o > 0; o >>= 1) u = join(u, shuffled(u, o), c);
        if (lane == 0) S.warp[warp] = u;
        __syncthreads();
        if (t == 0) {
            for (int i = 1; i < kStepWarps; ++i) u = join(u, S.warp[i], c);
            for (int i = 0; i < size; ++i) *cluster.map_shared_rank(&S.cta[rank], i) = u;
        }
        cluster.sync();
        if (t == 0) {
            u = S.cta[0];
            for (int i = 1; i < size; ++i) u = join(u, S.cta[i], c);
            float loss;
            S.row = finish(u, p.rest ? p.rest[n] : -INFINITY, inv_t, c, &loss);
            if (rank == 0) p.loss[n] = loss;
        }
        __syncthreads();
        const Stats st = S.row;
        w = st.has == 0.f ? 0.f : weight * inv_t;
        if (w != 0.f) {
            constexpr int P = Vec16<T>::kElems / 2;
            const float wc = w * st.co;
            const F2 cc = f2(c, c), minus = f2(-st.mo, -st.mo), scale = f2(wc, wc);
#pragma unroll 2
            for (int i = t; i < x.nvec; i += kStepThreads) {
                Vec16<T> v, g;
                v.q = x.vec[i];
#pragma unroll
                for (int k = 0; k < P; ++k) g.set(k, mul2(scale, ex2x2(mul2(add2(v.pair(k), minus), cc))));
                x.vec[i] = g.q;
            }
            __syncthreads();
            j = 0;
            for (int k = t; k < p.K; k += kStepThreads, ++j) {
                const int id = ids[k];
                if ((unsigned)id - (unsigned)x.v0 >= (unsigned)x.n || !takes_part(ids, k, id, p.V, twice)) continue;
                float v = 0.f;
                if (j < kHeld) {
#pragma unroll
                    for (int h = 0; h < kHeld; ++h)
                        if (h == j) v = held[h];
                } else {
                    v = to_f32(x.src[id - x.v0]);
                }
                const float q = st.qx * ex2((v - st.mx) * c), pk = st.pt * ex2((top[k] - st.mt) * c);
                x.data[id - x.v0] = from_f32<T>(w * (q - pk));
            }
        }
        if (S.abort && t == 0) {  // the copies' wait ran out: give them a last chance to land before the CTA leaves
            const unsigned long long t0 = tc::globaltimer();
            while (!tc::mbar_try_wait(bar, 0) && tc::globaltimer() - t0 < 2000000ull) {
            }
        }
    } else if (rank == 0 && t == 0) {
        p.loss[n] = 0.f;
    }
    if (w == 0.f)
        for (int i = t; i < x.nvec; i += kStepThreads) x.vec[i] = make_uint4(0, 0, 0, 0);
    // out: whole vectors by bulk copy where the gradient's row starts at the same place modulo 16 bytes
    const bool together = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x.src)) & 15) == 0;
    tc::fence_proxy_async();
    __syncthreads();
    if (together) {
        if (t < x.head) dx[t] = x.data[t];
        const int tail = x.n - x.head - x.body;
        if (t < tail) dx[x.head + x.body + t] = x.data[x.head + x.body + t];
        if (t == 0 && x.body) {
            bulk_store(dx + x.head, tc::smem_u32(x.data + x.head), (uint32_t)x.body * sizeof(T));
            bulk_store_wait_read();
        }
    } else {
        for (int i = t; i < x.n; i += kStepThreads) dx[i] = x.data[i];
    }
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

namespace {
template <typename T>
cudaError_t launch_step(domino_train_ctx* ctx, const DistillArgs& a, cudaStream_t st) {
    int size = 1;
    auto slice = [&](int parts) { return ((a.V + parts - 1) / parts + 63) / 64 * 64; };
    while (size < kMaxCluster && slice(size) * (int)sizeof(T) > kSliceBytes) size *= 2;
    while (size < kMaxCluster && (long long)a.n * size < 2 * ctx->num_sms && slice(2 * size) >= 4096) size *= 2;
    const int chunk = slice(size);
    const size_t smem = (size_t)chunk * sizeof(T) + 32 + (size_t)chunk / 8;
    cudaError_t e = cudaFuncSetAttribute(k_step<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n * size);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ctx->last_launches = 1;
    return cudaLaunchKernelEx(&cfg, k_step<T>, a, chunk);
}
}  // namespace

cudaError_t prepare_distill_kernels() {
    cudaError_t e = cudaFuncSetAttribute(k_step<float>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_step<__nv_bfloat16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

cudaError_t launch_distill_step(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_step<__nv_bfloat16>(c, a, st) : launch_step<float>(c, a, st);
}

}  // namespace train
}  // namespace domino
