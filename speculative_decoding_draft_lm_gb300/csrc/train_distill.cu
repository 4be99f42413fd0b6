// Distillation of a draft head from a record of its teacher's logits: the loss
// of each row and its gradient by the student's logits.
//
// With S the record's ids, u = x / T the student's scaled logits and t / T the
// teacher's, write
//   Z_S = sum_S e^u,  Z_o = sum_{v not in S} e^u,  W = sum_S e^(t/T) + e^rest,
//   p_k = e^(t_k/T) / W,  p_r = e^rest / W,  q_v = e^(u_v) / (Z_S + Z_o).
// Every sum is held as s e^(m / T) with m a maximum: m_S and m_o the student's, m_x
// the larger of them, m_t the teacher's over the record.  With d = m_t / T - rest and
// since P + p_r = 1 for P = sum_S p_k,
//   loss = sum_S p_k ((t_k - m_t) - (x_k - m_S)) / T + P ((m_x - m_S) / T + min(d, 0))
//          + p_r ((m_x - m_o) / T - max(d, 0) - log s_o) + log(s_x / s_W),
// s_W on the scale of the larger of m_t / T and rest.  What all logits of a row share
// cancels in differences of two of them, which are exact where they are close: a row
// masked by the type's lowest value throughout is as good as a row of zeros.  The two
// normalisers meet as one ratio.  Dividing the outside by its own sum,
//   T dloss/dx_v = q_v - p_v                                  v in S
//                = e^(u_v) (1 / (Z_S + Z_o) - p_r / Z_o)      otherwise.
// Z_o is summed over the ids outside the record and not taken as a difference:
// near convergence the record holds almost all of the mass.
#include <cooperative_groups.h>

#include "train_internal.h"
#include "train_slice.cuh"
#include "train_stream.cuh"

namespace cg = cooperative_groups;

namespace domino {
namespace train {

namespace {

// What a row's loss and gradient go by; row layout of `stats`.
struct Stats {
    float mo, co;   // outside: T dloss/dx = co 2^((x - mo) c)
    float mx, qx;   // record:  q = qx 2^((x - mx) c)
    float mt, pt;   //          p = pt 2^((t - mt) c)
    float has;      // 0: the record holds no mass
    float twice;    // an id occurs twice in the record
};
static_assert(sizeof(Stats) == DOMINO_TRAIN_STATS * sizeof(float), "stats row");

struct alignas(16) Sums {
    MaxSum t, s, o;  // teacher's record, student's record, student's outside
    float a;         // sum 2^((t - mt) c) ((t - mt) - (x - ms)) / T
    float twice;     // forward: an id was seen twice
};
__device__ __forceinline__ Sums no_sums() { return {empty_set(), empty_set(), empty_set(), 0.f, 0.f}; }

// One thread's sums into a CTA's shared memory, counted on that CTA's barrier:
// the reader waits for the bytes alone.  A barrier of the cluster would make
// every thread wait until its stores to global memory are done.
__device__ __forceinline__ void send(const Sums& u, Sums* to, unsigned long long* bar, int rank) {
    static_assert(sizeof(Sums) == 32, "two 16-byte stores");
    uint32_t dst, mbar;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(tc::smem_u32(to)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(mbar) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "f"(u.t.m), "f"(u.t.s), "f"(u.s.m), "f"(u.s.s), "r"(mbar)
                 : "memory");
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst + 16),
                 "f"(u.o.m), "f"(u.o.s), "f"(u.a), "f"(u.twice), "r"(mbar)
                 : "memory");
}

// a term scaled by a weight; an infinite one whose weight vanished is 0
__device__ __forceinline__ float weighted(float a, float f) { return f == 0.f ? 0.f : a * f; }

// u.a when mt and ms become those given, f = 2^((u.t.m - mt) c)
__device__ __forceinline__ float moved(const Sums& u, float mt, float ms, float f, float inv_t) {
    if (u.t.s == 0.f) return 0.f;
    return weighted(fmaf(u.t.s, ((u.t.m - mt) - (u.s.m - ms)) * inv_t, u.a), f);
}

// Adds an entry of the record: the teacher's logit and the student's.
__device__ __forceinline__ void add_entry(Sums& u, float tv, float v, float c, float inv_t) {
    if (tv > u.t.m || v > u.s.m) {
        const float mt = tv > u.t.m ? clamp_max(u.t.m, tv) : u.t.m, ms = v > u.s.m ? clamp_max(u.s.m, v) : u.s.m;
        const float f = ex2((u.t.m - mt) * c);
        u.a = moved(u, mt, ms, f, inv_t);
        u.t = {mt, u.t.s * f};
        u.s = {ms, u.s.s * ex2((u.s.m - ms) * c)};
    }
    const float e = ex2((tv - u.t.m) * c);
    u.t.s += e;
    u.s.s += ex2((v - u.s.m) * c);
    if (e != 0.f) u.a += e * ((tv - u.t.m) - (v - u.s.m)) * inv_t;
}

__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float c, float inv_t) {
    Sums r;
    r.t = join(x.t, y.t, c);
    r.s = join(x.s, y.s, c);
    r.o = join(x.o, y.o, c);
    r.a = moved(x, r.t.m, r.s.m, ex2((x.t.m - r.t.m) * c), inv_t) + moved(y, r.t.m, r.s.m, ex2((y.t.m - r.t.m) * c), inv_t);
    r.twice = fmaxf(x.twice, y.twice);
    return r;
}

// The warp's join of its lanes' sums: the maxima first, then one rescaling and
// plain sums (a third of the exponentials and half of the latency of five
// pairwise joins).  Every lane gets it.
__device__ __forceinline__ Sums warp_join(Sums u, float c, float inv_t) {
    const float mt = warp_max(u.t.m), ms = warp_max(u.s.m), mo = warp_max(u.o.m);
    const float ft = ex2((u.t.m - mt) * c);
    u.a = moved(u, mt, ms, ft, inv_t);
    u.t = {mt, u.t.s * ft};
    u.s = {ms, u.s.s * ex2((u.s.m - ms) * c)};
    u.o = {mo, u.o.s * ex2((u.o.m - mo) * c)};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        u.t.s += __shfl_xor_sync(0xffffffffu, u.t.s, o);
        u.a += __shfl_xor_sync(0xffffffffu, u.a, o);
        u.s.s += __shfl_xor_sync(0xffffffffu, u.s.s, o);
        u.o.s += __shfl_xor_sync(0xffffffffu, u.o.s, o);
    }
    return u;
}

// The teacher's two parts on the larger one's scale, e^(level): `part` times
// t.s and part_r; rest = -inf where there is none.
struct Teacher {
    float part, part_r, inv_w;  // and the reciprocal of their sum
    float d;                    // mt / T - rest
};
__device__ __forceinline__ Teacher teacher(const Sums& u, float rest, float inv_t) {
    Teacher r = {1.f, 0.f, 0.f, INFINITY};
    if (rest != -INFINITY) {
        r.d = u.t.s == 0.f ? -INFINITY : fmaf(u.t.m, inv_t, -rest);
        const float e = ex2(-fabsf(r.d) * kLog2e);  // NaN stays NaN
        r.part = r.d >= 0.f ? 1.f : e;
        r.part_r = r.d >= 0.f ? e : 1.f;
    }
    r.inv_w = 1.f / (u.t.s * r.part + r.part_r);
    return r;
}
__device__ __forceinline__ bool has_target(const Sums& u, float rest) { return !(u.t.s == 0.f && rest == -INFINITY); }

// What the gradient goes by, from the row's sums.
__device__ __forceinline__ Stats finish(const Sums& u, float rest, float inv_t, float c) {
    Stats st = {};
    if (!has_target(u, rest)) return st;
    const Teacher w = teacher(u, rest, inv_t);
    const float pr = w.part_r * w.inv_w;
    const MaxSum x = join(u.s, u.o, c);
    st.has = 1.f;
    st.mt = u.t.m;
    st.pt = w.part * w.inv_w;
    st.mx = x.m;
    st.qx = 1.f / x.s;
    st.mo = u.o.m;
    st.co = ex2((u.o.m - x.m) * c) * st.qx;
    if (pr != 0.f) st.co = u.o.s == 0.f ? 0.f : st.co - pr / u.o.s;
    return st;
}

// The row's loss, from the same sums.
__device__ __forceinline__ float row_loss(const Sums& u, float rest, float inv_t, float c) {
    if (!has_target(u, rest)) return 0.f;
    const Teacher w = teacher(u, rest, inv_t);
    const float pr = w.part_r * w.inv_w;
    const MaxSum x = join(u.s, u.o, c);
    const float ps = u.t.s * w.part * w.inv_w;
    float l = logf(x.s * w.inv_w);
    if (ps != 0.f) l += weighted(u.a, w.part) * w.inv_w + ps * ((x.m - u.s.m) * inv_t + fminf(w.d, 0.f));
    if (pr != 0.f) l += pr * ((x.m - u.o.m) * inv_t - fmaxf(w.d, 0.f) - logf(u.o.s));
    return l;
}

// Records that name an id of the slice [v0, v0 + n) more than once: one warp goes
// through the record, 32 entries a step, forwards or from the end, and calls
// f(k, id, a) for the entries of the slice, a their place in it, of which the
// lowest k where several of a step name one id.  What f does in one step is seen
// by all lanes in the next, so f can tell by a bit whether an id came before, or,
// backwards, write over what a later entry wrote.  8192 entries are 256 steps; a
// scan of all earlier entries for each took 12 ms.
template <bool kForwards, typename F>
__device__ __forceinline__ void walk(const int32_t* ids, int K, int v0, int n, F&& f) {
    const int lane = (int)threadIdx.x & 31, steps = (K + 31) / 32;
    const auto entry = [&](int i) { return (kForwards ? i : steps - 1 - i) * 32 + lane; };
    const auto load = [&](int i) { return i < steps && entry(i) < K ? ids[entry(i)] : -1; };
    int id = load(0);
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
        const int next = load(i + 1);
        const unsigned a = (unsigned)id - (unsigned)v0;
        const bool in = a < (unsigned)n;
        const unsigned peers = __match_any_sync(0xffffffffu, in ? a : 0x80000000u + lane);
        if (in && (peers & ((1u << lane) - 1u)) == 0) f(entry(i), id, a);
        __syncwarp();
        id = next;
    }
}

// ---- loss and gradient at once ---------------------------------------------------
//
// A cluster of CTAs holds one row in shared memory, a slice each: a bulk copy
// brings it in, the sums are a pass over shared memory, the cluster's CTAs send
// theirs into each other's shared memory, and a second pass writes the gradient.
// So the logits are read once and the gradient is written once, which is all the
// traffic there is: 3840 rows of 151,936 bf16 logits in 370 us, 6.3 TB/s, 0.94 of
// the measured copy rate (349 us); 15 rows in 8.2 us.
//
// What bounds it is HBM, and how long a slice stays in shared memory.  Hence
// slices of 40 KB, of which five fit an SM, in one wave of clusters that take rows
// in turn (20 and 80 KB: 438 and 437 us; 192 and 256 threads: 400 and 410); the
// sums by stores that count on the reader's barrier (with a barrier of the cluster,
// which also waits for the last row's gradient to arrive in memory: 433 us instead
// of 367); the gradient straight to memory, so that the buffer is free once it is
// read; everything of a row that is not its logits read a row ahead, two entries of
// the record a thread; the loss after the gradient's factors.  Forms tried while
// the step took about 500 to 600 us and not since: the gradient through the buffer
// and a bulk copy, 60 us more; two half-size buffers per CTA in clusters of 16,
// 744 us; the row read twice from global memory (the second time from L2), 564 us.
//
// Records above 256 entries go through loops without reads ahead: 15 rows with
// K = 2048 take 16.6 us, with K = 8192 47 us, 960 rows with K = 2048 262 us.
//
// The forward alone streams its rows instead (below): when it took 66 us for 960
// rows, this kernel without its second pass took 87 us.
//
// Entries of the record are taken out of the slice (set to -inf) once their
// logits are read, so that the first pass is a plain sum over the outside.

constexpr int kSliceBytes = 40 * 1024;
constexpr unsigned kNone = 0xFFFFFFFFu;
constexpr int kStepThreads = 128;
constexpr int kHeld = 2;  // entries of a record that a thread holds; later ones are read again
constexpr int kStepWarps = kStepThreads / 32;
struct StepShared {
    Sums part[2][kMaxCluster * kStepWarps];  // every warp of the row, by the row's parity
    Stats row;
    unsigned long long bar;          // the row's copy has come
    unsigned long long exchange[2];  // the row's sums have come, by the row's parity
    int twice, abort;
};

// Adds U vectors to a set: one look at their maximum, then the exponentials.
template <int U, typename T>
__device__ __forceinline__ void add_vectors(float& m, F2& s, const Vec16<T>* v, float c, F2 cc) {
    const float top = top_of<U>(v);
    if (top > m) {
        const float to = clamp_max(m, top), f = ex2((m - to) * c);
        s = mul2(s, f2(f, f));
        m = to;
    }
    const F2 minus = f2(-m, -m);
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int k = 0; k < Vec16<T>::kElems / 2; ++k) s = add2(s, ex2x2(mul2(add2(v[j].pair(k), minus), cc)));
}

// The set of the values of shared vectors (this thread's of them).
template <typename T>
__device__ __forceinline__ MaxSum sum_vectors(const uint4* vec, int nvec, float c) {
    constexpr int U = 4;
    const F2 cc = f2(c, c);
    float m = -FLT_MAX;
    F2 s = f2(0.f, 0.f);
    int i = threadIdx.x;
#pragma unroll 1
    for (; i + (U - 1) * kStepThreads < nvec; i += U * kStepThreads) {
        Vec16<T> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j].q = vec[i + j * kStepThreads];
        add_vectors<U>(m, s, v, c, cc);
    }
#pragma unroll 1
    for (; i < nvec; i += kStepThreads) {
        Vec16<T> v;
        v.q = vec[i];
        add_vectors<1>(m, s, &v, c, cc);
    }
    const float2 h = halves(s);
    return {m, h.x + h.y};
}

template <typename T>
__global__ void __launch_bounds__(kStepThreads, 8) k_step(DistillArgs p, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ StepShared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, stride = gridDim.x / size;
    const float inv_t = 1.f / p.temperature, c = kLog2e / p.temperature;
    const uint32_t buffer = (uint32_t)chunk * sizeof(T) + 32;
    unsigned* bits = reinterpret_cast<unsigned*>(smem + buffer);
    const uint32_t bar = tc::smem_u32(&S.bar);
    const auto slice = [&](int n) {
        return Slice<T>(static_cast<const T*>(p.x) + (size_t)n * p.ld, p.V, chunk, rank, smem);
    };
    const auto request = [&](const Slice<T>& x) {  // one thread, after a barrier behind the buffer's last use
        tc::fence_proxy_async();
        const uint32_t bytes = (uint32_t)x.body * sizeof(T);
        tc::mbar_arrive_expect_tx(bar, bytes);
        if (bytes) tc::bulk_load(tc::smem_u32(x.data + x.head), x.src + x.head, bytes, bar, tc::policy_evict_normal());
    };
    // what is read ahead of a row: its weight, its rest and this thread's first entries
    struct Ahead {
        float weight, rest, top[kHeld];
        int id[kHeld];
    };
    const auto ahead = [&](int n) {
        Ahead a;
        a.weight = 0.f;
        a.rest = -INFINITY;
        if (n < p.n) {
            a.weight = p.weight[n];
            if (p.rest) a.rest = p.rest[n];
#pragma unroll
            for (int j = 0; j < kHeld; ++j) {
                const int k = t + j * kStepThreads;
                a.id[j] = k < p.K ? p.ids[(size_t)n * p.K + k] : -1;
                a.top[j] = k < p.K ? p.top[(size_t)n * p.K + k] : 0.f;
            }
        }
        return a;
    };
    int n = blockIdx.x / size;
    Ahead now = ahead(n);
    if (t == 0) {
        tc::mbar_init(bar, 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(tc::smem_u32(&S.exchange[i]), 1);
        S.twice = S.abort = 0;
        tc::fence_barrier_init();
        if (now.weight != 0.f) request(slice(n));
    }
    if (now.weight != 0.f) slice(n).load_edges();
    for (int i = t; i < chunk / 32; i += kStepThreads) bits[i] = 0;
    cluster_barrier();  // every CTA of the cluster is running
    uint32_t turn = 0;  // rows so far that had weight
    for (; n < p.n; n += stride) {
        const Ahead next = ahead(n + stride);
        const Slice<T> x = slice(n);
        T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d + x.v0;
        const bool together = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x.src)) & 15) == 0;
        float w = 0.f, held[kHeld] = {};  // held: the logits of this thread's first entries; later entries' are read again
        bool twice = false;
        if (now.weight != 0.f) {
            const int32_t* ids = p.ids + (size_t)n * p.K;
            const float* top = p.top + (size_t)n * p.K;
            // entry k of the record (this thread's first is held): its place in the slice, or none
            const auto place = [&](int id) {
                const unsigned a = (unsigned)id - (unsigned)x.v0;
                return a < (unsigned)x.n ? a : kNone;
            };
            const auto mark = [&](int id) {
                const unsigned a = place(id);
                if (a != kNone) {
                    const unsigned bit = 1u << (a & 31);
                    if (atomicOr(&bits[a >> 5], bit) & bit) S.twice = 1;
                } else if (rank == 0 && id != -1 && (unsigned)id >= (unsigned)p.V) {
                    atomicOr(p.err, kErrBadToken);
                }
            };
#pragma unroll
            for (int j = 0; j < kHeld; ++j) mark(now.id[j]);
#pragma unroll 1
            for (int k = t + kHeld * kStepThreads; k < p.K; k += kStepThreads) mark(ids[k]);
            const uint32_t phase = turn & 1;  // of the copy, and which exchange it is
            if (t == 0) tc::mbar_wait(bar, phase, &S.abort, p.err);
            __syncthreads();
            twice = S.twice != 0;

            Sums u = no_sums();
            const auto gather = [&](unsigned a, float tv) {
                const float v = to_f32(x.data[a]);
                x.data[a] = from_f32<T>(-INFINITY);  // no part of the outside
                add_entry(u, tv, v, c, inv_t);
                return v;
            };
            const auto gather_once = [&](int id, float tv) {
                const unsigned a = place(id);
                if (a == kNone) return 0.f;
                bits[a >> 5] = 0;
                return gather(a, tv);
            };
            if (!twice) {
#pragma unroll
                for (int j = 0; j < kHeld; ++j) held[j] = gather_once(now.id[j], now.top[j]);
#pragma unroll 1
                for (int k = t + kHeld * kStepThreads; k < p.K; k += kStepThreads) gather_once(ids[k], top[k]);
            } else if (warp == 0) {
                walk<true>(ids, p.K, x.v0, x.n, [&](int k, int, unsigned a) {
                    const unsigned bit = 1u << (a & 31);
                    if (!(bits[a >> 5] & bit)) return;
                    gather(a, top[k]);
                    atomicAnd(&bits[a >> 5], ~bit);
                });
            }
            __syncthreads();
            if (t == 0) S.twice = 0;
            u.o = sum_vectors<T>(x.vec, x.nvec, c);
            u = warp_join(u, c, inv_t);
            // every warp's sums to every CTA of the row
            // (to the other place than the last row's: who sends for this row has seen
            // every CTA's sums of the last one, so all have read those of the one before)
            if (t == 0) tc::mbar_arrive_expect_tx(tc::smem_u32(&S.exchange[phase]), size * kStepWarps * sizeof(Sums));
            if (lane < size) send(u, &S.part[phase][rank * kStepWarps + warp], &S.exchange[phase], lane);
            if (warp == 0) {
                tc::mbar_wait(tc::smem_u32(&S.exchange[phase]), turn >> 1 & 1, &S.abort, p.err);
                const Sums* part = S.part[phase];
                u = part[min(lane, size * kStepWarps - 1)];
                if (lane >= size * kStepWarps) u = no_sums();
                for (int i = lane + 32; i < size * kStepWarps; i += 32) u = join(u, part[i], c, inv_t);
                u = warp_join(u, c, inv_t);
                const Stats st = finish(u, now.rest, inv_t, c);
                if (lane == 0) S.row = st;
            }
            __syncthreads();
            if (rank == 0 && warp == 0) {
                const float loss = row_loss(u, now.rest, inv_t, c);
                if (lane == 0) p.loss[n] = loss;
            }
            ++turn;
            const Stats st = S.row;
            w = st.has == 0.f ? 0.f : now.weight * inv_t;
            if (w != 0.f) {
                // the gradient straight to memory: the buffer is free as soon as it is read
                const float wc = w * st.co;
                const F2 cc = f2(c, c), minus = f2(-st.mo, -st.mo), scale = f2(wc, wc);
                if (together) {
                    constexpr int P = Vec16<T>::kElems / 2;
                    uint4* out = reinterpret_cast<uint4*>(dx + x.head);
                    const uint4* in = reinterpret_cast<const uint4*>(x.data + x.head);
#pragma unroll 2
                    for (int i = t; i < x.body / Vec16<T>::kElems; i += kStepThreads) {
                        Vec16<T> v, g;
                        v.q = in[i];
#pragma unroll
                        for (int k = 0; k < P; ++k) g.set(k, mul2(scale, ex2x2(mul2(add2(v.pair(k), minus), cc))));
                        out[i] = g.q;
                    }
                }
                // the elements beside whole vectors, or all where the two rows start differently modulo 16 bytes
                const int beside = x.n - (together ? x.body : 0);
                for (int i = t; i < beside; i += kStepThreads) {
                    const int e = together && i >= x.head ? i + x.body : i;
                    dx[e] = from_f32<T>(wc * ex2((to_f32(x.data[e]) - st.mo) * c));
                }
            }
        } else if (rank == 0 && t == 0) {
            p.loss[n] = 0.f;
        }
        if (w == 0.f) {
            if (together) {
                uint4* out = reinterpret_cast<uint4*>(dx + x.head);
                for (int i = t; i < x.body / Vec16<T>::kElems; i += kStepThreads) out[i] = make_uint4(0, 0, 0, 0);
            }
            const int beside = x.n - (together ? x.body : 0);
            for (int i = t; i < beside; i += kStepThreads)
                dx[together && i >= x.head ? i + x.body : i] = from_f32<T>(0.f);
        }
        __syncthreads();  // the buffer is read, and the outside's gradient written
        if (S.abort) break;  // a copy or a peer's sums never came: no further rows, so that no further copy is asked for
        if (next.weight != 0.f) {
            const Slice<T> y = slice(n + stride);
            if (t == 0) request(y);
            y.load_edges();
        }
        if (w != 0.f) {  // the record's entries over it
            const int32_t* ids = p.ids + (size_t)n * p.K;
            const float* top = p.top + (size_t)n * p.K;
            const Stats st = S.row;
            const auto entry = [&](int id, float tv, float v) {
                const float q = st.qx * ex2((v - st.mx) * c), pk = st.pt * ex2((tv - st.mt) * c);
                dx[id - x.v0] = from_f32<T>(w * (q - pk));
            };
            const auto here = [&](int id) { return (unsigned)id - (unsigned)x.v0 < (unsigned)x.n; };
            if (!twice) {
#pragma unroll
                for (int j = 0; j < kHeld; ++j)
                    if (here(now.id[j])) entry(now.id[j], now.top[j], held[j]);
#pragma unroll 1
                for (int k = t + kHeld * kStepThreads; k < p.K; k += kStepThreads)
                    if (here(ids[k])) entry(ids[k], top[k], to_f32(x.src[ids[k] - x.v0]));
            } else if (warp == 0) {
                walk<false>(ids, p.K, x.v0, x.n, [&](int k, int id, unsigned a) { entry(id, top[k], to_f32(x.src[a])); });
            }
        }
        now = next;
    }
    // after a break: the row's own copy, the last one asked for
    if (t == 0 && S.abort) last_chance(bar, (turn & 1) ^ 1);
    cluster_barrier();  // nobody leaves before all have their sums
}

// ---- forward by itself ---------------------------------------------------------------
//
// Every thread streams 16-byte vectors of its CTA's slice of the row, and skips
// the record's entries by a bit per element, one byte (half a byte) of which
// covers a vector.  A row is one CTA's, or a cluster's where there are few rows
// (until 4 CTAs an SM) or its slices would pass 160 KB; only rank 0 waits for the
// others' sums.  960 rows of 151,936 bf16 logits, 0.29 GB: 57 us, 5.1 TB/s, 0.76 of
// the measured copy rate; 240 fp32 rows of 79,999: 21 us.  What bounds it is how the
// CTAs start and end, and instructions (0.73 of the issue slots): without the masks
// and the additions it was 5 us faster.  Hence the first vectors are asked for
// before the record is read (else 5 us more), and the sums go by stores that count
// on rank 0's barrier (with barriers of the cluster 51 us instead of 47 for forward
// and backward of the fp32 rows).  For both directions, 156 and 47.2 us: 128 threads
// 166 and 47.7 us; 2 vectors at once and 3 stages 157 and 48.1 us.

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;
constexpr int kStages = 2;
constexpr size_t kRingBytes = (size_t)kThreads * kAhead * kStages * 16;

struct StreamShared {
    Sums part[kMaxCluster * kWarps];  // every warp of the row, at rank 0
    unsigned long long bar;           // they have come
    int twice, abort;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_forward(DistillArgs p, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ StreamShared S;
    uint4* ring = reinterpret_cast<uint4*>(smem);
    unsigned* bits = reinterpret_cast<unsigned*>(smem + kRingBytes);
    constexpr int kPer = Vec16<T>::kElems;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int n = blockIdx.x / size, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const float inv_t = 1.f / p.temperature, c = kLog2e / p.temperature;
    const int v0 = min(p.V, rank * chunk);
    const Vectors<T> x(static_cast<const T*>(p.x) + (size_t)n * p.ld + v0, min(p.V, v0 + chunk) - v0);
    // the first vectors are on their way while the record is read
    Streamer<kThreads, kAhead, kStages, false, T> vectors(x, ring);
    const int32_t* ids = p.ids + (size_t)n * p.K;
    const float* top = p.top + (size_t)n * p.K;

    const float rest = p.rest ? p.rest[n] : -INFINITY;
    for (int i = t; i <= (x.phase + x.n) / 32; i += kThreads) bits[i] = 0;
    if (t == 0) {
        S.twice = S.abort = 0;
        tc::mbar_init(tc::smem_u32(&S.bar), 1);
        tc::fence_barrier_init();
    }
    __syncthreads();
    if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
#pragma unroll 1
    for (int k = t; k < p.K; k += kThreads) {
        const int id = ids[k];
        const unsigned a = (unsigned)id - (unsigned)v0;
        if (a < (unsigned)x.n) {
            const unsigned b = a + x.phase, bit = 1u << (b & 31);
            if (atomicOr(&bits[b >> 5], bit) & bit) S.twice = 1;
        } else if (rank == 0 && id != -1 && (unsigned)id >= (unsigned)p.V) {
            atomicOr(p.err, kErrBadToken);
        }
    }
    __syncthreads();
    const bool twice = S.twice != 0;
    Sums u = no_sums();
    const auto gather = [&](unsigned a, float tv) { add_entry(u, tv, to_f32(x.src[a]), c, inv_t); };
    if (!twice) {
#pragma unroll 1
        for (int k = t; k < p.K; k += kThreads) {
            const unsigned a = (unsigned)ids[k] - (unsigned)v0;
            if (a < (unsigned)x.n) gather(a, top[k]);
        }
    } else {
        // the bits once more, in the order of the record
        for (int k = t; k < p.K; k += kThreads) {
            const unsigned a = (unsigned)ids[k] - (unsigned)v0, b = a + x.phase;
            if (a < (unsigned)x.n) bits[b >> 5] = 0;
        }
        __syncthreads();
        if (warp == 0)
            walk<true>(ids, p.K, v0, x.n, [&](int k, int, unsigned a) {
                const unsigned b = a + x.phase, bit = 1u << (b & 31);
                if (atomicOr(&bits[b >> 5], bit) & bit) return;
                gather(a, top[k]);
            });
        __syncthreads();
    }
    // the outside
    const unsigned char* masks = reinterpret_cast<const unsigned char*>(bits);
    const F2 cc = f2(c, c);
    F2 s = f2(0.f, 0.f);
    vectors.run([&](int i0, Vec16<T>* v, auto all) {
        unsigned m[kAhead], any = 0;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kThreads;
            m[j] = all() || i < x.last ? (kPer == 8 ? masks[i] : masks[i >> 1] >> (i & 1) * 4 & 15u) : 0u;
            any |= m[j];
        }
        if (any) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) strike(v[j], m[j]);
        }
        add_vectors<kAhead>(u.o.m, s, v, c, cc);
    });
    const float2 h = halves(s);
    u.o.s = h.x + h.y;
    const int side = t < 2 * kPer ? x.beside(t) : x.n;
    if (side < x.n && !(bits[(side + x.phase) >> 5] >> ((side + x.phase) & 31) & 1u)) add(u.o, to_f32(x.src[side]), c);
    u = warp_join(u, c, inv_t);
    // every warp's sums to rank 0, which is running by now; the others are done
    u.twice = twice ? 1.f : 0.f;
    const int parts = size * kWarps;
    if (size > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank == 0 && t == 0) tc::mbar_arrive_expect_tx(tc::smem_u32(&S.bar), parts * sizeof(Sums));
        if (lane == 0) send(u, &S.part[rank * kWarps + warp], &S.bar, 0);
        if (rank != 0 || warp != 0) return;
        const bool came = tc::mbar_wait(tc::smem_u32(&S.bar), 0, &S.abort, p.err);
        if (!__all_sync(0xffffffffu, came)) {
            // who was late sends all the same: this CTA's shared memory stays until the others have left
            cluster_barrier();
            last_chance(tc::smem_u32(&S.bar), 0);
        }
    } else {
        if (lane == 0) S.part[warp] = u;
        __syncthreads();
        if (warp != 0) return;
    }
    u = S.part[min(lane, parts - 1)];
    if (lane >= parts) u = no_sums();
    for (int i = lane + 32; i < parts; i += 32) u = join(u, S.part[i], c, inv_t);
    u = warp_join(u, c, inv_t);
    const bool any_twice = __any_sync(0xffffffffu, u.twice != 0.f);
    Stats st = finish(u, rest, inv_t, c);
    st.twice = any_twice ? 1.f : 0.f;
    const float loss = row_loss(u, rest, inv_t, c);
    if (lane == 0) {
        p.loss[n] = loss;
        reinterpret_cast<Stats*>(p.stats)[n] = st;
    }
}

// ---- backward by itself -------------------------------------------------------------
//
// Every thread streams 16-byte vectors of its block's slice of the row, writes
// every element as if it were outside the record and then, after a barrier, the
// record's entries again.  A row is one block's, or several where there are few
// rows (until 4 blocks an SM) or its slices would pass 160 KB.  Bound by HBM: 960
// rows of 151,936 bf16 logits, 0.58 GB, in 90 us alone, 6.5 TB/s, 0.97 of the
// measured copy rate (96 us in calls after one another, whose writes still leave L2
// when the next begins).

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_backward(DistillArgs p, int chunk, int size) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int P = Vec16<T>::kElems / 2, kPer = Vec16<T>::kElems;
    const int n = blockIdx.x / size, v0 = min(p.V, (int)(blockIdx.x % size) * chunk), t = threadIdx.x;
    const float inv_t = 1.f / p.temperature, c = kLog2e / p.temperature;
    const Vectors<T> x(static_cast<const T*>(p.x) + (size_t)n * p.ld + v0, min(p.V, v0 + chunk) - v0);
    T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d + v0;
    const bool together = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x.src)) & 15) == 0;
    uint4* out = reinterpret_cast<uint4*>(dx - x.phase);
    const int side = t < 2 * kPer ? x.beside(t) : x.n;
    const Stats st = reinterpret_cast<const Stats*>(p.stats)[n];
    const float w = st.has == 0.f ? 0.f : p.weight[n] * inv_t;
    if (w == 0.f) {
        if (together) {
            for (int i = x.first + t; i < x.last; i += kThreads) out[i] = make_uint4(0, 0, 0, 0);
            if (side < x.n) dx[side] = from_f32<T>(0.f);
        } else {
            for (int i = t; i < x.n; i += kThreads) dx[i] = from_f32<T>(0.f);
        }
        return;
    }
    const float wc = w * st.co;
    const F2 cc = f2(c, c), minus = f2(-st.mo, -st.mo), scale = f2(wc, wc);
    if (together) {
        stream<kThreads, kAhead, kStages>(x, reinterpret_cast<uint4*>(smem), [&](int i0, Vec16<T>* v, auto all) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                Vec16<T> g;
#pragma unroll
                for (int k = 0; k < P; ++k) g.set(k, mul2(scale, ex2x2(mul2(add2(v[j].pair(k), minus), cc))));
                if (all() || i0 + j * kThreads < x.last) out[i0 + j * kThreads] = g.q;
            }
        });
        if (side < x.n) dx[side] = from_f32<T>(wc * ex2((to_f32(x.src[side]) - st.mo) * c));
    } else {
        for (int i = t; i < x.n; i += kThreads) dx[i] = from_f32<T>(wc * ex2((to_f32(x.src[i]) - st.mo) * c));
    }
    __syncthreads();
    const int32_t* ids = p.ids + (size_t)n * p.K;
    const float* top = p.top + (size_t)n * p.K;
    const auto entry = [&](unsigned a, float tv) {
        const float q = st.qx * ex2((to_f32(x.src[a]) - st.mx) * c), pk = st.pt * ex2((tv - st.mt) * c);
        dx[a] = from_f32<T>(w * (q - pk));
    };
    if (st.twice == 0.f) {
#pragma unroll 1
        for (int k = t; k < p.K; k += kThreads) {
            const unsigned a = (unsigned)ids[k] - (unsigned)v0;
            if (a < (unsigned)x.n) entry(a, top[k]);
        }
    } else if (t < 32) {
        walk<false>(ids, p.K, v0, x.n, [&](int k, int, unsigned a) { entry(a, top[k]); });
    }
}

template <typename T>
cudaError_t launch_forward(domino_train_ctx* ctx, const DistillArgs& a, cudaStream_t st) {
    int size = 1;
    while (size < kMaxCluster && (long long)a.n * size < 4 * ctx->num_sms && slice_of(a.V, 2 * size) >= 2048) size *= 2;
    while (size < kMaxCluster && slice_of(a.V, size) * (int)sizeof(T) > 160 * 1024) size *= 2;
    const int chunk = slice_of(a.V, size);
    const size_t smem = kRingBytes + (size_t)chunk / 8 + 8;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_config((unsigned)a.n * size, kThreads, size, smem, st, &attr);
    ctx->last_launches = 1;
    return cudaLaunchKernelEx(&cfg, k_forward<T>, a, chunk);
}

template <typename T>
cudaError_t launch_backward(domino_train_ctx* ctx, const DistillArgs& a, cudaStream_t st) {
    int size = 1;
    while (size < 64 && (long long)a.n * size < 4 * ctx->num_sms && slice_of(a.V, 2 * size) >= 2048) size *= 2;
    while (slice_of(a.V, size) * (int)sizeof(T) > 160 * 1024) size *= 2;
    k_backward<T><<<(unsigned)a.n * size, kThreads, kRingBytes, st>>>(a, slice_of(a.V, size), size);
    ctx->last_launches = 1;
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step(domino_train_ctx* ctx, const DistillArgs& a, cudaStream_t st) {
    int size = 1;
    while (size < kMaxCluster && slice_of(a.V, size) * (int)sizeof(T) > kSliceBytes) size *= 2;
    while (size < kMaxCluster && (long long)a.n * size < 2 * ctx->num_sms && slice_of(a.V, 2 * size) >= 4096) size *= 2;
    const int chunk = slice_of(a.V, size);
    const size_t smem = (size_t)chunk * sizeof(T) + 32 + (size_t)chunk / 8;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = cluster_config(size, kStepThreads, size, smem, st, &attr);
    // one wave of clusters, each taking rows in turn; how many the GPU holds at
    // once depends on how its SMs are grouped, so it is asked (once per context
    // and cluster size)
    int& most = ctx->step_clusters[size];
    if (most == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&most, k_step<T>, &cfg);
        if (e != cudaSuccess) return e;
        if (most < 1) most = 1;
    }
    cfg.gridDim = dim3((unsigned)(a.n < most ? a.n : most) * size);
    ctx->last_launches = 1;
    return cudaLaunchKernelEx(&cfg, k_step<T>, a, chunk);
}

}  // namespace

cudaError_t prepare_distill_kernels() {
    cudaError_t e = allow_all(k_step<float>);
    if (e == cudaSuccess) e = allow_all(k_step<__nv_bfloat16>);
    if (e == cudaSuccess) e = allow_all(k_forward<float>);
    if (e == cudaSuccess) e = allow_all(k_forward<__nv_bfloat16>);
    return e;
}

cudaError_t launch_distill_forward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_forward<__nv_bfloat16>(c, a, st) : launch_forward<float>(c, a, st);
}
cudaError_t launch_distill_backward(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_backward<__nv_bfloat16>(c, a, st) : launch_backward<float>(c, a, st);
}
cudaError_t launch_distill_step(domino_train_ctx* c, const DistillArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_step<__nv_bfloat16>(c, a, st) : launch_step<float>(c, a, st);
}

}  // namespace train
}  // namespace domino
