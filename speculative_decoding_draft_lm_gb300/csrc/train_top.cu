// Record of a teacher's logits: the K largest of each row, ids ascending, and
// the log-sum-exp of all the others.
//
// Order: (logit descending, id ascending), with NaN above everything and the
// two zeros equal; a 64-bit word, orderable logit over inverted id, has that
// order.
//
// One pass over the row.  A CTA streams its slice and keeps the words that beat
// a bound, the K-th best so far, in a buffer in shared memory; when the buffer
// is full an exact radix select leaves the best K in it and raises the bound.
// Ids only grow along the stream, so after a select an equal logit is too late:
// the test of the stream is one comparison of a vector's maximum with the
// bound.  In a row without order the j-th piece passes K / j words, so the
// selects are few and most of the time goes into the exponentials of the
// others, which are summed as they are turned away.  The rest is never formed
// as a difference of sums: a peaked teacher leaves less in it than the
// rounding of the whole.  Places in the buffer come from scans, not from
// atomics, so that equal calls sum in equal order.
//
// Few rows are spread over a cluster each: every CTA finds its slice's best K
// and rank 0 takes the others' through distributed shared memory, in the order
// of the slices.
#include <cooperative_groups.h>

#include "train_internal.h"
#include "train_stream.cuh"

namespace cg = cooperative_groups;

namespace domino {
namespace train {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 2;
constexpr int kStages = 3;
constexpr size_t kRingBytes = (size_t)kThreads * kAhead * kStages * 16;
constexpr int kBins = 2048;

__device__ __forceinline__ unsigned top_key(float x) { return x != x ? 0xFFFFFFFFu : ord_f32(x); }
__device__ __forceinline__ float key_logit(unsigned k) { return k == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : unord_f32(k); }
__device__ __forceinline__ unsigned word_id(unsigned long long w) { return ~(unsigned)w; }
__device__ __forceinline__ unsigned long long word_of(unsigned key, unsigned id) {
    return (unsigned long long)key << 32 | (unsigned)~id;
}

// elements of one call of the stream
template <typename T>
constexpr int call_elems() { return kThreads * kAhead * Vec16<T>::kElems; }
// words that the buffer holds before a select is due (even: the ring behind the
// buffer starts on 16 bytes)
__host__ __device__ constexpr int due_words(int K) { return ((2 * K > K + 512 ? 2 * K : K + 512) + 1) & ~1; }
static_assert(call_elems<float>() % 2 == 0 && call_elems<__nv_bfloat16>() % 2 == 0, "the ring's alignment");

struct TopShared {
    unsigned hist[kBins];
    unsigned warp[kWarps];
    unsigned digit, need, in_bin;
    MaxSum part[kWarps];
    MaxSum rest;   // the CTA's rest
    int count;     // the CTA's words
};

// Exclusive scan of one value per thread; *total gets the sum.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned* warp_tot, unsigned* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    unsigned before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const unsigned v = warp_tot[w];
        if (w < warp) before += v;
        all += v;
    }
    __syncthreads();
    *total = all;
    return before + incl - x;
}

// A CTA's selection in progress.  `bound` is the key of the K-th best word once
// K words were seen (0 before: every word passes, and so does the test `>`).
struct Selection {
    TopShared& S;
    unsigned long long* buf;
    int K, due;
    float c;
    unsigned bound;
    float bound_logit;
    int count;
    MaxSum rest;  // this thread's share of what was turned away

    __device__ Selection(TopShared& s, unsigned long long* b, int k, float scale)
        : S(s), buf(b), K(k), due(due_words(k)), c(scale), bound(0), bound_logit(-INFINITY), count(0), rest(empty_set()) {}

    // The digit of the `need`-th largest among the words that match prefix
    // under mask, its count and what remains to be found in it.  All threads.
    __device__ void pass(unsigned long long prefix, unsigned long long mask, int shift, int bins, unsigned need) {
        for (int i = threadIdx.x; i < bins; i += kThreads) S.hist[i] = 0;
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int i0 = 0; i0 < count; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            const unsigned long long w = i < count ? buf[i] : 0;
            const bool in = i < count && (w & mask) == prefix;
            const unsigned act = __ballot_sync(0xffffffffu, in);
            if (in) {
                const unsigned d = (unsigned)(w >> shift) & (unsigned)(bins - 1);
                const unsigned peers = __match_any_sync(act, d);
                if (lane == __ffs(peers) - 1) atomicAdd(&S.hist[d], (unsigned)__popc(peers));
            }
        }
        __syncthreads();
        // thread t holds the bins from the top down: bins-1 - t*per ...
        const int per = bins / kThreads;
        unsigned mine = 0;
        for (int j = 0; j < per; ++j) mine += S.hist[bins - 1 - (int)threadIdx.x * per - j];
        unsigned all;
        unsigned above = block_scan(mine, S.warp, &all);
        if (above < need && above + mine >= need) {
            int b = bins - 1 - (int)threadIdx.x * per;
            while (above + S.hist[b] < need) above += S.hist[b--];
            S.digit = (unsigned)b;
            S.need = need - above;
            S.in_bin = S.hist[b];
        }
        __syncthreads();
    }

    // Leaves the best K words at the front of the buffer.  All threads.
    template <bool kShort>  // keys with 16 significant bits
    __device__ void select() {
        if (count <= K) return;
        unsigned long long prefix = 0, mask = 0;
        unsigned need = (unsigned)K;
        // logit: 11 + 11 + 10 bits; inverted id: 10 + 10 bits (the bits above are all ones)
        const int shift[5] = {53, 42, 32, 10, 0};
        const int bits[5] = {11, 11, 10, 10, 10};
#pragma unroll 1
        for (int p = 0; p < 5; ++p) {
            if (p == 2 && kShort) {
                // a 16-bit logit's key ends in ten zeros, or ten ones if negative or NaN
                const bool ones = !(prefix >> 63) || prefix >> 42 == 0x3FFFFFull;
                prefix |= ones ? 0x3FFull << 32 : 0ull;
                mask |= 0x3FFull << 32;
                continue;
            }
            if (p == 3) {
                prefix |= 0xFFF00000ull;
                mask |= 0xFFF00000ull;
            }
            pass(prefix, mask, shift[p], 1 << bits[p], need);
            prefix |= (unsigned long long)S.digit << shift[p];
            mask |= (unsigned long long)((1u << bits[p]) - 1) << shift[p];
            need = S.need;
            if (S.in_bin == need) break;  // the whole bin belongs: everything from `prefix` up
        }
        // words in the buffer from `prefix` up are exactly K
        unsigned kept = 0;
        unsigned low = 0xFFFFFFFFu;
        for (int i0 = 0; i0 < count; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            const unsigned long long w = i < count ? buf[i] : 0;
            const bool keep = i < count && w >= prefix;
            if (i < count && !keep) add(rest, key_logit((unsigned)(w >> 32)), c);
            if (keep) low = min(low, (unsigned)(w >> 32));
            unsigned all;
            const unsigned at = kept + block_scan(keep, S.warp, &all);  // its barriers part the reads from the writes
            if (keep) buf[at] = w;
            kept += all;
        }
        low = __reduce_min_sync(0xffffffffu, low);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) S.warp[threadIdx.x >> 5] = low;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) low = min(low, S.warp[w]);
        __syncthreads();
        count = K;
        bound = low;
        bound_logit = key_logit(low);
    }

    // Takes the words that `n` says this thread has.  All threads; room for one
    // call's words is left below the buffer's end by the select.
    template <bool kShort, typename F>
    __device__ __forceinline__ void take(unsigned n, F&& write) {
        if (!__syncthreads_or((int)n)) return;
        unsigned all;
        const unsigned at = block_scan(n, S.warp, &all);
        if (n) write(buf + count + at);
        count += (int)all;
        if (count > due) {
            __syncthreads();
            select<kShort>();
        }
    }

    // One logit per thread, or none.
    template <bool kShort>
    __device__ void one(bool in, float x, unsigned id) {
        const unsigned k = in ? top_key(x) : 0u;
        const bool pass = in && k > bound;
        if (in && !pass) add(rest, x, c);
        take<kShort>(pass, [&](unsigned long long* to) { *to = word_of(k, id); });
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_top(const T* __restrict__ logits, long long ld, int V, int K,
                                                  float temperature, int32_t* __restrict__ ids,
                                                  float* __restrict__ top, float* __restrict__ rest, int chunk) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ TopShared S;
    constexpr bool kShort = sizeof(T) == 2;
    constexpr int kPer = Vec16<T>::kElems, P = kPer / 2;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int n = blockIdx.x / size, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    unsigned long long* buf = reinterpret_cast<unsigned long long*>(smem);
    uint4* ring = reinterpret_cast<uint4*>(buf + due_words(K) + call_elems<T>());
    const int v0 = min(V, rank * chunk);
    const Vectors<T> x(logits + (size_t)n * ld + v0, min(V, v0 + chunk) - v0);
    Selection sel(S, buf, K, kLog2e / temperature);

    // the elements in front of the first whole vector, the vectors, the elements behind the last
    const int head = min(x.n, (kPer - x.phase) % kPer);
    if (head) sel.one<kShort>(t < head, t < head ? to_f32(x.src[t]) : 0.f, (unsigned)(v0 + t));
    {
        MaxSum r = sel.rest;
        F2 s = f2(r.s, 0.f);
        const F2 cc = f2(sel.c, sel.c);
        sel.rest = empty_set();  // what selects turn away meanwhile
        stream<kThreads, kAhead, kStages>(x, ring, [&](int i0, Vec16<T>* v) {
            // a bit per element that beats the bound
            unsigned pass = 0;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (!(v[j].top_nan() <= sel.bound_logit) || sel.bound == 0) {
                    if (i0 + j * kThreads < x.last) {
#pragma unroll
                        for (int e = 0; e < kPer; ++e) {
                            const float2 f = halves(v[j].pair(e / 2));
                            if (top_key(e & 1 ? f.y : f.x) > sel.bound) pass |= 1u << (j * kPer + e);
                        }
                    }
                }
            }
            const unsigned count = (unsigned)__popc(pass);
            Vec16<T> kept[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                kept[j] = v[j];
                if (pass) strike(v[j], pass >> (j * kPer) & ((1u << kPer) - 1u));
            }
            // the others' exponentials
            float most = v[0].top();
#pragma unroll
            for (int j = 1; j < kAhead; ++j) most = fmaxf(most, v[j].top());
            if (most > r.m) {
                const float m = clamp_max(r.m, most), f = ex2((r.m - m) * sel.c);
                s = mul2(s, f2(f, f));
                r.m = m;
            }
            const F2 minus = f2(-r.m, -r.m);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int k = 0; k < P; ++k) s = add2(s, ex2x2(mul2(add2(v[j].pair(k), minus), cc)));
            sel.take<kShort>(count, [&](unsigned long long* to) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        if (pass >> (j * kPer + e) & 1u) {
                            const float2 f = halves(kept[j].pair(e / 2));
                            const int at = (i0 + j * kThreads) * kPer - x.phase + e;
                            *to++ = word_of(top_key(e & 1 ? f.y : f.x), (unsigned)(v0 + at));
                        }
            });
        });
        const float2 h = halves(s);
        r.s = h.x + h.y;
        sel.rest = join(sel.rest, r, sel.c);
    }
    const int behind = max(head, x.last * kPer - x.phase);
    if (behind < x.n) {
        const int at = behind + t;
        sel.one<kShort>(at < x.n, at < x.n ? to_f32(x.src[at]) : 0.f, (unsigned)(v0 + at));
    }
    __syncthreads();
    sel.select<kShort>();

    if (size > 1) {
        if (t == 0) S.count = sel.count;
        cluster_barrier();
        if (rank == 0) {
            for (int r = 1; r < size; ++r) {
                const unsigned long long* from = cluster.map_shared_rank(buf, r);
                const int words = *cluster.map_shared_rank(&S.count, r);
                for (int i0 = 0; i0 < words; i0 += kThreads) {
                    const int i = i0 + t;
                    const unsigned long long w = i < words ? from[i] : 0;
                    const unsigned k = (unsigned)(w >> 32);
                    const bool pass = i < words && k > sel.bound;
                    if (i < words && !pass) add(sel.rest, key_logit(k), sel.c);
                    sel.take<kShort>(pass, [&](unsigned long long* to) { *to = w; });
                }
            }
            __syncthreads();
            sel.select<kShort>();
        }
    }
    // the CTA's rest
    {
        MaxSum r = sel.rest;
        const float m = warp_max(r.m);
        r.s = warp_sum(r.s * ex2((r.m - m) * sel.c));
        if (lane == 0) S.part[warp] = {m, r.s};
        __syncthreads();
        if (t == 0) {
            r = S.part[0];
            for (int w = 1; w < kWarps; ++w) r = join(r, S.part[w], sel.c);
            S.rest = r;
        }
    }
    if (size > 1) {
        cluster_barrier();
        if (rank == 0 && t == 0) {
            MaxSum r = S.rest;
            for (int i = 1; i < size; ++i) r = join(r, *cluster.map_shared_rank(&S.rest, i), sel.c);
            S.rest = r;
        }
        cluster_barrier();  // the others' shared memory was read
        if (rank != 0) return;
    }
    if (t == 0) rest[n] = S.rest.s == 0.f ? -INFINITY : S.rest.m / temperature + logf(S.rest.s);

    // ascending ids: a bit per id, counted in front of each thread's words of bits
    unsigned* bits = reinterpret_cast<unsigned*>(buf + K);  // what follows the record is free now
    unsigned* before = S.hist;
    const int words = (V + 31) / 32, per = (words + kThreads - 1) / kThreads;
    for (int i = t; i < per * kThreads; i += kThreads) bits[i] = 0;
    __syncthreads();
    for (int i = t; i < K; i += kThreads) {
        const unsigned id = word_id(buf[i]);
        atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    unsigned mine = 0, all;
    for (int j = 0; j < per; ++j) mine += (unsigned)__popc(bits[t * per + j]);
    before[t] = block_scan(mine, S.warp, &all);
    __syncthreads();
    for (int i = t; i < K; i += kThreads) {
        const unsigned long long w = buf[i];
        const unsigned id = word_id(w), at = id >> 5, owner = at / per;
        unsigned rk = before[owner] + (unsigned)__popc(bits[at] & ((1u << (id & 31)) - 1u));
        for (unsigned j = owner * per; j < at; ++j) rk += (unsigned)__popc(bits[j]);
        ids[(size_t)n * K + rk] = (int32_t)id;
        top[(size_t)n * K + rk] = key_logit((unsigned)(w >> 32));
    }
}

template <typename T>
cudaError_t launch(domino_train_ctx* c, const void* x, long long ld, int n, int K, float temperature, int32_t* ids,
                   float* top, float* rest, cudaStream_t st) {
    const int V = c->cfg.V;
    int size = 1;
    auto slice = [&](int parts) { return ((V + parts - 1) / parts + 63) / 64 * 64; };
    // few rows: spread them while the slices stay longer than what they keep
    while (size < kMaxCluster && (long long)n * size < 2 * c->num_sms && slice(2 * size) >= 2 * K + 2048) size *= 2;
    const size_t bits = (size_t)((V + 31) / 32 + kThreads) * 4;
    const size_t during = (size_t)(due_words(K) + call_elems<T>()) * 8 + kRingBytes, after = (size_t)K * 8 + bits;
    const size_t smem = during > after ? during : after;
    auto kern = k_top<T>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_config((unsigned)n * size, kThreads, size, smem, st, &attr);
    c->last_launches = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(x), ld, V, K, temperature, ids, top, rest, slice(size));
}

}  // namespace

cudaError_t launch_top(domino_train_ctx* c, const void* x, int dtype, long long ld, int n, int K, float temperature,
                       int32_t* ids, float* top, float* rest, cudaStream_t st) {
    return dtype == DOMINO_DTYPE_BF16 ? launch<__nv_bfloat16>(c, x, ld, n, K, temperature, ids, top, rest, st)
                                      : launch<float>(c, x, ld, n, K, temperature, ids, top, rest, st);
}

}  // namespace train
}  // namespace domino
