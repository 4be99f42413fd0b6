// Scores of rows of logits: the log probability of each row's token, the row's
// entropy and its most likely alternatives, and the gradient of the first two.
//
// With m the largest logit of a row, d_v = (x_v - m) / T, s = sum e^(d_v) and
// t = sum e^(d_v) d_v,
//   log q_v = d_v - log s,   H = log s - t / s,
//   T dx_v = g ([v = tok] - q_v) - h q_v (log q_v + H)
//          = g [v = tok] + e^(d_v) (a + b d_v),  a = -(g + h (H - log s)) / s,  b = -h / s.
// What all logits of a row share cancels in d, which is exact where it is small.
#include <cooperative_groups.h>

#include "train_internal.h"
#include "train_slice.cuh"
#include "train_stream.cuh"

namespace cg = cooperative_groups;

namespace domino {
namespace train {

namespace {

constexpr float kLn2 = 0.69314718055994531f;

// What a row's gradient goes by; row layout of `stats`.
struct LogprobStats {
    float m, inv_s;  // q = inv_s 2^((x - m) c); inv_s = 0: the row takes no part
    float log_s, entropy;
};
static_assert(sizeof(LogprobStats) == DOMINO_TRAIN_LOGPROB_STATS * sizeof(float), "stats row");

// A set of logits through its largest one, s and t (in units of the base-2 exponents).
struct alignas(16) Scores {
    float m, s, t, unused;
};
__device__ __forceinline__ Scores no_scores() { return {-FLT_MAX, 0.f, 0.f, 0.f}; }
// the same set from a larger m
__device__ __forceinline__ Scores moved(const Scores& a, float m, float c) {
    const float d = (a.m - m) * c, f = ex2(d);
    return {m, a.s * f, f == 0.f ? 0.f : f * fmaf(d, a.s, a.t), 0.f};
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
    return {m, a.s + b.s, a.t + b.t, 0.f};
}
// The warp's join: the maximum first, then plain sums.  Every lane gets it.
__device__ __forceinline__ Scores warp_join(Scores a, float c) {
    a = moved(a, warp_max(a.m), c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
        a.t += __shfl_xor_sync(0xffffffffu, a.t, o);
    }
    return a;
}

// ---- sums of many logits ---------------------------------------------------------
//
// In the stream a logit below kLow counts as kLow, so that no product of an
// exponential and its difference is 0 times infinity; as long as the largest logit
// lies between kFloor and -kFloor such a logit adds 0 either way.  Where it does not
// (rows masked throughout by the type's lowest value, infinite logits), the slice
// is summed once more, one logit at a time (add).
constexpr float kLow = -1e30f, kFloor = -1e29f;
__device__ __forceinline__ bool plain_range(float m) { return m > kFloor && m <= -kFloor; }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// the vector with kLow in the place of what is below it; NaN stays
__device__ __forceinline__ Vec16<float> raised(const Vec16<float>& v) {
    const auto one = [](uint32_t w) { return __float_as_uint(max_nan(__uint_as_float(w), kLow)); };
    Vec16<float> r;
    r.q = make_uint4(one(v.q.x), one(v.q.y), one(v.q.z), one(v.q.w));
    return r;
}
__device__ __forceinline__ Vec16<__nv_bfloat16> raised(const Vec16<__nv_bfloat16>& v) {
    const __nv_bfloat162 low = __float2bfloat162_rn(kLow);
    const auto two = [&](uint32_t w) {
        const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), low);
        return *reinterpret_cast<const uint32_t*>(&r);
    };
    Vec16<__nv_bfloat16> r;
    r.q = make_uint4(two(v.q.x), two(v.q.y), two(v.q.z), two(v.q.w));
    return r;
}

struct Running {
    float m = kFloor, top = -INFINITY;  // of the sums, and the largest logit
    F2 s = f2(0.f, 0.f), t = f2(0.f, 0.f);

    // U vectors whose largest logit is `high` (NaN among them or not)
    template <int U, typename T>
    __device__ __forceinline__ void add(const Vec16<T>* v, float high, float c, F2 cc) {
        if (high > m) {
            const float to = fminf(high, FLT_MAX), d = (m - to) * c, f = ex2(d);
            t = mul2(fma2(f2(d, d), s, t), f2(f, f));
            s = mul2(s, f2(f, f));
            m = to;
        }
        top = fmaxf(top, high);
        const F2 minus = f2(-m, -m);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const Vec16<T> x = raised(v[j]);
#pragma unroll
            for (int k = 0; k < Vec16<T>::kElems / 2; ++k) {
                const F2 d = mul2(add2(x.pair(k), minus), cc), e = ex2x2(d);
                s = add2(s, e);
                t = fma2(e, d, t);
            }
        }
    }
    __device__ __forceinline__ Scores scores() const {
        const float2 hs = halves(s), ht = halves(t);
        return {m, hs.x + hs.y, ht.x + ht.y, 0.f};
    }
};
// the largest logit of four vectors, NaN if any is
__device__ __forceinline__ float top4(const Vec16<float>* v) {
    float r = v[0].top_nan();
#pragma unroll
    for (int j = 1; j < 4; ++j) r = max_nan(r, v[j].top_nan());
    return r;
}
__device__ __forceinline__ float top4(const Vec16<__nv_bfloat16>* v) {
    const auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(v[0].q.x), h(v[0].q.y)), __hmax2_nan(h(v[0].q.z), h(v[0].q.w)));
#pragma unroll
    for (int j = 1; j < 4; ++j)
        m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(h(v[j].q.x), h(v[j].q.y)), __hmax2_nan(h(v[j].q.z), h(v[j].q.w))));
    return max_nan(__low2float(m), __high2float(m));
}
// a vector with one logit and nothing else
template <typename T>
__device__ __forceinline__ Vec16<T> alone(T x) {
    Vec16<T> v;
    const unsigned inf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    v.q = make_uint4(inf, inf, inf, inf);
    if (sizeof(T) == 2) v.q.x = 0xFF800000u | *reinterpret_cast<const uint16_t*>(&x);
    else v.q.x = *reinterpret_cast<const uint32_t*>(&x);
    return v;
}

// ---- a row's scores ------------------------------------------------------------------

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
        r.st.entropy = r.st.log_s - a.t / a.s * kLn2;
    }
    return r;
}
__device__ __forceinline__ float log_q(const LogprobStats& st, float x, float T) {
    return (x - st.m) / T - st.log_s;
}
__device__ __forceinline__ float row_logprob(const RowScore& r, float x, float T) {
    return r.some ? log_q(r.st, x, T) : -INFINITY;
}

// ---- forward ----------------------------------------------------------------------
//
// Every thread streams vectors of its CTA's slice of the row, four in a row at a
// time: 64 bytes, a group.  A row is one CTA's, or a cluster's where there are few.
//
// The alternatives come from the groups' largest logits.  Order groups by (largest
// logit, lower place): an element of a group outside the first k has k others before
// it, one at least in each of these groups, ties included.  So the k best elements
// are in the k best groups, whatever the logits, and those are read again, mostly from
// L2.  The k best groups are found the same way: among those at least as good as the
// k-th best of the threads' best groups.
//
// A word orders both: the logit in orderable form over the inverted place.  What is
// not above -inf is below kLeast.
//
// 960 rows of 151,936 bf16 logits, 0.29 GB: without alternatives 45.8 us, 6.4 TB/s, 0.94
// of the measured copy rate; with 20 of them 51 us.  What they cost is the chain of small
// steps behind a row's stream (bound, collection, two rankings, a second read from L2,
// about 10 K cycles), which the two other CTAs of an SM hide but for the last rows.
// Three CTAs an SM with three stages: four CTAs with two 56 us.  A CTA a row from as many
// rows as SMs on: rows split over twice as many CTAs cost 300 rows 24 us instead of 19.
// One row: 7.1 us with 20 alternatives, 3.5 without, over a cluster of 16.
// Forms that were slower: every thread ranking its best group among all 256 (73 us for
// the 960 rows), atomics in loops over a thread's groups and elements (65).

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;
constexpr int kStages = 3;
constexpr size_t kRingBytes = (size_t)kThreads * kAhead * kStages * 16;
constexpr int kMaxK = DOMINO_TRAIN_MAX_ALTERNATIVES;
constexpr int kMaxCalls = 32;  // of the stream, in a CTA that looks for alternatives
typedef unsigned long long Word;

constexpr Word kLeast = (Word)0x00800000u << 32;
__device__ __forceinline__ Word word_of(float x, int at) {
    return (Word)(x != x ? 0xFFFFFFFFu : ord_f32(x)) << 32 | (unsigned)~at;
}
__device__ __forceinline__ float word_logit(Word w) {
    const unsigned k = (unsigned)(w >> 32);
    return k == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : unord_f32(k);
}

// A group's largest logit as it is stored, in orderable form: 16 bits of it hold all
// of a bf16.
template <typename T>
struct Stored;
template <>
struct Stored<float> {
    typedef uint32_t Key;
    static __device__ __forceinline__ Key key(unsigned ord) { return ord; }
    // whether group g with this key reaches the bound
    static __device__ __forceinline__ bool reaches(Key k, int g, Word bound) {
        return ((Word)k << 32 | (unsigned)~g) >= bound;
    }
    static __device__ __forceinline__ Word word(Key k, int g) { return (Word)k << 32 | (unsigned)~g; }
};
template <>
struct Stored<__nv_bfloat16> {
    typedef uint16_t Key;
    static __device__ __forceinline__ Key key(unsigned ord) { return (Key)(ord >> 16); }
    // the key's 16 bits and the place's in one word: both sides have 0 or all ones between them
    static __device__ __forceinline__ bool reaches(Key k, int g, Word bound) {
        return ((unsigned)k << 16 | (unsigned)(0xFFFF - g)) >= ((unsigned)(bound >> 48) << 16 | (unsigned)(bound & 0xFFFFu));
    }
    static __device__ __forceinline__ Word word(Key k, int g) {
        // as word_of's of that logit: a negative one's lower bits are ones, and so are a NaN's
        const unsigned low = k & 0x8000u && k != 0xFFFFu ? 0u : 0xFFFFu;
        return (Word)((unsigned)k << 16 | low) << 32 | (unsigned)~g;
    }
};

struct ForwardShared {
    Scores part[kWarps];
    float top[kWarps];
    float m, log_s;                      // of the whole row
    Scores of[kMaxCluster];              // every CTA's, at rank 0
    alignas(16) Word best[kMaxCluster * kMaxK];  // every CTA's alternatives, at rank 0
    Word bound, least, of8[kWarps], nth[kWarps];
    int groups, words;
    int chosen[kMaxK];
};
// the lists of words lie in the ring, which is read by then: the threads' best groups,
// the groups that may be chosen, the elements that may be
static_assert(kMaxK * kAhead <= kThreads, "a thread for every vector of the chosen groups");
constexpr int kListed = kMaxK * kMaxCalls, kElements = kMaxK * kAhead * 8 + 16;
static_assert((kThreads + kListed + kElements) * sizeof(Word) <= kRingBytes, "the lists fit the ring");

// The words that reach a bound to a list whose length is *count, in any order.
// hit: a bit for each of the thread's words, of which get(j) is the j-th.
template <typename Get>
__device__ __forceinline__ void collect(unsigned hit, Word* list, int most, int* count, Get&& get) {
    if (!hit) return;
    int at = atomicAdd(count, __popc(hit));
    for (; hit; hit &= hit - 1, ++at)
        if (at < most) list[at] = get(__ffs(hit) - 1);
}
// f(word, rank) for the n words of a list (all different, or 0) that are in a rank
// below k: four threads a word, which count what is larger.
template <typename F>
__device__ __forceinline__ void rank_words(const Word* list, int n, int k, F&& f) {
    const int part = threadIdx.x & 3;
    for (int i = threadIdx.x >> 2; i - (int)(threadIdx.x >> 2) < n; i += kThreads / 4) {
        const Word w = i < n ? list[i] : 0;
        int r = 0;
#pragma unroll 4
        for (int j = part; j < n; j += 4) r += list[j] > w ? 1 : 0;
        r += __shfl_xor_sync(0xffffffffu, r, 1);
        r += __shfl_xor_sync(0xffffffffu, r, 2);
        if (part == 0 && i < n && w && r < k) f(w, r);
    }
}

// The n-th best of the lanes' words (0: there are fewer), n >= 1, and into *first the
// early-th, early <= n.
__device__ __forceinline__ Word warp_nth(Word w, int n, int early, Word* first) {
    unsigned hi = (unsigned)(w >> 32), lo = (unsigned)w, h = 0, l = 0;
    for (int i = 0; i < n; ++i) {
        h = __reduce_max_sync(0xffffffffu, hi);
        l = __reduce_max_sync(0xffffffffu, hi == h ? lo : 0u);
        if (hi == h && lo == l) hi = lo = 0;
        if (i == early - 1) *first = (Word)h << 32 | l;
    }
    return (Word)h << 32 | l;
}
__device__ __forceinline__ Word warp_nth(Word w, int n) {
    Word unused;
    return warp_nth(w, n, 0, &unused);
}

// The k best elements of the CTA's slice to S.best[0 .. k), in order, 0 where there
// are no more.  mine: the word of the thread's best group, side: its element beside
// the vectors (0: none).
//
// The bound on groups: the h-th best of the warps' n-th best of their threads' best
// groups, n = k / h upwards, which h n groups at least reach; the better one for h = 8, all
// warps, and h = 4, or that for h = 2 or 1 where fewer warps have any (a mask can have it
// so).  Where many more groups reach it, or no warp has k, the k-th best of the threads'
// best groups, which k threads reach, each with as many groups as the stream had calls.
//
// S.nth and the rest of S is set before the call's barrier (start_best); any: some
// thread has a group above -inf.  meanwhile() is called by the last warp, while others
// wait for the chosen groups.
__device__ __forceinline__ void start_best(ForwardShared& S, int k, Word mine) {
    const int t = threadIdx.x;
    Word of8 = 0;
    const Word of4 = warp_nth(mine, (k + 3) / 4, (k + 7) / 8, &of8);
    if (t % 32 == 0) {
        S.of8[t / 32] = of8;
        S.nth[t / 32] = of4;
    }
    if (t == 0) {
        S.groups = S.words = 0;
        S.bound = S.least = kLeast;
    }
    if (t < k) S.best[t] = 0;
}
template <typename T, typename F>
__device__ __forceinline__ void slice_best(ForwardShared& S, Word* lists, const Vectors<T>& x,
                                           const typename Stored<T>::Key* tops, int v0, int k, bool any, Word mine,
                                           Word side, F&& meanwhile) {
    const int t = threadIdx.x, lane = t & 31, groups = (x.last - x.first + kAhead - 1) / kAhead;
    Word *firsts = lists, *listed = firsts + kThreads, *elements = listed + kListed;
    static_assert(kWarps == 8, "the bounds' warps");
    Word bound = S.of8[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) bound = min(bound, S.of8[i]);
    bound = max(bound, warp_nth(lane < kWarps ? S.nth[lane] : 0, 4));
    const auto group = [&](int call) { return Stored<T>::word(tops[t + call * kThreads], t + call * kThreads); };
    const auto collect_groups = [&] {
        unsigned hit = 0;
        if (mine >= bound) {
#pragma unroll 4
            for (int call = 0; t + call * kThreads < groups; ++call)
                hit |= Stored<T>::reaches(tops[t + call * kThreads], t + call * kThreads, bound) ? 1u << call : 0u;
        }
        collect(hit, listed, kListed, &S.groups, group);
    };
    static_assert(kMaxCalls <= 32, "a bit for every call");
    for (int h = 2; any && !bound && h > 0; --h) {  // the same for all threads
        const Word nth = warp_nth(mine, (k + h - 1) / h);
        __syncthreads();  // S.nth is read
        if (lane == 0) S.nth[t / 32] = nth;
        __syncthreads();
        bound = warp_nth(lane < kWarps ? S.nth[lane] : 0, h);
    }
    if (bound) collect_groups();
    __syncthreads();
    int n = S.groups;
    if (any && (n == 0 || n > kListed)) {  // the same for all threads
        firsts[t] = mine;
        __syncthreads();
        rank_words(firsts, kThreads, k, [&](Word w, int r) {
            if (r == k - 1) S.bound = w;
        });
        __syncthreads();
        bound = S.bound;
        if (t == 0) S.groups = 0;
        __syncthreads();
        collect_groups();
        __syncthreads();
        n = S.groups;
    }
    rank_words(listed, n, k, [&](Word w, int r) {
        S.chosen[r] = (int)~(unsigned)w;
        if (r == k - 1) S.least = w >> 32 << 32;
    });
    __syncthreads();
    const Word least = S.least;
    if (t < min(n, k) * kAhead) {
        const int at = x.first + S.chosen[t / kAhead] * kAhead + t % kAhead;
        if (at < x.last) {
            Vec16<T> v;
            v.q = __ldcg(x.vec() + at);
            const int id = v0 + at * Vectors<T>::kPer - x.phase;
            Word w[Vectors<T>::kPer];
            unsigned hit = 0;
#pragma unroll
            for (int j = 0; j < Vectors<T>::kPer; ++j) {
                const float2 h = halves(v.pair(j / 2));
                w[j] = word_of(j % 2 ? h.y : h.x, id + j);
                hit |= w[j] >= least ? 1u << j : 0u;
            }
            int to = hit ? atomicAdd(&S.words, __popc(hit)) : 0;
#pragma unroll
            for (int j = 0; j < Vectors<T>::kPer; ++j)
                if (hit >> j & 1u) elements[to++] = w[j];
        }
    }
    if (side >= least) elements[atomicAdd(&S.words, 1)] = side;
    if (t / 32 == kWarps - 1) meanwhile();
    __syncthreads();
    rank_words(elements, S.words, k, [&](Word w, int r) { S.best[r] = w; });
    __syncthreads();
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kThreads, 3) k_scores(LogprobArgs p, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ForwardShared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int n = blockIdx.x / size, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const float c = kLog2e / p.temperature;
    const int v0 = min(p.V, rank * chunk);
    const T* row = static_cast<const T*>(p.x) + (size_t)n * p.ld;
    const Vectors<T> x(row + v0, min(p.V, v0 + chunk) - v0);
    uint4* ring = reinterpret_cast<uint4*>(smem);
    typename Stored<T>::Key* tops = reinterpret_cast<typename Stored<T>::Key*>(smem + kRingBytes);
    pdl_wait();
    // the first vectors are on their way while the token is read
    Streamer<kThreads, kAhead, kStages, true, T> vectors(x, ring);
    const int tok = p.tokens[n];
    const bool in = (unsigned)tok < (unsigned)p.V;
    if (!in) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (rank == 0) {
            if (t == 0) {
                if (tok != -1) atomicOr(p.err, kErrBadToken);
                p.logprob[n] = 0.f;
                if (p.entropy) p.entropy[n] = 0.f;
                if (p.stats) reinterpret_cast<LogprobStats*>(p.stats)[n] = {0.f, 0.f, 0.f, 0.f};
            }
            for (int k = t; k < p.k; k += kThreads) {
                p.alt_ids[(size_t)n * p.k + k] = -1;
                p.alt_logprobs[(size_t)n * p.k + k] = -INFINITY;
            }
        }
        return;
    }
    if (size > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const float said = to_f32(row[tok]);
    const int side_at = t < 2 * Vectors<T>::kPer ? x.beside(t) : x.n;
    const bool has_side = side_at < x.n;
    const T side = has_side ? x.src[side_at] : from_f32<T>(-INFINITY);

    const F2 cc = f2(c, c);
    Running a;
    unsigned best = 0;  // of the thread's groups, in orderable form; the first of equals
    int best_g = 0, g = t;
    vectors.run([&](int, Vec16<T>* v, auto) {
        const float high = top4(v);
        a.template add<kAhead>(v, high, c, cc);
        if (kTop) {
            const unsigned o = high != high ? 0xFFFFFFFFu : ord_f32(high);
            tops[g] = Stored<T>::key(o);
            if (o > best) {
                best = o;
                best_g = g;
            }
            g += kThreads;
        }
    });
    if (has_side) {
        const Vec16<T> one = alone(side);
        a.template add<1>(&one, to_f32(side), c, cc);
    }
    Scores u = warp_join(a.scores(), c);
    const float top = warp_max(a.top);
    Word mine = 0;
    if (kTop) {
        mine = (Word)best << 32 | (unsigned)~best_g;
        if (mine < kLeast) mine = 0;
        start_best(S, p.k, mine);
    }
    if (lane == 0) {
        S.part[warp] = u;
        S.top[warp] = top;
    }
    const bool any = __syncthreads_or(mine != 0);
    const float high = warp_max(S.top[lane % kWarps]);
    u = warp_join(lane < kWarps ? S.part[lane] : no_scores(), c);
    if (!plain_range(u.m)) {
        if (high == -INFINITY && u.s == 0.f) {
            u = no_scores();
        } else {  // the same for all threads
            u = no_scores();
            for (int i = t; i < x.n; i += kThreads) add(u, to_f32(x.src[i]), c);
            u = warp_join(u, c);
            __syncthreads();
            if (lane == 0) S.part[warp] = u;
            __syncthreads();
            u = warp_join(lane < kWarps ? S.part[lane] : no_scores(), c);
        }
    }
    // the row's values, by one warp
    const auto tell = [&] {
        const RowScore r = finish(u);
        if (lane == 0) {
            p.logprob[n] = row_logprob(r, said, p.temperature);
            if (p.entropy) p.entropy[n] = r.st.entropy;
            if (p.stats) reinterpret_cast<LogprobStats*>(p.stats)[n] = r.st;
            S.m = r.st.m;
            S.log_s = r.st.log_s;
        }
    };
    if (kTop) {
        slice_best<T>(S, reinterpret_cast<Word*>(ring), x, tops, v0, p.k, any, mine,
                      has_side ? word_of(to_f32(side), v0 + side_at) : 0, [&] {
                          if (size == 1) tell();
                      });
    }
    if (size > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (t == 0) *cluster.map_shared_rank(&S.of[rank], 0) = u;
        if (kTop && rank > 0 && t < p.k) *cluster.map_shared_rank(&S.best[rank * p.k + t], 0) = S.best[t];
        cluster_barrier();
        if (rank != 0) return;
        u = warp_join(lane < size ? S.of[lane] : no_scores(), c);
    }
    if ((!kTop || size > 1) && warp == 0) tell();
    if (kTop) {
        int* ids = p.alt_ids + (size_t)n * p.k;
        float* scores = p.alt_logprobs + (size_t)n * p.k;
        int some = p.k;
        const auto put = [&](Word w, int at) {
            ids[at] = (int)~(unsigned)w;
            scores[at] = (word_logit(w) - S.m) / p.temperature - S.log_s;
        };
        if (size == 1) {
            const Word w = t < p.k ? S.best[t] : 0;
            if (w) put(w, t);
            some = __syncthreads_count(w != 0);
        } else {
            // nothing is among the best that is worse than some CTA's k-th, or than the n-th of
            // h of them, n = k / h upwards
            const int h = size < 4 ? size : 4;
            Word *elements = reinterpret_cast<Word*>(ring);
            Word least = warp_nth(lane < size ? S.best[lane * p.k + (p.k + h - 1) / h - 1] : 0, h);
            least = max(max(least, (Word)1), warp_nth(lane < size ? S.best[lane * p.k + p.k - 1] : 0, 1));
            if (t == 0) S.words = 0;
            __syncthreads();
            for (int i = t; i < size * p.k; i += kThreads)
                if (S.best[i] >= least) elements[atomicAdd(&S.words, 1)] = S.best[i];
            __syncthreads();
            some = S.words;
            rank_words(elements, some, p.k, put);
        }
        // places behind the last alternative
        if (t >= some && t < p.k) {
            ids[t] = -1;
            scores[t] = -INFINITY;
        }
    }
}

// ---- gradient -----------------------------------------------------------------------
//
// By itself a stream as the forward's, each vector written where it was read: bound by
// HBM, 960 rows of 151,936 bf16 logits, 0.58 GB, in 91 us, 6.4 TB/s.

// What turns a logit into its gradient: e (a + b d) with e = 2^d, d = (x - m) c.
struct Slope {
    float m, a, b, hot;  // hot: added at the token
};
__device__ __forceinline__ Slope slope(const LogprobStats& st, float g, float h, float T) {
    const float w = -st.inv_s / T;
    return {st.m, w * (g + h * (st.entropy - st.log_s)), w * h * kLn2, g / T};
}
// d is held above -200, where e is 0: a masked logit's is not infinite
__device__ __forceinline__ float gradient(const Slope& k, float x, float c) {
    const float d = max_nan((x - k.m) * c, -200.f);
    return ex2(d) * fmaf(k.b, d, k.a);
}
template <typename T>
__device__ __forceinline__ Vec16<T> gradient(const Slope& k, const Vec16<T>& v, F2 cc) {
    Vec16<T> r;
    const F2 minus = f2(-k.m, -k.m), a = f2(k.a, k.a), b = f2(k.b, k.b);
#pragma unroll
    for (int i = 0; i < Vec16<T>::kElems / 2; ++i) {
        const float2 h = halves(mul2(add2(v.pair(i), minus), cc));
        const F2 d = f2(max_nan(h.x, -200.f), max_nan(h.y, -200.f));
        r.set(i, mul2(ex2x2(d), fma2(b, d, a)));
    }
    return r;
}
// zeros to the elements [0, n) of a row's slice
template <typename T>
__device__ __forceinline__ void clear(T* dx, int n, int threads) {
    const int t = threadIdx.x, head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(dx) & 15)) & 15) / (int)sizeof(T));
    const int whole = (n - head) / Vec16<T>::kElems;
    uint4* out = reinterpret_cast<uint4*>(dx + head);
    for (int i = t; i < whole; i += threads) out[i] = make_uint4(0, 0, 0, 0);
    const int body = whole * Vec16<T>::kElems;
    for (int i = t; i < n - body; i += threads) dx[i < head ? i : i + body] = from_f32<T>(0.f);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_scores_backward(LogprobArgs p, int chunk, int size) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kPer = Vec16<T>::kElems;
    const int n = blockIdx.x / size, v0 = min(p.V, (int)(blockIdx.x % size) * chunk), t = threadIdx.x;
    const float c = kLog2e / p.temperature;
    const Vectors<T> x(static_cast<const T*>(p.x) + (size_t)n * p.ld + v0, min(p.V, v0 + chunk) - v0);
    T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d + v0;
    pdl_wait();
    const LogprobStats st = reinterpret_cast<const LogprobStats*>(p.stats)[n];
    const float g = p.dlogprob ? p.dlogprob[n] : 0.f, h = p.dentropy ? p.dentropy[n] : 0.f;
    const int tok = p.tokens[n] - v0;
    if (st.inv_s == 0.f || (g == 0.f && h == 0.f)) {
        clear(dx, x.n, kThreads);
        return;
    }
    const Slope k = slope(st, g, h, p.temperature);
    if (((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x.src)) & 15) == 0) {
        uint4* out = reinterpret_cast<uint4*>(dx - x.phase);
        const F2 cc = f2(c, c);
        stream<kThreads, kAhead, kStages>(x, reinterpret_cast<uint4*>(smem), [&](int i0, Vec16<T>* v, auto all) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (all() || i0 + j * kThreads < x.last) out[i0 + j * kThreads] = gradient(k, v[j], cc).q;
        });
        const int side = t < 2 * kPer ? x.beside(t) : x.n;
        if (side < x.n) dx[side] = from_f32<T>(gradient(k, to_f32(x.src[side]), c));
    } else {
        for (int i = t; i < x.n; i += kThreads) dx[i] = from_f32<T>(gradient(k, to_f32(x.src[i]), c));
    }
    if ((unsigned)tok < (unsigned)x.n) {  // the same for all threads
        __syncthreads();
        if (t == 0) dx[tok] = from_f32<T>(gradient(k, to_f32(x.src[tok]), c) + k.hot);
    }
}

// ---- scores and gradient at once -------------------------------------------------------
//
// A cluster of CTAs holds one row in shared memory, a slice each: a bulk copy brings
// it in, the sums are a pass over shared memory, the CTAs send theirs into each
// other's shared memory, and a second pass writes the gradient.  So the logits are
// read once and the gradient is written once.  One wave of clusters takes rows in
// turn; a row's token and weights are read a row ahead.
//
// Bound by HBM: 3840 rows of 151,936 bf16 logits, 2.33 GB, in 368 us, 6.3 TB/s, 0.93 of
// the measured copy rate.  1021 fp32 rows of 4097 that L2 does not hold take 9.4 us: one
// wave of CTAs that all load, sum and write at the same time.  With every thread forming
// the row's statistics instead of one warp the 3840 rows took 424 us.

constexpr int kSliceBytes = 40 * 1024;
constexpr int kStepThreads = 128;
constexpr int kStepWarps = kStepThreads / 32;
struct StepShared {
    Scores part[2][kMaxCluster * kStepWarps];  // every warp of the row, by the row's parity
    LogprobStats row;
    unsigned long long bar;          // the row's copy has come
    unsigned long long exchange[2];  // the row's sums have come, by the row's parity
    int abort;
};

// One thread's sums into a CTA's shared memory, counted on that CTA's barrier.
__device__ __forceinline__ void send(const Scores& u, Scores* to, unsigned long long* bar, int rank) {
    static_assert(sizeof(Scores) == 16, "one 16-byte store");
    uint32_t dst, mbar;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(tc::smem_u32(to)), "r"(rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(mbar) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(dst),
                 "f"(u.m), "f"(u.s), "f"(u.t), "f"(u.unused), "r"(mbar)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ Scores warp_scores(const Slice<T>& x, float c) {
    constexpr int U = 4;
    const F2 cc = f2(c, c);
    Running a;
    int i = threadIdx.x;
#pragma unroll 1
    for (; i + (U - 1) * kStepThreads < x.nvec; i += U * kStepThreads) {
        Vec16<T> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) v[j].q = x.vec[i + j * kStepThreads];
        a.template add<U>(v, top_of<U>(v), c, cc);
    }
#pragma unroll 1
    for (; i < x.nvec; i += kStepThreads) {
        Vec16<T> v;
        v.q = x.vec[i];
        a.template add<1>(&v, v.top(), c, cc);
    }
    Scores u = warp_join(a.scores(), c);
    if (!plain_range(u.m)) {  // the warp's own elements once more
        const bool none = warp_max(a.top) == -INFINITY && u.s == 0.f;
        u = no_scores();
        if (!none) {
            const T* e = reinterpret_cast<const T*>(x.vec);
            constexpr int kPer = Vec16<T>::kElems;
            for (int k = threadIdx.x; k < x.nvec; k += kStepThreads)
                for (int j = 0; j < kPer; ++j) add(u, to_f32(e[k * kPer + j]), c);
            u = warp_join(u, c);
        }
    }
    return u;
}

template <typename T>
__global__ void __launch_bounds__(kStepThreads, 8) k_scores_step(LogprobArgs p, int chunk) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ StepShared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const unsigned rows = p.n, stride = gridDim.x / size;  // a row's number and a stride fit 32 bits together
    const float c = kLog2e / p.temperature;
    const uint32_t bar = tc::smem_u32(&S.bar);
    const auto slice = [&](unsigned n) {
        return Slice<T>(static_cast<const T*>(p.x) + (size_t)n * p.ld, p.V, chunk, rank, smem);
    };
    const auto request = [&](const Slice<T>& x) {  // one thread, after a barrier behind the buffer's last use
        tc::fence_proxy_async();
        const uint32_t bytes = (uint32_t)x.body * sizeof(T);
        tc::mbar_arrive_expect_tx(bar, bytes);
        if (bytes) tc::bulk_load(tc::smem_u32(x.data + x.head), x.src + x.head, bytes, bar, tc::policy_evict_normal());
    };
    // what is read ahead of a row
    struct Ahead {
        float g, h;
        int tok;
        bool part;  // the row takes part
    };
    const auto ahead = [&](unsigned n) {
        Ahead a = {0.f, 0.f, -1, false};
        if (n < rows) {
            if (p.dlogprob) a.g = p.dlogprob[n];
            if (p.dentropy) a.h = p.dentropy[n];
            a.tok = p.tokens[n];
            const bool in = (unsigned)a.tok < (unsigned)p.V;
            if (!in && a.tok != -1 && rank == 0 && t == 0) atomicOr(p.err, kErrBadToken);
            a.part = in && (a.g != 0.f || a.h != 0.f);
        }
        return a;
    };
    unsigned n = blockIdx.x / size;
    pdl_wait();
    Ahead now = ahead(n);
    if (t == 0) {
        tc::mbar_init(bar, 1);
        for (int i = 0; i < 2; ++i) tc::mbar_init(tc::smem_u32(&S.exchange[i]), 1);
        S.abort = 0;
        tc::fence_barrier_init();
        if (now.part) request(slice(n));
    }
    if (now.part) slice(n).load_edges();
    cluster_barrier();  // every CTA of the cluster is running
    uint32_t turn = 0;  // rows so far that took part
    for (; n < rows; n += stride) {
        const Ahead next = ahead(n + stride);
        const Slice<T> x = slice(n);
        T* dx = static_cast<T*>(p.dx) + (size_t)n * p.ld_d + x.v0;
        bool hot = false;
        Slope k = {};
        if (now.part) {
            const uint32_t phase = turn & 1;  // of the copy, and which exchange it is
            const float said = rank == 0 && t == 0 ? to_f32(static_cast<const T*>(p.x)[(size_t)n * p.ld + now.tok]) : 0.f;
            if (t == 0) tc::mbar_wait(bar, phase, &S.abort, p.err);
            __syncthreads();
            Scores u = warp_scores(x, c);
            // every warp's sums to every CTA of the row
            // (to the other place than the last row's: who sends for this row has seen
            // every CTA's sums of the last one, so all have read those of the one before)
            if (t == 0) tc::mbar_arrive_expect_tx(tc::smem_u32(&S.exchange[phase]), size * kStepWarps * sizeof(Scores));
            if (lane < size) send(u, &S.part[phase][rank * kStepWarps + warp], &S.exchange[phase], lane);
            if (warp == 0) {
                tc::mbar_wait(tc::smem_u32(&S.exchange[phase]), turn >> 1 & 1, &S.abort, p.err);
                const Scores* part = S.part[phase];
                u = part[min(lane, size * kStepWarps - 1)];
                if (lane >= size * kStepWarps) u = no_scores();
                for (int i = lane + 32; i < size * kStepWarps; i += 32) u = join(u, part[i], c);
                u = warp_join(u, c);
                const RowScore r = finish(u);
                if (lane == 0) {
                    S.row = r.st;
                    if (rank == 0) {
                        p.logprob[n] = row_logprob(r, said, p.temperature);
                        p.entropy[n] = r.st.entropy;
                    }
                }
            }
            __syncthreads();
            ++turn;
            const LogprobStats st = S.row;
            if (st.inv_s != 0.f) {
                k = slope(st, now.g, now.h, p.temperature);
                hot = (unsigned)(now.tok - x.v0) < (unsigned)x.n;
                // the gradient straight to memory: the buffer is free as soon as it is read
                const bool together = ((reinterpret_cast<uintptr_t>(dx) ^ reinterpret_cast<uintptr_t>(x.src)) & 15) == 0;
                if (together) {
                    const F2 cc = f2(c, c);
                    uint4* out = reinterpret_cast<uint4*>(dx + x.head);
                    const uint4* in = reinterpret_cast<const uint4*>(x.data + x.head);
#pragma unroll 2
                    for (int i = t; i < x.body / Vec16<T>::kElems; i += kStepThreads) {
                        Vec16<T> v;
                        v.q = in[i];
                        out[i] = gradient(k, v, cc).q;
                    }
                }
                // the elements beside whole vectors, or all where the two rows start differently modulo 16 bytes
                const int beside = x.n - (together ? x.body : 0);
                for (int i = t; i < beside; i += kStepThreads) {
                    const int e = together && i >= x.head ? i + x.body : i;
                    dx[e] = from_f32<T>(gradient(k, to_f32(x.data[e]), c));
                }
            } else {
                clear(dx, x.n, kStepThreads);
            }
        } else {
            if (rank == 0 && t == 0) p.logprob[n] = p.entropy[n] = 0.f;
            clear(dx, x.n, kStepThreads);
        }
        __syncthreads();  // the buffer is read, and the gradient written
        if (S.abort) break;  // a copy or a peer's sums never came: no further rows, so that no further copy is asked for
        if (hot && t == 0) {
            const int e = now.tok - x.v0;
            dx[e] = from_f32<T>(gradient(k, to_f32(x.src[e]), c) + k.hot);
        }
        if (next.part) {
            const Slice<T> y = slice(n + stride);
            if (t == 0) request(y);
            y.load_edges();
        }
        now = next;
    }
    // after a break: the row's own copy, the last one asked for
    if (t == 0 && S.abort) last_chance(bar, (turn & 1) ^ 1);
    cluster_barrier();  // nobody leaves before all have their sums
}

// A launch in clusters of `size` CTAs that may be set up while the stream's last
// kernel ends (every kernel here waits for that one before it reads memory): in
// calls after one another a kernel of a few us comes 1 to 2 us earlier.
struct Launch {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg;
    Launch(unsigned blocks, int threads, int size, size_t smem, cudaStream_t st)
        : cfg(cluster_config(blocks, threads, size, smem, st, attr)) {
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    }
};

// most CTAs a row of `n` rows takes until there are `per_sm` of them on every SM
int few_rows(const domino_train_ctx* ctx, int n, int V, int per_sm, int least, int most) {
    int size = 1;
    while (size < most && (long long)n * size < (long long)per_sm * ctx->num_sms && slice_of(V, 2 * size) >= least)
        size *= 2;
    return size;
}

template <typename T>
cudaError_t launch_forward(domino_train_ctx* ctx, const LogprobArgs& a, cudaStream_t st) {
    constexpr int kCall = kThreads * kAhead * Vec16<T>::kElems;  // elements
    int size = few_rows(ctx, a.n, a.V, 1, 4096, kMaxCluster);
    while (size < kMaxCluster && slice_of(a.V, size) > kMaxCalls * kCall) size *= 2;
    const int chunk = slice_of(a.V, size), calls = (chunk + kCall - 1) / kCall;
    const size_t smem = kRingBytes + (a.k > 0 ? (size_t)calls * kThreads * sizeof(typename Stored<T>::Key) : 0);
    Launch l((unsigned)a.n * size, kThreads, size, smem, st);
    ctx->last_launches = 1;
    return a.k > 0 ? cudaLaunchKernelEx(&l.cfg, k_scores<T, true>, a, chunk)
                   : cudaLaunchKernelEx(&l.cfg, k_scores<T, false>, a, chunk);
}

template <typename T>
cudaError_t launch_backward(domino_train_ctx* ctx, const LogprobArgs& a, cudaStream_t st) {
    int size = few_rows(ctx, a.n, a.V, 4, 2048, 64);
    while (slice_of(a.V, size) * (int)sizeof(T) > 160 * 1024) size *= 2;
    ctx->last_launches = 1;
    return launch_pdl(k_scores_backward<T>, dim3((unsigned)a.n * size), dim3(kThreads), kRingBytes, st, a,
                      slice_of(a.V, size), size);
}

template <typename T>
cudaError_t launch_step(domino_train_ctx* ctx, const LogprobArgs& a, cudaStream_t st) {
    int size = 1;
    while (size < kMaxCluster && slice_of(a.V, size) * (int)sizeof(T) > kSliceBytes) size *= 2;
    while (size < kMaxCluster && (long long)a.n * size < 2 * ctx->num_sms && slice_of(a.V, 2 * size) >= 4096) size *= 2;
    const int chunk = slice_of(a.V, size);
    const size_t smem = (size_t)chunk * sizeof(T) + 32;
    Launch l(size, kStepThreads, size, smem, st);
    // one wave of clusters, each taking rows in turn; how many the GPU holds at once
    // is asked once per context and cluster size.  (Clusters of one CTA are launched as
    // such too: the kernel's barriers and stores address a cluster.)
    int& most = ctx->score_clusters[size];
    if (most == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&most, k_scores_step<T>, &l.cfg);
        if (e != cudaSuccess) return e;
        if (most < 1) most = 1;
    }
    l.cfg.gridDim = dim3((unsigned)(a.n < most ? a.n : most) * size);
    ctx->last_launches = 1;
    return cudaLaunchKernelEx(&l.cfg, k_scores_step<T>, a, chunk);
}

}  // namespace

cudaError_t prepare_logprob_kernels() {
    cudaError_t e = allow_all(k_scores_step<float>);
    if (e == cudaSuccess) e = allow_all(k_scores_step<__nv_bfloat16>);
    if (e == cudaSuccess) e = allow_all(k_scores<float, true>);
    if (e == cudaSuccess) e = allow_all(k_scores<__nv_bfloat16, true>);
    if (e == cudaSuccess) e = allow_all(k_scores<float, false>);
    if (e == cudaSuccess) e = allow_all(k_scores<__nv_bfloat16, false>);
    return e;
}

cudaError_t launch_logprobs_forward(domino_train_ctx* c, int dtype, const LogprobArgs& a, cudaStream_t st) {
    return dtype == DOMINO_DTYPE_BF16 ? launch_forward<__nv_bfloat16>(c, a, st) : launch_forward<float>(c, a, st);
}
cudaError_t launch_logprobs_backward(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_backward<__nv_bfloat16>(c, a, st) : launch_backward<float>(c, a, st);
}
cudaError_t launch_logprobs_step(domino_train_ctx* c, const LogprobArgs& a, cudaStream_t st) {
    return c->cfg.dtype == DOMINO_DTYPE_BF16 ? launch_step<__nv_bfloat16>(c, a, st) : launch_step<float>(c, a, st);
}

}  // namespace train
}  // namespace domino
