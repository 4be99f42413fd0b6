// Record of a teacher's logits: the K largest of each row, ids ascending, and
// the log-sum-exp of all the others.
//
// Order: (logit descending, id ascending), with NaN above everything and the
// two zeros equal; a 64-bit word, orderable logit over inverted id, has that
// order.
//
// The row is read once.  Four vectors in a row, 64 bytes, are a group; the CTA
// keeps every group's largest logit and the sum of its exponentials in shared
// memory, so the stream itself has no block-wide barrier and no branch on the
// data.  A bound that K elements reach and few others comes from two maxima per
// thread (small K) or the groups'.  The groups below it are in the
// rest with their sums, the others (about K of them) are read again, mostly from
// L2: what lies above the bound becomes a word in a buffer, of which an exact
// radix select leaves K; what equals it only leaves a bit in the order of the
// ids, from which the lowest ids are taken where the buffer lacks words, so that
// rows full of equal logits (masked ones) cost no more than others.  The rest is
// never formed as a difference of sums: a peaked teacher leaves less in it than
// the rounding of the whole.  Places in lists come from scans, not from atomics,
// so that equal calls sum in equal order.
//
// fp32 rows whose groups do not fit one CTA are spread over a cluster: every CTA finds
// its slice's best K and rank 0 takes the others' through distributed shared
// memory.  Few rows are not: the merge costs more than the stream gains (15 rows,
// a CTA each or eight: K = 64 14.4 and 17.5 us, K = 512 25 and 54 us, K = 2048 45
// and 150 us).
//
// 960 rows of 151,936 bf16 logits, K = 256: 84 us, 3.5 TB/s, 0.52 of the measured
// copy rate.  Of a row's 66 K cycles (three CTAs an SM) the stream takes 35 K, the
// second read 12 K, the select 6 K, the bound, the list of groups and the order of
// the ids 3 K each: the chains of small steps behind the stream and the
// instructions (half of the issue slots) bound it, not HBM.  333 rows of 79,999
// fp32 logits, K = 2048: 90 us (41 % of the row is read again); 15 rows, K = 64:
// 14.4 us.  Groups of four vectors 4 or 8 KB apart: 93 us for the 960 rows (half of
// every sector read again was not wanted); several groups per thread between two
// counts of the words: 87 to 89 us.  A running bound raised by selects during the
// stream took 369, 281 and 76 us.
#include <cooperative_groups.h>

#include <type_traits>

#include "train_internal.h"
#include "train_stream.cuh"

namespace cg = cooperative_groups;

namespace domino {
namespace train {

namespace {

constexpr int kAhead = 4;
constexpr int kStages = 2;
constexpr int kBins = 2048;
constexpr int kFew = 64;     // a record whose ids are ordered by counting
constexpr int kDue = 512;    // words beyond K that make a select due
constexpr int kStep = 1024;  // words that are sure to fit then, a multiple of the threads
constexpr size_t kMaxSmem = 224 * 1024;  // of a CTA, beside its static variables
// A CTA has 256 threads where three such fit an SM: every step that the whole CTA
// takes costs instructions by the warp (960 rows, K = 256: 86 us with 256, 95 with
// 512).  It has 512 where fewer fit (333 rows, K = 2048: 105 and 92 us) and where
// rows are alone on their SMs, if the record is not small (15 rows, K = 2048: 56 and
// 48 us, K = 256: 23 and 21; K = 64: 14.8 and 16.5).
constexpr size_t kThirdSmem = 74 * 1024;  // of one of three CTAs on an SM

__device__ __forceinline__ unsigned top_key(float x) { return x != x ? 0xFFFFFFFFu : ord_f32(x); }
__device__ __forceinline__ float key_logit(unsigned k) { return k == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : unord_f32(k); }
__device__ __forceinline__ unsigned word_id(unsigned long long w) { return ~(unsigned)w; }
__device__ __forceinline__ unsigned long long word_of(unsigned key, unsigned id) {
    return (unsigned long long)key << 32 | (unsigned)~id;
}

template <typename T>
struct Group {
    static constexpr int kElems = kAhead * Vec16<T>::kElems;
};
// a group's maximum as it is stored: the logits' own type
template <typename T>
using Raw = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
template <typename T>
__device__ __forceinline__ Raw<T> to_raw(float m) {
    return (Raw<T>)(sizeof(T) == 2 ? __float_as_uint(m) >> 16 : __float_as_uint(m));
}
__device__ __forceinline__ float from_raw(uint16_t r) { return __uint_as_float((unsigned)r << 16); }
__device__ __forceinline__ float from_raw(uint32_t r) { return __uint_as_float(r); }
__device__ __forceinline__ float from_raw(float r) { return r; }
__device__ __forceinline__ float from_raw(__nv_bfloat16 r) { return to_f32(r); }

constexpr int kTies = 64;  // equal logits that are ordered by counting
constexpr int kTile = 8;  // words per thread that a select moves at once

struct TopShared {
    unsigned warp[16];  // 512 threads at most
    unsigned digit, need, in_bin, ties;
    unsigned long long last;
    unsigned bound;
    MaxSum part[16];
    MaxSum rest[kMaxCluster];  // of every CTA of the row, at rank 0
};

// A bit per element of v that lies above b (NaN does) and per element that
// equals it; v without either (-inf in their places).  b is a logit of the type.
__device__ __forceinline__ Vec16<float> above(const Vec16<float>& v, float b, unsigned* in, unsigned* eq) {
    Vec16<float> r;
    const auto one = [&](unsigned w, int e) {
        const float y = __uint_as_float(w);
        const bool gt = !(y <= b), same = y == b;
        *in |= gt ? 1u << e : 0u;
        *eq |= same ? 1u << e : 0u;
        return gt || same ? 0xFF800000u : w;
    };
    r.q = make_uint4(one(v.q.x, 0), one(v.q.y, 1), one(v.q.z, 2), one(v.q.w, 3));
    return r;
}
__device__ __forceinline__ Vec16<__nv_bfloat16> above(const Vec16<__nv_bfloat16>& v, float b, unsigned* in,
                                                      unsigned* eq) {
    Vec16<__nv_bfloat16> r;
    const __nv_bfloat162 bb = __float2bfloat162_rn(b);
    unsigned gt_bits = 0, eq_bits = 0;  // elements 0, 2, 4, 6 in bits 0..3, elements 1, 3, 5, 7 in bits 16..19
    const auto two = [&](unsigned w, int k) {
        const __nv_bfloat162 y = *reinterpret_cast<const __nv_bfloat162*>(&w);
        const unsigned le = __hle2_mask(y, bb), same = __heq2_mask(y, bb);
        gt_bits |= ~le & (0x00010001u << k);
        eq_bits |= same & (0x00010001u << k);
        return (w & le & ~same) | (0xFF80FF80u & (~le | same));
    };
    r.q = make_uint4(two(v.q.x, 0), two(v.q.y, 1), two(v.q.z, 2), two(v.q.w, 3));
    // bit k of either half to bits 2k and 2k + 1
    const auto spread = [](unsigned m) {
        const unsigned lo = m & 15u, hi = m >> 16 & 15u;
        const auto wide = [](unsigned x) { return (x & 1u) | (x & 2u) << 1 | (x & 4u) << 2 | (x & 8u) << 3; };
        return wide(lo) | wide(hi) << 1;
    };
    if (gt_bits | eq_bits) {
        *in = spread(gt_bits);
        *eq = spread(eq_bits);
    }
    return r;
}

// Exclusive scan of one value per thread; *total gets the sum.
template <int kThreads>
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
    for (int w = 0; w < kThreads / 32; ++w) {
        const unsigned v = warp_tot[w];
        if (w < warp) before += v;
        all += v;
    }
    __syncthreads();
    *total = all;
    return before + incl - x;
}

template <int kThreads>
__device__ __forceinline__ unsigned block_max(unsigned x, unsigned* warp_tot) {
    x = __reduce_max_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) warp_tot[threadIdx.x >> 5] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x = max(x, warp_tot[w]);
    __syncthreads();
    return x;
}

// Shared memory of a slice of `elems` elements: the ring of the stream, in whose
// place come the histogram, the buffer of K + kDue + kStep words and the list of
// groups; behind it the groups' sums and maxima, in whose place comes a bit per id.
template <typename T, int kThreads>
__host__ __device__ constexpr int groups_of(int elems) {
    return (elems / Group<T>::kElems + kThreads) / kThreads * kThreads;  // one vector more than elems if unaligned
}
__host__ __device__ constexpr size_t words_bytes(int K) { return (size_t)(K + kDue + kStep) * 8; }
template <int kThreads>
__host__ __device__ constexpr size_t front_bytes(int groups, int K) {
    constexpr size_t kRingBytes = (size_t)kThreads * kAhead * kStages * 16;
    const size_t later = (size_t)kBins * 4 + words_bytes(K) + (size_t)groups * 2;
    return ((kRingBytes > later ? kRingBytes : later) + 15) / 16 * 16;
}
template <typename T>
__host__ __device__ constexpr size_t group_bytes(int groups) { return (size_t)groups * (4 + sizeof(Raw<T>)); }

// The digit of the `need`-th largest among the words word(0..n-1) that match
// prefix under mask, its count and what remains to be found in it, to S.  All
// threads; hist is all zeros before and after.
template <int kThreads, typename F>
__device__ __forceinline__ void digit_pass(TopShared& S, unsigned* hist, F&& word, int n, unsigned long long prefix,
                                           unsigned long long mask, int shift, int bins, unsigned need) {
    const int t = threadIdx.x;
#pragma unroll 2
    for (int i = t; i < n; i += kThreads) {
        const unsigned long long w = word(i);
        if ((w & mask) == prefix) atomicAdd(&hist[(unsigned)(w >> shift) & (unsigned)(bins - 1)], 1u);
    }
    __syncthreads();
    // thread t holds `per` bins, from the top down
    const int per = bins > kThreads ? bins / kThreads : 1, first = bins - 1 - t * per;
    unsigned mine = 0, all;
    if (first >= 0)
        for (int j = 0; j < per; ++j) mine += hist[first - j];
    unsigned above = block_scan<kThreads>(mine, S.warp, &all);
    if (above < need && above + mine >= need) {
        int b = first;
        while (above + hist[b] < need) above += hist[b--];
        S.digit = (unsigned)b;
        S.need = need - above;
        S.in_bin = hist[b];
    }
    if (first >= 0)
        for (int j = 0; j < per; ++j) hist[first - j] = 0;
    __syncthreads();
}

// Where to look for the K-th of keys between `low` and the largest: the bits
// from `bit` up are common to all.
__device__ __forceinline__ void search_range(unsigned low, unsigned largest, int floor, int* bit,
                                             unsigned long long* prefix, unsigned long long* mask) {
    *bit = max(floor, 32 - __clz((int)(largest ^ low)));
    *mask = *bit == 32 ? 0ull : ~0ull << (32 + *bit);
    *prefix = ((unsigned long long)largest << 32) & *mask;
}

// A bound for the K largest of n logits: the K-th largest's key, or a little
// less.  All keys lie in [lowest, largest].
template <int kThreads, bool kShort, typename R>
__device__ __noinline__ unsigned bound_by(TopShared& S, unsigned* hist, const R* raw, int n, int K, unsigned lowest,
                                          unsigned largest) {
    constexpr int kFloor = kShort ? 16 : 0;
    int bit;
    unsigned long long prefix, mask;
    search_range(lowest, largest, kFloor, &bit, &prefix, &mask);
    unsigned need = (unsigned)K;
    while (bit > kFloor) {
        const int bits = min(11, bit - kFloor);
        bit -= bits;
        digit_pass<kThreads>(S, hist, [&](int i) { return (unsigned long long)top_key(from_raw(raw[i])) << 32; }, n, prefix, mask,
                   32 + bit, 1 << bits, need);
        prefix |= (unsigned long long)S.digit << (32 + bit);
        mask |= (unsigned long long)((1u << bits) - 1) << (32 + bit);
        need = S.need;
        if (S.in_bin <= need + (unsigned)(K / 8)) break;  // few more than needed lie in the bin
    }
    return (unsigned)(prefix >> 32);
}

// What a select leaves beside the words: the bound (the K-th best key) and the
// thread's share of the rest.
struct Selected {
    unsigned bound;
    MaxSum rest;
};

// Leaves the best K of `count` words at the front of the buffer; every word's
// key lies in [low, largest].  kShort: logits with 16 significant bits.  All
// threads, after a barrier, count > K.
template <int kThreads, bool kShort, bool kWantBound>
__device__ __noinline__ Selected select(TopShared& S, unsigned long long* buf, unsigned* hist, int count, int K,
                                        unsigned low, unsigned largest, MaxSum rest, float c) {
    const int t = threadIdx.x;
    constexpr int kFloor = kShort ? 16 : 0;
    int bit;
    unsigned long long prefix, mask;
    search_range(low, largest, kFloor, &bit, &prefix, &mask);
    const auto word = [&](int i) { return buf[i]; };
    unsigned need = (unsigned)K, equal = (unsigned)count;  // words that match the prefix, and how many of them stay
    bool found = false;
    while (bit > kFloor && !found) {
        const int bits = min(11, bit - kFloor);
        bit -= bits;
        digit_pass<kThreads>(S, hist, word, count, prefix, mask, 32 + bit, 1 << bits, need);
        prefix |= (unsigned long long)S.digit << (32 + bit);
        mask |= (unsigned long long)((1u << bits) - 1) << (32 + bit);
        need = S.need;
        equal = S.in_bin;
        found = equal == need;  // the whole bin belongs: everything from `prefix` up
    }
    if (!found && equal <= kTies) {
        // a few equal logits: each one's place among them
        if (t == 0) S.ties = 0;
        __syncthreads();
        unsigned long long* tie = reinterpret_cast<unsigned long long*>(hist);
        for (int i = t; i < count; i += kThreads)
            if ((buf[i] & mask) == prefix) tie[atomicAdd(&S.ties, 1u)] = buf[i];
        __syncthreads();
        const int ties = (int)S.ties;
        if (t < ties) {
            const unsigned long long w = tie[t];
            unsigned place = 0;
            for (int i = 0; i < ties; ++i) place += tie[i] > w;
            if (place == need - 1) S.last = w;  // the last one to stay
        }
        __syncthreads();
        prefix = S.last;
        if (t < 2 * ties) hist[t] = 0;
        __syncthreads();
    } else if (!found) {
        // equal logits: the lowest ids, two digits of the inverted id (the bits above are all ones).  A 16-bit
        // logit's key ends in zeros, or in ones if it is negative or NaN
        if (kShort && (!(prefix >> 63) || prefix >> 48 == 0xFFFFull)) prefix |= 0xFFFFull << 32;
        prefix |= 0xFFF00000ull;
        mask = ~0ull << 20;
        for (int shift = 10; shift >= 0 && !found; shift -= 10) {
            digit_pass<kThreads>(S, hist, word, count, prefix, mask, shift, 1024, need);
            prefix |= (unsigned long long)S.digit << shift;
            mask |= 1023ull << shift;
            need = S.need;
            found = S.in_bin == need;
        }
    }
    // the words from `prefix` up, exactly K, to the front; a thread's words of a
    // tile are read before the scan's barriers and written after them
    unsigned kept = 0, least = 0xFFFFFFFFu;
    for (int i0 = 0; i0 < count; i0 += kTile * kThreads) {
        unsigned long long w[kTile];
        unsigned keep = 0, all;
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
            const int i = i0 + j * kThreads + t;
            if (i0 + j * kThreads >= count) break;
            w[j] = i < count ? buf[i] : 0;
            if (w[j] >= prefix) {
                keep |= 1u << j;
                least = min(least, (unsigned)(w[j] >> 32));
            } else if (i < count) {
                add(rest, key_logit((unsigned)(w[j] >> 32)), c);
            }
        }
        unsigned at = kept + block_scan<kThreads>((unsigned)__popc(keep), S.warp, &all);
#pragma unroll
        for (int j = 0; j < kTile; ++j) {
            if (i0 + j * kThreads >= count) break;
            if (keep >> j & 1u) buf[at++] = w[j];
        }
        kept += all;
    }
    return {kWantBound ? ~block_max<kThreads>(~least, S.warp) : 0u, rest};
}

// kSplit: a row is a cluster's, else one CTA's.
template <typename T, int kThreads, bool kSplit>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 3 : 2) k_top(const T* __restrict__ logits, long long ld, int V, int K,
                                                     float temperature, int32_t* __restrict__ ids,
                                                     float* __restrict__ top, float* __restrict__ rest, int chunk) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ TopShared S;
    constexpr bool kShort = sizeof(T) == 2;
    constexpr int kWarps = kThreads / 32;
    constexpr int kSlots = 2 * kThreads;  // maxima that a bound may be taken from: of every thread's even and odd steps
    constexpr int kPer = Vec16<T>::kElems, P = kPer / 2;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = kSplit ? (int)cluster.block_rank() : 0, size = kSplit ? (int)cluster.num_blocks() : 1;
    const int n = blockIdx.x / size, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    unsigned* hist = reinterpret_cast<unsigned*>(smem);
    unsigned long long* buf = reinterpret_cast<unsigned long long*>(hist + kBins);
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + kBins * 4 + words_bytes(K));
    const int most_groups = groups_of<T, kThreads>(chunk);
    float* sums = reinterpret_cast<float*>(smem + front_bytes<kThreads>(most_groups, K));
    Raw<T>* maxima = reinterpret_cast<Raw<T>*>(sums + most_groups);
    const int v0 = min(V, rank * chunk);
    const Vectors<T> x(logits + (size_t)n * ld + v0, min(V, v0 + chunk) - v0);
    const float c = kLog2e / temperature;
    const F2 cc = f2(c, c);

    // the groups: a thread's vectors of a step, kThreads groups a step (-inf where there is nothing)
    float slot[2] = {-INFINITY, -INFINITY};
    int at_group = t;
    Streamer<kThreads, kAhead, kStages, true, T> vectors(x, reinterpret_cast<uint4*>(smem));
    vectors.run([&](int, Vec16<T>* v, auto) {
        float m = v[0].top_nan();
#pragma unroll
        for (int j = 1; j < kAhead; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(v[j].top_nan()));
        // exponentials on the group's own scale
        const float at = clamp_max(-FLT_MAX, m);
        const F2 minus = f2(-at, -at);
        F2 s = f2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) s = add2(s, ex2x2(mul2(add2(v[j].pair(e), minus), cc)));
        const float2 h = halves(s);
        sums[at_group] = h.x + h.y;
        maxima[at_group] = to_raw<T>(m);
        at_group += kThreads;
        asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(slot[0]));
        slot[0] = slot[1];
        slot[1] = m;
    });
    const int groups = at_group - t;
    __syncthreads();  // the ring is free, the groups are there

    // The bound.  For a K well below the number of slots in use (every thread's even
    // and odd steps) the K-th largest of their maxima does: K elements reach it, and
    // in a row without order about -ln(1 - K / slots) slots do.  Else the K-th
    // largest of the groups', or, where the groups are few, of the elements
    // themselves (19 rows of 12,064 bf16 logits, K = 1888: 23 us; with every group
    // read again without a bound 69 us), or not twice K and the row short (400 rows of
    // 9,001 fp32 logits, K = 380: 33 us, by the slots 76; but 400 rows of 60,000 bf16
    // logits, K = 1200: 107 us by the elements, 66 by the groups).
    unsigned bound = 0;
    {
        for (int i = t; i < kBins; i += kThreads) hist[i] = 0;
        const int nvec = x.last - x.first, used = min(nvec / kAhead, kSlots);
        const bool loose = nvec < 2 * K * kAhead && nvec * kPer <= 16384;  // many elements may pass, few are to be read
        const bool by_slots = !loose && 4 * K <= 3 * used, by_groups = !loose && 4 * K * kAhead <= 3 * nvec;
        const unsigned keys[2] = {top_key(slot[0]), top_key(slot[1])};
        unsigned lowest = min(keys[0], keys[1]);
        const unsigned largest = block_max<kThreads>(max(keys[0], keys[1]), S.warp);
        uint32_t* all = reinterpret_cast<uint32_t*>(buf);
        if (by_slots) {
            all[t] = __float_as_uint(slot[0]);
            all[kThreads + t] = __float_as_uint(slot[1]);
        } else if (by_groups) {
            for (int g = t; g < groups; g += kThreads) lowest = min(lowest, top_key(from_raw(maxima[g])));
        }
        lowest = ~block_max<kThreads>(~lowest, S.warp);
        if (by_slots)
            bound = bound_by<kThreads, kShort>(S, hist, all, kSlots, K, lowest, largest);
        else if (by_groups)
            bound = bound_by<kThreads, kShort>(S, hist, maxima, groups, K, lowest, largest);
        else if (nvec * kPer > K + kDue)
            bound = bound_by<kThreads, kShort>(S, hist, reinterpret_cast<const T*>(x.vec() + x.first), nvec * kPer, K, 0u, largest);
        if (kShort) bound &= 0xFFFF0000u;
        bound = min(bound, 0xFF800000u);  // +inf: a NaN is never below the bound
    }
    // as a logit; keys up to -inf's: -inf; a 16-bit logit's key ends in ones if it is negative
    const float bound_logit =
        bound <= 0x007FFFFFu ? -INFINITY : unord_f32(kShort && !(bound >> 31) ? bound | 0xFFFFu : bound);

    // the groups below the bound are in the rest; the others' list, a thread's after another's
    MaxSum r = empty_set();
    int listed;
    {
        struct alignas(4 * sizeof(Raw<T>)) Four {
            Raw<T> m[4];
        };
        const Four* four = reinterpret_cast<const Four*>(maxima);
        int mine = 0;
        float m = -INFINITY;
#pragma unroll 2
        for (int i = t; i < groups / 4; i += kThreads) {
            const Four y4 = four[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float y = from_raw(y4.m[j]);
                const bool in = !(y < bound_logit);
                mine += in;
                if (!in) m = fmaxf(m, y);
            }
        }
        unsigned all, at = block_scan<kThreads>((unsigned)mine, S.warp, &all);  // this thread's first place
        listed = (int)all;
        r.m = clamp_max(-FLT_MAX, m);
#pragma unroll 1
        for (int i = t; i < groups / 4; i += kThreads) {
            const Four y4 = four[i];
            const float4 s4 = reinterpret_cast<const float4*>(sums)[i];
            const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float y = from_raw(y4.m[j]);
                if (!(y < bound_logit)) list[at++] = (uint16_t)(4 * i + j);
                else r.s += s[j] * ex2((clamp_max(-FLT_MAX, y) - r.m) * c);
            }
        }
    }
    __syncthreads();

    // Words are made of what lies above the bound.  What equals it (masked rows
    // are full of -inf, 16-bit rows of any value) only leaves a bit in `equal`,
    // in the order of the ids, over the groups' place.
    unsigned* equal = reinterpret_cast<unsigned*>(sums);
    const int equal_words = (x.phase + x.n + 31) / 32;
    for (int i = t; i < equal_words; i += kThreads) equal[i] = 0;
    __syncthreads();
    unsigned most = 0;  // largest key of this thread's words
    int count = 0;      // words in the buffer
    unsigned last = bound;  // no larger than the key of the K-th best
    int equals = 0;         // this thread's elements that equal the bound
    const auto reduce = [&] {  // the buffer's best K
        if (count <= K) return;
        const unsigned top_key_seen = block_max<kThreads>(most, S.warp);
        const Selected got = select<kThreads, kShort, kSplit>(S, buf, hist, count, K, bound, top_key_seen, r, c);
        last = got.bound;
        r = got.rest;
        count = K;
    };
    // Takes `n` words of this thread; says no, and takes none, where the buffer
    // has no room for all threads' words (for kStep it always has).
    const auto take = [&](unsigned n_words, auto&& write) {
        unsigned all;
        const unsigned at = block_scan<kThreads>(n_words, S.warp, &all);
        if (count + (int)all > K + kDue + kStep) return false;
        if (n_words) write(buf + count + at);
        count += (int)all;
        if (count > K + kDue) {
            __syncthreads();
            reduce();
        }
        return true;
    };
    // the listed groups again, a group per thread
#pragma unroll 1
    for (int l0 = 0; l0 < listed; l0 += kThreads) {
        unsigned pass = 0;  // a bit per element above the bound; those below it into the rest
        const int i0 = x.first + (l0 + t < listed ? list[l0 + t] : groups) * kAhead;
        if (l0 + t - lane < listed) {
            Vec16<T> v[kAhead];
            const unsigned inf = kShort ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                v[j].q = make_uint4(inf, inf, inf, inf);
                if (i0 + j < x.last) v[j].q = x.vec()[i0 + j];
            }
            MaxSum o = empty_set();
            F2 s = f2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                unsigned in = 0, eq = 0;
                Vec16<T> others = v[j];
                if (i0 + j < x.last) others = above(v[j], bound_logit, &in, &eq);
                pass |= in << (j * kPer);
                if (in) most = max(most, top_key(v[j].top_nan()));
                if (eq) {
                    const int at = (i0 + j) * kPer;
                    atomicOr(&equal[at >> 5], eq << (at & 31));
                    equals += __popc(eq);
                }
                v[j] = others;
            }
            o.m = clamp_max(-FLT_MAX, top_of<kAhead>(v));
            const F2 minus = f2(-o.m, -o.m);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int e = 0; e < P; ++e) s = add2(s, ex2x2(mul2(add2(v[j].pair(e), minus), cc)));
            const float2 h = halves(s);
            o.s = h.x + h.y;
            r = join(r, o, c);
        }
        // the words of the elements that `some` names, their logits once more from memory
        const auto write = [&](unsigned long long* to, unsigned some) {
#pragma unroll 1
            for (; some; some &= some - 1) {
                const int at = i0 * kPer - x.phase + __ffs((int)some) - 1;
                *to++ = word_of(top_key(to_f32(x.src[at])), (unsigned)(v0 + at));
            }
        };
        if (!take((unsigned)__popc(pass), [&](unsigned long long* to) { write(to, pass); })) {
            constexpr int kSome = kStep / kThreads;  // elements of each group at a time
#pragma unroll 1
            for (int b = 0; b < kAhead * kPer; b += kSome) {
                const unsigned some = pass & (((1u << kSome) - 1u) << b);
                take((unsigned)__popc(some), [&](unsigned long long* to) { write(to, some); });
            }
        }
    }
    if (x.n > (x.last - x.first) * kPer) {  // the elements beside the whole vectors
        const int at = t < 2 * kPer ? x.beside(t) : x.n;
        const float y = at < x.n ? to_f32(x.src[at]) : 0.f;
        const bool in = at < x.n && !(y <= bound_logit);
        if (in) most = max(most, top_key(y));
        else if (at < x.n && y == bound_logit) atomicOr(&equal[(at + x.phase) >> 5], 1u << ((at + x.phase) & 31)), ++equals;
        else if (at < x.n) add(r, y, c);
        take(in, [&](unsigned long long* to) { *to = word_of(top_key(y), (unsigned)(v0 + at)); });
    }
    __syncthreads();
    reduce();
    __syncthreads();
    if (count < K) {  // of what equals the bound: the lowest ids, as many as the buffer still lacks
        const int lack = K - count, per = (equal_words + kThreads - 1) / kThreads;
        const int from = min(equal_words, t * per), to = min(equal_words, from + per);
        unsigned mine = 0, all;
        for (int i = from; i < to; ++i) mine += (unsigned)__popc(equal[i]);
        int at = (int)block_scan<kThreads>(mine, S.warp, &all);
        const int taken = min(lack, (int)all);
        for (int i = from; i < to && at < taken; ++i)
            for (unsigned m = equal[i]; m && at < taken; m &= m - 1)
                buf[count + at++] = word_of(top_key(bound_logit), (unsigned)(v0 + i * 32 + __ffs((int)m) - 1 - x.phase));
        if (taken) most = max(most, top_key(bound_logit));
        equals = t == 0 ? (int)all - taken : 0;
        count += taken;
        __syncthreads();
    }
    if (equals && bound_logit != -INFINITY)
        r = join(r, MaxSum{clamp_max(-FLT_MAX, bound_logit), bound_logit == INFINITY ? INFINITY : (float)equals}, c);

    if constexpr (kSplit) {
        cluster_barrier();
        if (rank == 0) {
            // the other slices' words: a warp per slice, kWords of a lane at once
            const unsigned beaten = count == K ? last : 0u;  // a higher id with this key comes after all K of this slice
            constexpr int kWords = kStep / kThreads;
            const int each = min(K, chunk);
#pragma unroll 1
            for (int from = 1 + warp; from - warp < size; from += kWarps) {
                const int here = from < size ? min(K, min(V, (from + 1) * chunk) - min(V, from * chunk)) : 0;
                const unsigned long long* theirs = cluster.map_shared_rank(buf, min(from, size - 1));
                for (int i0 = 0; i0 < each; i0 += 32 * kWords) {
                    unsigned long long w[kWords];
                    unsigned pass = 0;
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        const int i = i0 + 32 * j + lane;
                        w[j] = i < here ? theirs[i] : 0;
                    }
#pragma unroll
                    for (int j = 0; j < kWords; ++j) {
                        const unsigned k = (unsigned)(w[j] >> 32);  // 0: no word
                        if (k == 0) continue;
                        if (k > beaten) {
                            pass |= 1u << j;
                            most = max(most, k);
                        } else {
                            add(r, key_logit(k), c);
                        }
                    }
                    take((unsigned)__popc(pass), [&](unsigned long long* to) {
#pragma unroll
                        for (int j = 0; j < kWords; ++j)
                            if (pass >> j & 1u) *to++ = w[j];
                    });
                }
            }
            __syncthreads();
            reduce();
        }
    }
    // the CTA's rest
    {
        const float m = warp_max(r.m);
        r.s = warp_sum(r.s * ex2((r.m - m) * c));
        if (lane == 0) S.part[warp] = {m, r.s};
        __syncthreads();
        if (warp == 0) {
            r = lane < kWarps ? S.part[lane] : empty_set();
            const float all = warp_max(r.m);
            r.s = warp_sum(r.s * ex2((r.m - all) * c));
            r.m = all;
            if (kSplit && lane == 0) *cluster.map_shared_rank(&S.rest[rank], 0) = r;
        }
    }
    if constexpr (kSplit) {
        cluster_barrier();
        if (rank != 0) return;
        if (warp == 0) {
            r = lane < size ? S.rest[lane] : empty_set();
            const float all = warp_max(r.m);
            r.s = warp_sum(r.s * ex2((r.m - all) * c));
            r.m = all;
        }
    }
    if (t == 0) rest[n] = r.s == 0.f ? -INFINITY : r.m / temperature + logf(r.s);

    if (K <= kFew) {  // ascending ids: a word's place is the number of lower ids
        if (t - lane >= K) return;
        const unsigned long long w = t < K ? buf[t] : 0;
        const unsigned id = word_id(w);
        int place = 0;
#pragma unroll 8
        for (int i = 0; i < K; ++i) place += word_id(buf[i]) < id;
        if (t < K) {
            ids[(size_t)n * K + place] = (int32_t)id;
            top[(size_t)n * K + place] = key_logit((unsigned)(w >> 32));
        }
        return;
    }
    // many: a bit per id, counted in front of each thread's words of bits
    unsigned* bits = reinterpret_cast<unsigned*>(sums);  // over the groups
    unsigned* before = hist;
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
    before[t] = block_scan<kThreads>(mine, S.warp, &all);
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

// shared memory of each of a row's `size` CTAs
template <typename T, int kThreads>
constexpr size_t smem_of(int V, int K, int size) {
    const size_t bits = (size_t)((V + 31) / 32 + kThreads) * 4;
    const int groups = groups_of<T, kThreads>(slice_of(V, size));
    const size_t back = group_bytes<T>(groups);
    return front_bytes<kThreads>(groups, K) + (back > bits ? back : bits);
}
static_assert(smem_of<__nv_bfloat16, 512>(DOMINO_TRAIN_MAX_V, DOMINO_TRAIN_MAX_K, 1) <= kMaxSmem,
              "every bf16 row is one CTA's");
static_assert(smem_of<float, 512>(DOMINO_TRAIN_MAX_V, DOMINO_TRAIN_MAX_K, 4) <= kMaxSmem, "of fp32 rows four CTAs'");

template <typename T, int kThreads, bool kSplit>
cudaError_t launch_with(int size, int V, const void* x, long long ld, int n, int K, float temperature, int32_t* ids,
                        float* top, float* rest, cudaStream_t st) {
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg =
        cluster_config((unsigned)n * size, kThreads, size, smem_of<T, kThreads>(V, K, size), st, &attr);
    if (!kSplit) cfg.numAttrs = 0;
    return cudaLaunchKernelEx(&cfg, k_top<T, kThreads, kSplit>, static_cast<const T*>(x), ld, V, K, temperature, ids, top,
                              rest, slice_of(V, size));
}

template <typename T>
cudaError_t launch(domino_train_ctx* c, const void* x, long long ld, int n, int K, float temperature, int32_t* ids,
                   float* top, float* rest, cudaStream_t st) {
    const int V = c->cfg.V;
    c->last_launches = 1;
    if (smem_of<T, 256>(V, K, 1) <= kThirdSmem && (n > c->num_sms || K <= kFew))
        return launch_with<T, 256, false>(1, V, x, ld, n, K, temperature, ids, top, rest, st);
    if constexpr (sizeof(T) == 4) {
        // fp32 rows from 229,313 (K = 8192) or 327,617 (K <= 64) entries on
        int size = 1;
        while (smem_of<T, 512>(V, K, size) > kMaxSmem) size *= 2;
        if (size > 1) return launch_with<T, 512, true>(size, V, x, ld, n, K, temperature, ids, top, rest, st);
    }
    return launch_with<T, 512, false>(1, V, x, ld, n, K, temperature, ids, top, rest, st);
}

}  // namespace

cudaError_t prepare_top_kernels() {
    cudaError_t e = allow_all(k_top<float, 256, false>);
    if (e == cudaSuccess) e = allow_all(k_top<float, 512, false>);
    if (e == cudaSuccess) e = allow_all(k_top<float, 512, true>);
    if (e == cudaSuccess) e = allow_all(k_top<__nv_bfloat16, 256, false>);
    if (e == cudaSuccess) e = allow_all(k_top<__nv_bfloat16, 512, false>);
    return e;
}

cudaError_t launch_top(domino_train_ctx* c, const void* x, int dtype, long long ld, int n, int K, float temperature,
                       int32_t* ids, float* top, float* rest, cudaStream_t st) {
    return dtype == DOMINO_DTYPE_BF16 ? launch<__nv_bfloat16>(c, x, ld, n, K, temperature, ids, top, rest, st)
                                      : launch<float>(c, x, ld, n, K, temperature, ids, top, rest, st);
}

}  // namespace train
}  // namespace domino
