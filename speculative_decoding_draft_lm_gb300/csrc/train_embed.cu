// Scaled embedding lookup and the gradient of its table.
//
//   lookup:    out[i] = scale * table[tok_i]
//   gradient:  dtable[v] = scale * sum_{i: tok_i = v} dout[i]
//
// Both only move rows, so both are bound by HBM.  The gradient writes the whole
// table and touches few of its rows (1024 tokens: under 1 % of 151,936), so most
// of its time is the zeros, and nothing must wait in front of them.
//
// The gradient sorts the tokens with their positions (stable), so that every
// row's sum has one owner and one order: no atomics on the gradient, the same
// bits every time.  Launches:
//   k_mark          finds the rows that tokens name;
//   k_fill          writes zeros to the others;
//   k_sort_cluster  beside it, one cluster sorts all tokens through distributed
//                   shared memory (up to 16 x 8192; more take the tiled passes);
//   k_sum_runs      every group of threads sums `unit` consecutive sorted places,
//                   so that a frequent token's thousands of rows are spread over
//                   the chip; a run of equal tokens that lies inside a unit goes
//                   straight to its row, one that crosses a unit's edge leaves
//                   a partial row;
//   k_join_runs     adds a crossing run's partial rows in their order.
#include <cooperative_groups.h>

#include "train_internal.h"
#include "train_stream.cuh"

namespace cg = cooperative_groups;

namespace domino {
namespace train {

namespace {

// ---- vectors of four elements ------------------------------------------------

template <typename T, int VEC>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    T raw;
    __device__ __forceinline__ void load(const T* p) { raw = *p; }
    __device__ __forceinline__ void get(float* f) const { f[0] = to_f32(raw); }
};
template <>
struct Vec<float, 4> {
    float4 raw;
    __device__ __forceinline__ void load(const float* p) { raw = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float* f) const { f[0] = raw.x; f[1] = raw.y; f[2] = raw.z; f[3] = raw.w; }
};
template <>
struct Vec<__nv_bfloat16, 4> {
    uint2 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(float* f) const {
        bf16x2_to_f32(raw.x, f[0], f[1]);
        bf16x2_to_f32(raw.y, f[2], f[3]);
    }
};
template <>
struct Vec<__nv_bfloat16, 8> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float* f) const {
        bf16x2_to_f32(raw.x, f[0], f[1]);
        bf16x2_to_f32(raw.y, f[2], f[3]);
        bf16x2_to_f32(raw.z, f[4], f[5]);
        bf16x2_to_f32(raw.w, f[6], f[7]);
    }
};
__device__ __forceinline__ unsigned pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&v);
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const float* f) {
    if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
        *p = f[0];
}
template <int VEC>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    else if constexpr (VEC == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    else
        *p = __float2bfloat16_rn(f[0]);
}

// rows of `e`-byte elements can be moved `vec` elements at a time
inline bool by_vec(const void* p, long long ld, int E, int e, int vec) {
    return E % vec == 0 && ld % vec == 0 && (uintptr_t)p % (uintptr_t)(vec * e) == 0;
}

// Threads over the columns of rows of `cols` vectors, and rows per block.
inline void row_block(int cols, int threads, dim3* block, int* col_blocks) {
    int tx = 1;
    while (tx < cols && tx < 32) tx *= 2;
    *col_blocks = (cols + threads - 1) / threads;
    if (cols > 32) tx = ((cols + *col_blocks - 1) / *col_blocks + 31) / 32 * 32;  // equal blocks of whole warps
    *block = dim3(tx, threads / tx);
}

// ---- lookup ------------------------------------------------------------------

constexpr int kEmbedThreads = 256;

// Threads over a row's 16-byte vectors; each thread moves ROWS tokens' vectors
// at once.  Bound by HBM and, for frequent tokens' rows, L2: 61,440 tokens of
// E = 1536 bf16 in 47 us (0.38 GB: 8.0 TB/s, above the copy rate by what L2 holds).
// Widths or strides off 16 bytes go by single elements: E = 1535 takes 152 us.
template <typename T, int VEC, int ROWS>
__global__ void __launch_bounds__(kEmbedThreads) k_embed(const T* __restrict__ table,
                                                         const int32_t* __restrict__ tokens, int n, int V, int E,
                                                         float scale, T* __restrict__ out, long long ld, int* err) {
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    const long long i0 = ((long long)blockIdx.x * blockDim.y + threadIdx.y) * ROWS;
    if (col >= E) return;
    Vec<T, VEC> v[ROWS];
    bool in[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int tok = i0 + r < n ? tokens[i0 + r] : -1;
        in[r] = (unsigned)tok < (unsigned)V;
        if (in[r]) v[r].load(table + (size_t)tok * E + col);
        else if (tok != -1 && col == 0) atomicOr(err, kErrBadToken);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (i0 + r >= n) break;
        float f[VEC];
        v[r].get(f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = in[r] ? scale * f[k] : 0.f;
        store<VEC>(out + (size_t)(i0 + r) * ld + col, f);
    }
}

// ---- sort --------------------------------------------------------------------
//
// Two passes of a stable counting sort, low digit first.  A tile's tokens are
// split into 32-token steps in their order, a warp's steps adjacent; a token's
// place is (smaller digits) + (its digit in the tiles before) + (in the warps
// before) + (in its warp before it), the last from ballots.  Tokens
// outside [0, V) sort last, as V.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortSteps = kSortTile / kSortThreads;  // tokens per thread
static_assert(kSortTile % kSortThreads == 0 && kSortMaxBins <= kSortThreads, "one bin per thread");
static_assert(kSortTile == 1 << 13, "the largest tile of a cluster's sort");

struct SortShared {
    uint16_t warp[kSortWarps][kSortMaxBins];  // a warp's counts, then the tile's counts in the warps before it
    unsigned total[kSortMaxBins];             // the tile's count
    unsigned base[kSortMaxBins];              // first place of the tile's tokens of a digit
    unsigned sums[kSortWarps];
};
struct SortClusterShared {
    SortShared s;
    uint32_t key[kSortTile];
    int32_t pos[kSortTile];
};

__device__ __forceinline__ uint32_t token_key(int tok, int V, int* err) {
    if ((unsigned)tok < (unsigned)V) return (uint32_t)tok;
    if (tok != -1) atomicOr(err, kErrBadToken);
    return (uint32_t)V;
}

// The tile's tokens by thread: step j of this thread's warp.  A tile that is not
// full spreads over all warps.
__device__ __forceinline__ int tile_steps(int count) { return (count + kSortThreads - 1) / kSortThreads; }
__device__ __forceinline__ int tile_place(int j, int steps) {
    return ((int)(threadIdx.x >> 5) * steps + j) * 32 + (int)(threadIdx.x & 31);
}

// Counts the digits of this tile: rank[j] = this thread's j-th token's place
// among its warp's tokens of that digit; s.warp and s.total as above.
__device__ void tile_count(SortShared& s, const uint32_t* key, unsigned* rank, int count, int shift, int bins) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, steps = tile_steps(count);
    for (int b = lane; b < bins; b += 32) s.warp[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        if (j >= steps) break;
        const bool in = tile_place(j, steps) < count;
        const unsigned d = key[j] >> shift & (unsigned)(bins - 1);
        // the lanes with the same digit, a ballot per bit (__match_any_sync took
        // 3.3 K cycles a step of 32 warps)
        unsigned peers = __ballot_sync(0xffffffffu, in);
        for (int b = 1; b < bins; b <<= 1) {
            const unsigned ones = __ballot_sync(0xffffffffu, (d & (unsigned)b) != 0);
            peers &= d & (unsigned)b ? ones : ~ones;
        }
        const unsigned below = __popc(peers & ((1u << lane) - 1u));
        if (in) rank[j] = s.warp[warp][d] + below;
        __syncwarp();
        if (in && below == 0) s.warp[warp][d] += (uint16_t)__popc(peers);
        __syncwarp();
    }
    __syncthreads();
    if ((int)threadIdx.x < bins) {
        unsigned run = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const unsigned c = s.warp[w][threadIdx.x];
            s.warp[w][threadIdx.x] = (uint16_t)run;
            run += c;
        }
        s.total[threadIdx.x] = run;
    }
}

// s.base from this thread's digit's count in the tiles before and in all tiles.
__device__ void tile_base(SortShared& s, unsigned before, unsigned all, int bins) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned incl = all;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s.sums[warp] = incl;
    __syncthreads();
    unsigned w = s.sums[lane], wi = w;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) wi += y;
    }
    const unsigned smaller = __shfl_sync(0xffffffffu, wi - w, warp) + incl - all;
    if ((int)threadIdx.x < bins) s.base[threadIdx.x] = smaller + before;
    __syncthreads();
}

// All tokens in one cluster: a tile of 2^log_tile tokens per CTA, exchanged
// through distributed shared memory.  Alone, most of a pass are the scattered
// stores, 32 sectors each, so the tokens are spread over up to 16 CTAs (65,536
// tokens: 26 us against 37 us on 8; 8,192 tokens: 13 us against 26 us on 1; the
// tiled passes below took 42 us for either).  Beside k_fill, whose stores crowd theirs out, full
// tiles on fewer CTAs end earlier (the whole gradient of 65,536 tokens: 196 us
// against 205 us).
__global__ void __launch_bounds__(kSortThreads) k_sort_cluster(const int32_t* __restrict__ tokens, int n, int V,
                                                               int digit, int log_tile, uint32_t* __restrict__ keys_out,
                                                               int32_t* __restrict__ pos_out, int* err) {
    extern __shared__ __align__(16) uint8_t smem[];
    SortClusterShared& S = *reinterpret_cast<SortClusterShared*>(smem);
    cg::cluster_group cluster = cg::this_cluster();
    const int tiles = (int)cluster.num_blocks(), tile = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, bins = 1 << digit;
    const int count = max(0, min(1 << log_tile, n - (tile << log_tile))), steps = tile_steps(count);
    uint32_t key[kSortSteps];
    unsigned rank[kSortSteps];
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int i = tile_place(j, steps);
        key[j] = j < steps && i < count ? token_key(tokens[(tile << log_tile) + i], V, err) : 0u;
    }
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const int shift = pass * digit;
        tile_count(S.s, key, rank, count, shift, bins);
        cluster_barrier();
        unsigned before = 0, all = 0;
        if ((int)threadIdx.x < bins)
#pragma unroll
            for (int t = 0; t < kSortMaxCluster; ++t) {
                const unsigned c = t < tiles ? cluster.map_shared_rank(S.s.total, t)[threadIdx.x] : 0u;
                if (t < tile) before += c;
                all += c;
            }
        tile_base(S.s, before, all, bins);
#pragma unroll
        for (int j = 0; j < kSortSteps; ++j)
            if (j < steps && tile_place(j, steps) < count) {
                const unsigned d = key[j] >> shift & (unsigned)(bins - 1);
                const unsigned at = S.s.base[d] + S.s.warp[warp][d] + rank[j];
                const int i = tile_place(j, steps);
                if (pass == 0) {
                    cluster.map_shared_rank(S.key, at >> log_tile)[at & ((1u << log_tile) - 1u)] = key[j];
                    cluster.map_shared_rank(S.pos, at >> log_tile)[at & ((1u << log_tile) - 1u)] = (tile << log_tile) + i;
                } else {
                    keys_out[at] = key[j];
                    pos_out[at] = S.pos[i];
                }
            }
        cluster_barrier();  // the tile's new tokens are here; nobody reads these counts any more
        if (pass == 0) {
#pragma unroll
            for (int j = 0; j < kSortSteps; ++j)
                if (j < steps && tile_place(j, steps) < count) key[j] = S.key[tile_place(j, steps)];
        }
    }
    // launched beside k_fill (whose kernels before it are done and write nothing
    // read here): end after it, so that what waits for this kernel has waited for both
    pdl_wait();
}

// The same passes for more tokens than a cluster holds: digit counts of every
// tile, then the tiles' tokens to their places.  tokens is null in pass 2.
__device__ __forceinline__ void load_tile(const int32_t* tokens, const uint32_t* keys, const int32_t* pos, int V,
                                          int count, uint32_t* key, int32_t* at, int* err) {
    const int steps = tile_steps(count);
    const size_t lo = (size_t)blockIdx.x * kSortTile;
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j) {
        const int i = tile_place(j, steps);
        key[j] = 0;
        if (j < steps && i < count) {
            key[j] = tokens ? token_key(tokens[lo + i], V, err) : keys[lo + i];
            if (at) at[j] = tokens ? (int32_t)(lo + i) : pos[lo + i];
        }
    }
}
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const int32_t* __restrict__ tokens,
                                                             const uint32_t* __restrict__ keys, int n, int V,
                                                             int shift, int bins, unsigned* __restrict__ hist,
                                                             int* err) {
    extern __shared__ __align__(16) uint8_t smem[];
    SortShared& s = *reinterpret_cast<SortShared*>(smem);
    const int count = min(kSortTile, n - (int)blockIdx.x * kSortTile);
    uint32_t key[kSortSteps];
    unsigned rank[kSortSteps];
    load_tile(tokens, keys, nullptr, V, count, key, nullptr, err);
    tile_count(s, key, rank, count, shift, bins);
    if ((int)threadIdx.x < bins) hist[(size_t)blockIdx.x * kSortMaxBins + threadIdx.x] = s.total[threadIdx.x];
}
__global__ void __launch_bounds__(kSortThreads) k_sort_place(const int32_t* __restrict__ tokens,
                                                             const uint32_t* __restrict__ keys_in,
                                                             const int32_t* __restrict__ pos_in, int n, int V,
                                                             int shift, int bins, const unsigned* __restrict__ hist,
                                                             uint32_t* __restrict__ keys_out,
                                                             int32_t* __restrict__ pos_out, int* err) {
    extern __shared__ __align__(16) uint8_t smem[];
    SortShared& s = *reinterpret_cast<SortShared*>(smem);
    const int count = min(kSortTile, n - (int)blockIdx.x * kSortTile);
    const int warp = threadIdx.x >> 5, steps = tile_steps(count);
    uint32_t key[kSortSteps];
    int32_t pos[kSortSteps];
    unsigned rank[kSortSteps];
    load_tile(tokens, keys_in, pos_in, V, count, key, pos, err);
    tile_count(s, key, rank, count, shift, bins);
    unsigned before = 0, all = 0;
    if ((int)threadIdx.x < bins)
        for (int t = 0; t < (int)gridDim.x; ++t) {
            const unsigned c = hist[(size_t)t * kSortMaxBins + threadIdx.x];
            if (t < (int)blockIdx.x) before += c;
            all += c;
        }
    tile_base(s, before, all, bins);
#pragma unroll
    for (int j = 0; j < kSortSteps; ++j)
        if (j < steps && tile_place(j, steps) < count) {
            const unsigned d = key[j] >> shift & (unsigned)(bins - 1);
            const unsigned at = s.base[d] + s.warp[warp][d] + rank[j];
            keys_out[at] = key[j];
            pos_out[at] = pos[j];
        }
}

// ---- zeros ---------------------------------------------------------------------

constexpr int kMarkThreads = 1024;
constexpr int kMarkBlocks = 8;
constexpr int kFillThreads = 512;
constexpr int kFillBlocksPerSm = 2;  // half of an SM's threads: the sort needs the others
constexpr int kFillRows = 32;     // rows per claim: one word of the bits

// A bit per row of the table that some token names, and the claim counter of
// k_fill.  One cluster: every CTA marks its share of the tokens in a copy of the
// bits of its own, then puts together its slice of all copies.
__global__ void __launch_bounds__(kMarkThreads) k_mark(const int32_t* __restrict__ tokens, int n, int V,
                                                       unsigned* __restrict__ named, unsigned* __restrict__ claim) {
    extern __shared__ unsigned bits[];
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), words = (V + 31) / 32, t = threadIdx.x;
    for (int i = t; i < words; i += kMarkThreads) bits[i] = 0;
    if (rank == 0 && t == 0) *claim = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = rank * kMarkThreads + t; i < n; i += kMarkBlocks * kMarkThreads) {
        const int tok = tokens[i];
        if ((unsigned)tok >= (unsigned)V) continue;
        const unsigned bit = 1u << (tok & 31);
        // look first: a frequent token's thousands of places would queue at its word
        if (!(reinterpret_cast<volatile unsigned*>(bits)[tok >> 5] & bit)) atomicOr(&bits[tok >> 5], bit);
    }
    cluster_barrier();
    const int slice = (words + kMarkBlocks - 1) / kMarkBlocks, to = min(words, (rank + 1) * slice);
    for (int i = rank * slice + t; i < to; i += kMarkThreads) {
        unsigned w = 0;
#pragma unroll
        for (int r = 0; r < kMarkBlocks; ++r) w |= cluster.map_shared_rank(bits, r)[i];
        named[i] = w;
    }
    cluster_barrier();  // nobody leaves while its copy is read
}

// Bound by HBM writes: 151,936 rows of 1024 fp32, 0.62 GB, in 84 us.
// Zeros to the rows that no token names.  One wave of blocks that claims 32
// rows at a time: an SM that also sorts, or meets many named rows, takes fewer.
template <typename G, bool VEC16>
__global__ void __launch_bounds__(kFillThreads) k_fill(const unsigned* __restrict__ named, unsigned* __restrict__ claim,
                                                       int V, int E, G* __restrict__ dtable) {
    __shared__ unsigned next[2];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, words = (V + 31) / 32;
    for (int turn = 0;; turn ^= 1) {
        if (threadIdx.x == 0) next[turn] = atomicAdd(claim, 1u);
        __syncthreads();
        const unsigned w = next[turn];
        if (w >= (unsigned)words) return;
        const unsigned bits = named[w];
        for (int r = warp; r < kFillRows; r += kFillThreads / 32) {
            const int v = (int)w * 32 + r;
            if (v >= V || (bits >> r & 1u)) continue;
            G* row = dtable + (size_t)v * E;
            if constexpr (VEC16) {
                uint4* p = reinterpret_cast<uint4*>(row);
                const int quads = E * (int)sizeof(G) / 16;
                for (int i = lane; i < quads; i += 32) p[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int e = lane; e < E; e += 32) row[e] = from_f32<G>(0.f);
            }
        }
    }
}

// ---- sums ----------------------------------------------------------------------

constexpr int kSumThreads = 256;
constexpr int kSumAhead = 4;    // rows in flight per thread, and as many being added
constexpr int kJoinAhead = 8;   // parts in flight per thread
constexpr int kMinUnit = 4, kMaxUnit = 64, kUnitsPerSm = 8;
constexpr int kJoinThreads = 256;  // 128: 198 us, 256: 194, 512: 196, 1024: 207 (the gradient of 65,536 tokens)

struct SumArgs {
    const void* dout;
    long long ld;
    const uint32_t* keys;
    const int32_t* pos;
    int n, V, E;
    int unit;       // sorted places per group of threads
    float scale;
    void* dtable;
    bool accumulate;
    float* part;    // [units][2][E]: the sums of a unit's first run, begun before it, and of its last run, not ended in it
};

template <typename G, int VEC>
__device__ __forceinline__ void write_row(const SumArgs& p, uint32_t key, int col, const float* acc) {
    G* to = static_cast<G*>(p.dtable) + (size_t)key * p.E + col;
    float f[VEC];
    if (p.accumulate) {
        Vec<G, VEC> old;
        old.load(to);
        old.get(f);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = p.accumulate ? f[j] + p.scale * acc[j] : p.scale * acc[j];
    store<VEC>(to, f);
}

// 65,536 tokens of E = 1536 bf16 (0.2 GB) into 18,000 fp32 rows (0.11 GB): 65 us,
// 0.7 of the copy rate (115 us where they are added to the rows).  Four columns a thread, four rows in flight and four
// being added, units of 64: eight columns 213 us for the whole gradient against
// 196 us, eight rows 249 us (eight columns), units of 32 208 us.
template <typename T, typename G, int VEC>
__global__ void __launch_bounds__(kSumThreads) k_sum_runs(SumArgs p) {
    extern __shared__ uint32_t entries[];  // per group of threads: the unit's keys, then their positions
    pdl_trigger();
    pdl_wait();
    const int unit = blockIdx.x * blockDim.y + threadIdx.y;
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    const int lo = (int)min((size_t)unit * p.unit, (size_t)p.n), hi = min(p.n, lo + p.unit), count = hi - lo;
    uint32_t* keys = entries + threadIdx.y * 2 * p.unit;
    int32_t* pos = reinterpret_cast<int32_t*>(keys + p.unit);
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        keys[i] = p.keys[lo + i];
        pos[i] = p.pos[lo + i];
    }
    const uint32_t none = 0xFFFFFFFFu, V = (uint32_t)p.V;
    const uint32_t key_before = lo > 0 ? p.keys[lo - 1] : none, key_after = hi < p.n ? p.keys[hi] : none;
    __syncthreads();
    if (count == 0 || col >= p.E) return;
    const T* dout = static_cast<const T*>(p.dout) + col;
    float* part = p.part + ((size_t)unit * 2) * p.E + col;
    float acc[VEC] = {};
    uint32_t run = none;
    int begun = 0;
    auto end_run = [&](int end) {  // the run [begun, end) of token `run` is summed
        if (run >= V) return;
        if (begun == 0 && run == key_before)
            store<VEC>(part, acc);
        else if (end == count && run == key_after)
            store<VEC>(part + p.E, acc);
        else
            write_row<G, VEC>(p, run, col, acc);
    };
    Vec<T, VEC> row[2][kSumAhead];
    auto load = [&](Vec<T, VEC>* r, int i0) {
#pragma unroll
        for (int j = 0; j < kSumAhead; ++j)
            if (i0 + j < count && keys[i0 + j] < V) r[j].load(dout + (size_t)pos[i0 + j] * p.ld);
    };
    auto sum = [&](const Vec<T, VEC>* r, int i0) {
#pragma unroll
        for (int j = 0; j < kSumAhead; ++j) {
            if (i0 + j >= count) break;
            const uint32_t key = keys[i0 + j];
            if (key != run) {
                end_run(i0 + j);
                run = key;
                begun = i0 + j;
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
            }
            if (key < V) {
                float f[VEC];
                r[j].get(f);
#pragma unroll
                for (int k = 0; k < VEC; ++k) acc[k] += f[k];
            }
        }
    };
    load(row[0], 0);
    for (int i0 = 0; i0 < count; i0 += 2 * kSumAhead) {
        load(row[1], i0 + kSumAhead);
        sum(row[0], i0);
        load(row[0], i0 + 2 * kSumAhead);
        sum(row[1], i0 + kSumAhead);
    }
    end_run(count);
}

// The unit in which a crossing run begins adds up its parts: its own last sum,
// then the first sums of the units after it that the run reaches.  One block
// per unit and column block; the block's rows of threads take the parts in
// turns and their sums are added in a fixed order, so that a run of thousands
// of tokens costs a few round trips.
template <typename G, int VEC>
__global__ void __launch_bounds__(kJoinThreads) k_join_runs(SumArgs p, int units) {
    __shared__ float sums[kJoinThreads * VEC];
    pdl_wait();
    const int unit = blockIdx.x, me = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    const size_t lo = (size_t)unit * p.unit, hi = lo + p.unit;  // hi < n: the grid leaves out the last unit
    const uint32_t run = p.keys[hi];
    if (run >= (uint32_t)p.V || p.keys[hi - 1] != run) return;        // nothing crosses this edge
    if (lo > 0 && p.keys[lo] == run && p.keys[lo - 1] == run) return;  // begun in an earlier unit
    // units after this one whose first place belongs to the run
    int reached = 0;
    for (int more = threads; more == threads; reached += more) {
        const int u = unit + 1 + reached + me;
        more = __syncthreads_count(u < units && p.keys[(size_t)u * p.unit] == run);
    }
    const int col = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
    const float* part = p.part + ((size_t)unit * 2) * p.E + col;  // part r > 0 is 2 r rows on, part 0 one row on
    float acc[VEC] = {};
    if (col < p.E) {
        for (int r0 = threadIdx.y; r0 <= reached; r0 += kJoinAhead * blockDim.y) {
            Vec<float, VEC> row[kJoinAhead];
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j) {
                const int r = r0 + j * blockDim.y;
                if (r <= reached) row[j].load(part + (size_t)(r == 0 ? 1 : 2 * r) * p.E);
            }
#pragma unroll
            for (int j = 0; j < kJoinAhead; ++j)
                if (r0 + j * blockDim.y <= reached) {
                    float f[VEC];
                    row[j].get(f);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) acc[k] += f[k];
                }
        }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) sums[me * VEC + k] = acc[k];
    __syncthreads();
    if (threadIdx.y != 0 || col >= p.E) return;
    for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += sums[(y * blockDim.x + threadIdx.x) * VEC + k];
    write_row<G, VEC>(p, run, col, acc);
}

// A unit's edges cost two partial rows, so units are as long as leaves
// kUnitsPerSm groups of threads per SM, and no longer than kMaxUnit.
int sum_unit(int n, int num_sms) {
    int unit = kMinUnit;
    while (unit < kMaxUnit && (long long)unit * num_sms * kUnitsPerSm < n) unit *= 2;
    return unit;
}

// ---- launches --------------------------------------------------------------------

// `beside`: it may start while the launch in front of it runs.
cudaError_t launch_sort(domino_train_ctx* c, const int32_t* tokens, int n, bool beside, cudaStream_t st) {
    const int V = c->cfg.V;
    int bits = 1;
    while ((V >> bits) != 0) ++bits;  // keys 0..V
    const int digit = (bits + 1) / 2, bins = 1 << digit, tiles = (n + kSortTile - 1) / kSortTile;
    if (tiles <= kSortMaxCluster) {
        int log_tile = beside ? 13 : 10, size = 1;
        while ((n - 1) >> log_tile >= kSortMaxCluster) ++log_tile;
        while (size << log_tile < n) size *= 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = sizeof(SortClusterShared);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = beside ? 2 : 1;
        c->last_launches += 1;
        return cudaLaunchKernelEx(&cfg, k_sort_cluster, tokens, n, V, digit, log_tile, c->keys[0], c->pos[0], c->err);
    }
    for (int pass = 0; pass < 2; ++pass) {
        const int32_t* tok = pass == 0 ? tokens : nullptr;
        const int from = pass, to = 1 - pass, shift = pass * digit;
        k_sort_count<<<tiles, kSortThreads, sizeof(SortShared), st>>>(tok, c->keys[from], n, V, shift, bins, c->hist,
                                                                      c->err);
        k_sort_place<<<tiles, kSortThreads, sizeof(SortShared), st>>>(tok, c->keys[from], c->pos[from], n, V, shift,
                                                                      bins, c->hist, c->keys[to], c->pos[to], c->err);
        c->last_launches += 2;
    }
    return cudaGetLastError();
}

template <typename G>
cudaError_t launch_fill(domino_train_ctx* c, const int32_t* tokens, int n, G* dtable, cudaStream_t st) {
    const int V = c->cfg.V, E = c->cfg.E;
    const int all = (V + 31) / 32;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        cluster_config(kMarkBlocks, kMarkThreads, kMarkBlocks, (size_t)all * 4, st, &attr);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_mark, tokens, n, V, c->named, c->claim);
    if (e != cudaSuccess) return e;
    const int most = c->num_sms * kFillBlocksPerSm, blocks = all < most ? all : most;
    const bool vec = ((uintptr_t)dtable & 15) == 0 && (size_t)E * sizeof(G) % 16 == 0;
    c->last_launches += 2;
    return launch_pdl(vec ? k_fill<G, true> : k_fill<G, false>, blocks, kFillThreads, 0, st,
                      static_cast<const unsigned*>(c->named), c->claim, V, E, dtable);
}

template <typename T, typename G, int VEC>
cudaError_t launch_sums(domino_train_ctx* c, const SumArgs& p, cudaStream_t st) {
    const int cols = (p.E + VEC - 1) / VEC, units = (p.n + p.unit - 1) / p.unit;
    dim3 block;
    int col_blocks;
    row_block(cols, kSumThreads, &block, &col_blocks);
    if (block.y > 64) block.y = 64;  // their entries: 32 KB
    const dim3 grid((units + block.y - 1) / block.y, col_blocks);
    cudaError_t e = launch_pdl(k_sum_runs<T, G, VEC>, grid, block, (size_t)block.y * 2 * p.unit * 4, st, p);
    c->last_launches += 1;
    if (e != cudaSuccess || units < 2) return e;
    row_block(cols, 128, &block, &col_blocks);
    block.y = kJoinThreads / block.x;
    c->last_launches += 1;
    return launch_pdl(k_join_runs<G, VEC>, dim3(units - 1, col_blocks), block, 0, st, p, units);
}

template <typename T, typename G>
cudaError_t launch_grad(domino_train_ctx* c, SumArgs p, const int32_t* tokens, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (!p.accumulate) e = launch_fill(c, tokens, p.n, static_cast<G*>(p.dtable), st);
    if (e == cudaSuccess && p.n > 0) e = launch_sort(c, tokens, p.n, !p.accumulate, st);
    if (e != cudaSuccess || p.n == 0) return e;
    const bool four = by_vec(p.dout, p.ld, p.E, sizeof(T), 4) && by_vec(p.dtable, p.E, p.E, sizeof(G), 4);
    return four ? launch_sums<T, G, 4>(c, p, st) : launch_sums<T, G, 1>(c, p, st);
}

}  // namespace

int max_sum_units(int max_tokens, int num_sms) {
    // calls that a unit of less than kMaxUnit suffices for have at most
    // kUnitsPerSm * num_sms units, the others fewer than their tokens / kMaxUnit
    const int a = kUnitsPerSm * num_sms, b = (max_tokens + kMaxUnit - 1) / kMaxUnit;
    return a > b ? a : b;
}

cudaError_t prepare_embed_kernels() {
    cudaError_t e = allow_all(k_sort_cluster);
    if (e == cudaSuccess) e = allow_all(k_sort_count);
    if (e == cudaSuccess) e = allow_all(k_sort_place);
    if (e == cudaSuccess) e = allow_all(k_mark);
    return e;
}

namespace {
template <typename T, int VEC>
cudaError_t embed(domino_train_ctx* c, const void* table, const int32_t* tokens, int n, float scale, void* out,
                  long long ld, cudaStream_t st) {
    const int V = c->cfg.V, E = c->cfg.E;
    dim3 block;
    int col_blocks;
    row_block((E + VEC - 1) / VEC, kEmbedThreads, &block, &col_blocks);
    // several rows a thread once that still fills the chip
    const bool many = (long long)n * col_blocks >= (long long)c->num_sms * 32 * (int)block.y;
    const int rows = (many ? 4 : 1) * (int)block.y;
    const dim3 grid((unsigned)(((long long)n + rows - 1) / rows), col_blocks);
    auto kern = many ? k_embed<T, VEC, 4> : k_embed<T, VEC, 1>;
    kern<<<grid, block, 0, st>>>(static_cast<const T*>(table), tokens, n, V, E, scale, static_cast<T*>(out), ld,
                                 c->err);
    c->last_launches = 1;
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_embed(domino_train_ctx* c, const void* table, const int32_t* tokens, int n, float scale, void* out,
                         long long ld, cudaStream_t st) {
    const int E = c->cfg.E;
    if (c->cfg.dtype == DOMINO_DTYPE_BF16)
        return by_vec(table, E, E, 2, 8) && by_vec(out, ld, E, 2, 8)
                   ? embed<__nv_bfloat16, 8>(c, table, tokens, n, scale, out, ld, st)
                   : embed<__nv_bfloat16, 1>(c, table, tokens, n, scale, out, ld, st);
    return by_vec(table, E, E, 4, 4) && by_vec(out, ld, E, 4, 4)
               ? embed<float, 4>(c, table, tokens, n, scale, out, ld, st)
               : embed<float, 1>(c, table, tokens, n, scale, out, ld, st);
}

cudaError_t launch_embed_grad(domino_train_ctx* c, const void* dout, long long ld, const int32_t* tokens, int n,
                              float scale, void* dtable, int grad_dtype, bool accumulate, cudaStream_t st) {
    SumArgs p = {};
    p.dout = dout;
    p.ld = ld;
    p.keys = c->keys[0];
    p.pos = c->pos[0];
    p.n = n;
    p.V = c->cfg.V;
    p.E = c->cfg.E;
    p.unit = sum_unit(n, c->num_sms);
    p.scale = scale;
    p.dtable = dtable;
    p.accumulate = accumulate;
    p.part = c->part;
    const bool in16 = c->cfg.dtype == DOMINO_DTYPE_BF16, out16 = grad_dtype == DOMINO_DTYPE_BF16;
    if (in16)
        return out16 ? launch_grad<__nv_bfloat16, __nv_bfloat16>(c, p, tokens, st)
                     : launch_grad<__nv_bfloat16, float>(c, p, tokens, st);
    return out16 ? launch_grad<float, __nv_bfloat16>(c, p, tokens, st) : launch_grad<float, float>(c, p, tokens, st);
}

}  // namespace train
}  // namespace domino
