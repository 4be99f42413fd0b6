// Scaled embedding lookup and the gradient of its table.
//
// The gradient sums the rows of dout that share a token.  The tokens are sorted
// first (stable, least significant digit first, with their positions), so that
// every sum has one owner and one order: no atomics on the gradient, the same
// bits every time.
#include "train_internal.h"
#include "train_math.cuh"

namespace domino {
namespace train {

namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

template <typename T>
__global__ void __launch_bounds__(256) k_embed(const T* __restrict__ table, const int32_t* __restrict__ tokens, int n,
                                               int V, int E, float scale, T* __restrict__ out, long long ld, int* err) {
    const int i = blockIdx.x;
    const int tok = tokens[i];
    const bool in = (unsigned)tok < (unsigned)V;
    if (!in && tok != -1 && threadIdx.x == 0) atomicOr(err, kErrBadToken);
    const T* src = table + (size_t)(in ? tok : 0) * E;
    for (int e = threadIdx.x; e < E; e += 256)
        out[(size_t)i * ld + e] = from_f32<T>(in ? scale * to_f32(src[e]) : 0.f);
}

// Digit counts of each tile.  The first pass reads the tokens themselves (an
// id outside [0, V) becomes V, which sorts last).
__global__ void __launch_bounds__(kSortThreads) k_sort_count(const int32_t* __restrict__ tokens,
                                                             const uint32_t* __restrict__ keys, int n, int V,
                                                             int shift, int bins, unsigned* __restrict__ hist,
                                                             int* err) {
    __shared__ unsigned h[kSortMaxBins];
    for (int b = threadIdx.x; b < bins; b += kSortThreads) h[b] = 0;
    __syncthreads();
    const int lo = blockIdx.x * kSortTile, hi = min(n, lo + kSortTile);
    for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) {
        uint32_t k;
        if (tokens) {
            const int t = tokens[i];
            k = (unsigned)t < (unsigned)V ? (uint32_t)t : (uint32_t)V;
            if (k == (uint32_t)V && t != -1) atomicOr(err, kErrBadToken);
        } else {
            k = keys[i];
        }
        atomicAdd(&h[k >> shift & (unsigned)(bins - 1)], 1u);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[(size_t)blockIdx.x * kSortMaxBins + b] = h[b];
}

// Moves each tile's tokens to their places.  A bin's first place is the count
// of all smaller bins plus this bin's count in the tiles before.
__global__ void __launch_bounds__(kSortThreads) k_sort_place(const int32_t* __restrict__ tokens,
                                                             const uint32_t* __restrict__ keys_in,
                                                             const int32_t* __restrict__ pos_in, int n, int V,
                                                             int shift, int bins, const unsigned* __restrict__ hist,
                                                             uint32_t* __restrict__ keys_out,
                                                             int32_t* __restrict__ pos_out) {
    __shared__ unsigned base[kSortMaxBins], total[kSortMaxBins];
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        unsigned before = 0, all = 0;
        for (int t = 0; t < (int)gridDim.x; ++t) {
            const unsigned v = hist[(size_t)t * kSortMaxBins + b];
            if (t < (int)blockIdx.x) before += v;
            all += v;
        }
        base[b] = before;
        total[b] = all;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned run = 0;
        for (int b = 0; b < bins; ++b) {
            base[b] += run;
            run += total[b];
        }
    }
    __syncthreads();
    // one warp walks the tile 32 tokens at a time
    const int lo = blockIdx.x * kSortTile, hi = min(n, lo + kSortTile);
    if (threadIdx.x >= 32) return;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + (int)threadIdx.x;
        const bool in = i < hi;
        uint32_t k = 0;
        int32_t p = 0;
        if (in) {
            if (tokens) {
                const int t = tokens[i];
                k = (unsigned)t < (unsigned)V ? (uint32_t)t : (uint32_t)V;
                p = i;
            } else {
                k = keys_in[i];
                p = pos_in[i];
            }
        }
        const unsigned active = __ballot_sync(0xffffffffu, in);
        if (in) {
            const unsigned d = k >> shift & (unsigned)(bins - 1);
            const unsigned peers = __match_any_sync(active, d);
            const unsigned rank = __popc(peers & ((1u << threadIdx.x) - 1u));
            const unsigned at = base[d] + rank;
            __syncwarp(active);
            if (rank == 0) base[d] += __popc(peers);
            keys_out[at] = k;
            pos_out[at] = p;
        }
        __syncwarp();
    }
}

template <typename G>
__global__ void __launch_bounds__(256) k_zero(G* __restrict__ p, size_t n) {
    for (size_t i = blockIdx.x * (size_t)256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = from_f32<G>(0.f);
}

// One block per sorted place; the first place of a token sums its whole run.
template <typename T, typename G>
__global__ void __launch_bounds__(256) k_sum_runs(const T* __restrict__ dout, long long ld,
                                                  const uint32_t* __restrict__ keys, const int32_t* __restrict__ pos,
                                                  int n, int V, int E, float scale, G* __restrict__ dtable,
                                                  bool accumulate) {
    const int i = blockIdx.x;
    const uint32_t k = keys[i];
    if (k >= (uint32_t)V || (i > 0 && keys[i - 1] == k)) return;
    for (int e = threadIdx.x; e < E; e += 256) {
        float s = 0.f;
        for (int j = i; j < n && keys[j] == k; ++j) s += to_f32(dout[(size_t)pos[j] * ld + e]);
        G* to = dtable + (size_t)k * E + e;
        *to = from_f32<G>(accumulate ? to_f32(*to) + scale * s : scale * s);
    }
}

template <typename T, typename G>
cudaError_t sum_runs(domino_train_ctx* c, const void* dout, long long ld, int n, float scale, void* dtable,
                     bool accumulate, cudaStream_t st) {
    const int V = c->cfg.V, E = c->cfg.E;
    if (!accumulate) {
        k_zero<G><<<c->num_sms * 8, 256, 0, st>>>(static_cast<G*>(dtable), (size_t)V * E);
        c->last_launches += 1;
    }
    if (n > 0) {
        k_sum_runs<T, G><<<n, 256, 0, st>>>(static_cast<const T*>(dout), ld, c->keys[0], c->pos[0], n, V, E, scale,
                                            static_cast<G*>(dtable), accumulate);
        c->last_launches += 1;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(domino_train_ctx* c, const void* table, const int32_t* tokens, int n, float scale, void* out,
                         long long ld, cudaStream_t st) {
    const int V = c->cfg.V, E = c->cfg.E;
    if (c->cfg.dtype == DOMINO_DTYPE_BF16)
        k_embed<<<n, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(table), tokens, n, V, E, scale,
                                   static_cast<__nv_bfloat16*>(out), ld, c->err);
    else
        k_embed<<<n, 256, 0, st>>>(static_cast<const float*>(table), tokens, n, V, E, scale, static_cast<float*>(out),
                                   ld, c->err);
    c->last_launches = 1;
    return cudaGetLastError();
}

cudaError_t launch_embed_grad(domino_train_ctx* c, const void* dout, long long ld, const int32_t* tokens, int n,
                              float scale, void* dtable, int grad_dtype, bool accumulate, cudaStream_t st) {
    const int V = c->cfg.V;
    if (n > 0) {
        int bits = 1;
        while ((V >> bits) != 0) ++bits;  // keys 0..V
        const int digit = (bits + 1) / 2, bins = 1 << digit, tiles = (n + kSortTile - 1) / kSortTile;
        for (int pass = 0; pass < 2; ++pass) {
            const int32_t* tok = pass == 0 ? tokens : nullptr;
            const int from = pass, to = 1 - pass, shift = pass * digit;
            k_sort_count<<<tiles, kSortThreads, 0, st>>>(tok, c->keys[from], n, V, shift, bins, c->hist, c->err);
            k_sort_place<<<tiles, kSortThreads, 0, st>>>(tok, c->keys[from], c->pos[from], n, V, shift, bins, c->hist,
                                                        c->keys[to], c->pos[to]);
            c->last_launches += 2;
        }
    }
    const bool in16 = c->cfg.dtype == DOMINO_DTYPE_BF16, out16 = grad_dtype == DOMINO_DTYPE_BF16;
    if (in16)
        return out16 ? sum_runs<__nv_bfloat16, __nv_bfloat16>(c, dout, ld, n, scale, dtable, accumulate, st)
                     : sum_runs<__nv_bfloat16, float>(c, dout, ld, n, scale, dtable, accumulate, st);
    return out16 ? sum_runs<float, __nv_bfloat16>(c, dout, ld, n, scale, dtable, accumulate, st)
                 : sum_runs<float, float>(c, dout, ld, n, scale, dtable, accumulate, st);
}

}  // namespace train
}  // namespace domino
