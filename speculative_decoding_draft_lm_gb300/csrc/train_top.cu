// Record of a teacher's logits: the K largest of each row, ids ascending, and
// the log-sum-exp of all the others.
//
// Order: (logit descending, id ascending), with NaN above everything and the
// two zeros equal.  A radix select over the 32-bit orderable keys finds the
// K-th largest key; of the ids that share it the lowest are taken.  The rest is
// summed over the ids that were not taken, never as a difference: a peaked
// teacher leaves less in it than the rounding of the whole.
#include "train_internal.h"
#include "train_math.cuh"

namespace domino {
namespace train {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ unsigned top_key(float x) { return x != x ? 0xFFFFFFFFu : ord_f32(x); }

// Exclusive scan of one value per thread; *total gets the sum.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned* warp_tot, unsigned* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned incl = x;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    unsigned before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_tot[w];
        all += warp_tot[w];
    }
    __syncthreads();
    *total = all;
    return before + incl - x;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_top(const T* __restrict__ logits, long long ld, int V, int K,
                                                  float temperature, int32_t* __restrict__ ids,
                                                  float* __restrict__ top, float* __restrict__ rest) {
    __shared__ unsigned hist[256], warp_tot[kWarps];
    __shared__ unsigned s_digit, s_need;
    __shared__ MaxSum part[kWarps];
    const int n = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* x = logits + (size_t)n * ld;
    const float c = kLog2e / temperature;
    // the K-th largest key, one byte a pass
    unsigned prefix = 0, mask = 0, need = (unsigned)K;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const unsigned k = top_key(to_f32(x[v]));
            if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned above = 0;
            int d = 255;
            while (above + hist[d] < need) above += hist[d--];
            s_digit = (unsigned)d;
            s_need = need - above;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= 255u << shift;
        need = s_need;
    }
    // in the order of the ids: all keys above `prefix`, the first `need` equal to it; the others into the rest
    MaxSum r = empty_set();
    unsigned done = 0, ties = 0, total;
    for (int v0 = 0; v0 < V; v0 += kThreads) {
        const int v = v0 + threadIdx.x;
        const float f = v < V ? to_f32(x[v]) : 0.f;
        const unsigned k = v < V ? top_key(f) : 0u;
        const bool eq = v < V && k == prefix, gt = v < V && k > prefix;
        const unsigned t = ties + block_scan(eq, warp_tot, &total);
        ties += total;
        const bool take = gt || (eq && t < need);
        const unsigned at = done + block_scan(take, warp_tot, &total);
        done += total;
        if (take) {
            ids[(size_t)n * K + at] = v;
            top[(size_t)n * K + at] = f;
        } else if (v < V) {
            add(r, f, c);
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const MaxSum other = {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o)};
        r = join(r, other, c);
    }
    if (lane == 0) part[warp] = r;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) r = join(r, part[w], c);
        rest[n] = r.s == 0.f ? -INFINITY : r.m / temperature + logf(r.s);
    }
}

}  // namespace

cudaError_t launch_top(domino_train_ctx* c, const void* x, int dtype, long long ld, int n, int K, float temperature,
                       int32_t* ids, float* top, float* rest, cudaStream_t st) {
    const int V = c->cfg.V;
    if (dtype == DOMINO_DTYPE_BF16)
        k_top<<<n, kThreads, 0, st>>>(static_cast<const __nv_bfloat16*>(x), ld, V, K, temperature, ids, top, rest);
    else
        k_top<<<n, kThreads, 0, st>>>(static_cast<const float*>(x), ld, V, K, temperature, ids, top, rest);
    c->last_launches = 1;
    return cudaGetLastError();
}

}  // namespace train
}  // namespace domino
