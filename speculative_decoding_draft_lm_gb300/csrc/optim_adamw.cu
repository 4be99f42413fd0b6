// One AdamW step over many tensors, and the norm of their gradients.
//
// Per element, with g' the scaled gradient:
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2,
//   p = p (1 - rate decay) - rate / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
#include "optim_internal.h"

namespace domino {
namespace optim {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = DOMINO_ADAMW_BLOCK;
constexpr float kPerTop = 1.f / 448.f;  // of the largest e4m3 value

template <int NT>
struct Table {
    int tensors;
    unsigned tiles;
    Entry e[NT];
};

// the tensor of a tile: the last entry that does not begin behind it
template <int NT>
__device__ __forceinline__ int find(const Table<NT>& w, unsigned tile) {
    int lo = 0, hi = w.tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (w.e[mid].tile <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ unsigned mix(unsigned h) {
    h = (h ^ (h >> 15)) * 0x6A09E667u;
    h = (h ^ (h >> 13)) * 0xBB67AE85u;
    return h ^ (h >> 16);
}

// The e4m3 code of y in [0, 448] (NaN: 127), rounded up where the 20 random bits
// carry: in normal places the fp32 word's first 11 bits below the sign are the
// code but for the exponents' offset, and below 2^-6 those of y + 2^-6 are.
__device__ __forceinline__ unsigned e4m3_code(float y, unsigned random) {
    const bool low = y < 0.015625f;
    const unsigned w = __float_as_uint(low ? y + 0.015625f : y);
    return y != y ? 127u : ((w + random) >> 20) - (low ? 121u << 3 : 120u << 3);
}
__device__ __forceinline__ float e4m3_value(unsigned code) {
    const unsigned e = code >> 3 & 15u, f = code & 7u;
    float a = e ? __uint_as_float((e + 120u) << 23 | f << 20) : (float)f * 0x1p-9f;
    if ((code & 127u) == 127u) a = __uint_as_float(0x7FC00000u);
    return code & 128u ? -a : a;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

struct Coefficients {
    float scale, decay, rate, root;  // rate: of m; root: of sqrt(v)
    unsigned key;
    bool skip;
};
__device__ __forceinline__ Coefficients coefficients(const AdamArgs& a) {
    Coefficients r;
    const long long t = *a.count + 1;
    const float lr = a.lr * (a.lr_factor ? *a.lr_factor : 1.f), tf = (float)t;
    r.scale = a.scale ? *a.scale : 1.f;
    r.skip = !(fabsf(r.scale) < INFINITY);
    r.decay = 1.f - lr * a.decay;
    r.rate = lr / -expm1f(tf * a.log_beta1);
    r.root = rsqrtf(-expm1f(tf * a.log_beta2));
    r.key = mix(mix((unsigned)t + 0x9E3779B9u) + a.seed);
    return r;
}

// A CTA counts itself done; the last one of the step counts the step.
__device__ __forceinline__ void done(const AdamArgs& a, bool skip) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicInc(a.ticket, gridDim.x - 1) == gridDim.x - 1 && a.last && !skip) ++*a.count;
    }
}

template <int NT, bool kNarrow>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Table<NT> w, AdamArgs a) {
    const Coefficients k = coefficients(a);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (unsigned tile = blockIdx.x; !k.skip && tile < w.tiles; tile += gridDim.x) {
        const Entry& e = w.e[find(w, tile)];
        const long long n = e.n & kElements, at = (long long)e.block * kBlock;
        for (int b = warp; b < kTile / kBlock; b += kThreads / 32) {
            const long long first = (long long)(tile - e.tile) * kTile + b * kBlock;
            if (first >= n) break;
            const long long block = e.block + first / kBlock;
            float m[4], v[4], top_m = 0.f, top_v = 0.f;
            unsigned h[4];
            for (int j = 0; j < 4; ++j) {
                const long long i = first + lane + 32 * j, pos = at + i;
                m[j] = v[j] = 0.f;
                h[j] = mix((unsigned)pos * 0x9E3779B9u + (unsigned)(pos >> 32) * 0x3C6EF373u + k.key);
                if (i >= n) continue;
                const float g = k.scale * (e.n & kGradBf16 ? to_f32(static_cast<const __nv_bfloat16*>(e.g)[i])
                                                           : static_cast<const float*>(e.g)[i]);
                if (kNarrow) {
                    m[j] = e4m3_value(static_cast<const uint8_t*>(a.m)[pos]) * a.m_scale[block];
                    v[j] = e4m3_value(static_cast<const uint8_t*>(a.v)[pos]) * a.v_scale[block];
                } else {
                    m[j] = static_cast<const float*>(a.m)[pos];
                    v[j] = static_cast<const float*>(a.v)[pos];
                }
                m[j] = __fadd_rn(__fmul_rn(a.beta1, m[j]), __fmul_rn(a.rest1, g));
                v[j] = __fadd_rn(__fmul_rn(a.beta2, v[j]), __fmul_rn(__fmul_rn(a.rest2, g), g));
                float p = e.n & kMaster      ? a.master[pos]
                          : e.n & kParamBf16 ? to_f32(static_cast<const __nv_bfloat16*>(e.p)[i])
                                             : static_cast<const float*>(e.p)[i];
                p = p * k.decay - k.rate * (m[j] / (sqrtf(v[j]) * k.root + a.eps));
                if (e.n & kMaster) {
                    a.master[pos] = p;
                    static_cast<__nv_bfloat16*>(e.p)[i] = __float2bfloat16_rn(p);
                } else if (e.n & kParamBf16) {
                    if (fabsf(p) < INFINITY) p = __uint_as_float((__float_as_uint(p) + (h[j] >> 4 & 0xFFFFu)) & 0xFFFF0000u);
                    static_cast<__nv_bfloat16*>(e.p)[i] = __float2bfloat16_rn(p);
                } else {
                    static_cast<float*>(e.p)[i] = p;
                }
                if (!kNarrow) {
                    static_cast<float*>(a.m)[pos] = m[j];
                    static_cast<float*>(a.v)[pos] = v[j];
                }
                top_m = fmaxf(top_m, fabsf(m[j]));
                top_v = fmaxf(top_v, v[j]);
            }
            if (!kNarrow) continue;
            const float sm = fmaxf(warp_max(top_m) * kPerTop, 0x1p-120f), sv = fmaxf(warp_max(top_v) * kPerTop, 0x1p-120f);
            for (int j = 0; j < 4; ++j) {
                const long long i = first + lane + 32 * j, pos = at + i;
                if (i >= n) continue;
                const float ym = fabsf(m[j]) / sm, yv = v[j] / sv;
                unsigned cm = e4m3_code(ym > 448.f ? 448.f : ym, h[j] & 0xFFFFFu);
                unsigned cv = e4m3_code(yv > 448.f ? 448.f : yv, h[j] >> 12);
                if (m[j] < 0.f) cm |= 128u;
                if (v[j] > 0.f && cv == 0) cv = 1;
                static_cast<uint8_t*>(a.m)[pos] = (uint8_t)cm;
                static_cast<uint8_t*>(a.v)[pos] = (uint8_t)cv;
            }
            __syncwarp();
            if (lane == 0) {
                a.m_scale[block] = sm;
                a.v_scale[block] = sv;
            }
        }
    }
    done(a, k.skip);
}

// A running sum s with what its additions rounded off, c.
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(s, x), b = __fadd_rn(t, -s);
        c += __fadd_rn(s, -__fadd_rn(t, -b)) + __fadd_rn(x, -b);
        s = t;
    }
    __device__ __forceinline__ double value() const { return s < INFINITY ? (double)s + (double)c : (double)s; }
};

// The sum over a CTA's threads, in an order of its own; every thread gets it.
__device__ __forceinline__ double block_sum(double s) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    s = 0;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

template <int NT>
__global__ void __launch_bounds__(kThreads) k_norm(const __grid_constant__ Table<NT> w, NormArgs a) {
    __shared__ bool is_last;
    Sum sum;
    for (unsigned tile = blockIdx.x; tile < w.tiles; tile += gridDim.x) {
        const Entry& e = w.e[find(w, tile)];
        const long long n = e.n & kElements;
        for (int j = threadIdx.x; j < kTile; j += kThreads) {
            const long long i = (long long)(tile - e.tile) * kTile + j;
            if (i >= n) break;
            const float g = e.n & kGradBf16 ? to_f32(static_cast<const __nv_bfloat16*>(e.g)[i])
                                            : static_cast<const float*>(e.g)[i];
            sum.add(g * g);
        }
    }
    double s = block_sum(sum.value());
    if (threadIdx.x == 0) {
        a.part[a.first + blockIdx.x] = s;
        __threadfence();
        is_last = atomicInc(a.ticket, a.ctas - 1) == a.ctas - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    s = 0;
    for (unsigned i = threadIdx.x; i < a.ctas; i += kThreads) s += __ldcg(a.part + i);
    s = block_sum(s);
    if (threadIdx.x == 0) {
        const double norm = sqrt(s);
        *a.norm = (float)norm;
        if (a.scale)
            *a.scale = *a.norm < INFINITY ? (float)fmin(1.0, a.max_norm / (norm + 1e-6)) : __uint_as_float(0x7FC00000u);
    }
}

template <int NT>
Table<NT> table(const Work& w) {
    Table<NT> t;
    t.tensors = w.tensors;
    t.tiles = w.tiles;
    for (int i = 0; i < w.tensors; ++i) t.e[i] = w.entry[i];
    return t;
}

template <int NT>
cudaError_t launch_adamw_of(domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    const unsigned most = (unsigned)c->num_sms * 4, grid = w.tiles < 1 ? 1 : w.tiles < most ? w.tiles : most;
    if (c->cfg.state_bits == 8) k_adamw<NT, true><<<grid, kThreads, 0, st>>>(table<NT>(w), a);
    else k_adamw<NT, false><<<grid, kThreads, 0, st>>>(table<NT>(w), a);
    return cudaGetLastError();
}

template <int NT>
cudaError_t launch_norm_of(const Work& w, const NormArgs& a, unsigned ctas, cudaStream_t st) {
    k_norm<NT><<<ctas, kThreads, 0, st>>>(table<NT>(w), a);
    return cudaGetLastError();
}

constexpr int kSmall = 16, kMedium = 100;  // tensors: parameters of 0.5 KB, and of less than 4 KB

}  // namespace

unsigned norm_ctas(const domino_adamw_ctx* c, unsigned tiles) {
    const unsigned most = (unsigned)c->num_sms * 4;
    return tiles < most ? tiles : most;
}

cudaError_t launch_adamw(domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    if (w.tensors <= kSmall) return launch_adamw_of<kSmall>(c, w, a, st);
    if (w.tensors <= kMedium) return launch_adamw_of<kMedium>(c, w, a, st);
    return launch_adamw_of<kMaxPerLaunch>(c, w, a, st);
}

cudaError_t launch_norm(domino_adamw_ctx* c, const Work& w, const NormArgs& a, unsigned ctas, cudaStream_t st) {
    if (w.tensors <= kSmall) return launch_norm_of<kSmall>(w, a, ctas, st);
    if (w.tensors <= kMedium) return launch_norm_of<kMedium>(w, a, ctas, st);
    return launch_norm_of<kMaxPerLaunch>(w, a, ctas, st);
}

}  // namespace optim
}  // namespace domino
