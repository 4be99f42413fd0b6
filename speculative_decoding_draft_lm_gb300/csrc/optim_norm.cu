// The norm of the gradients of many tensors, and the factor that clips it.
//
// Every thread adds two or four squares in fp32 and keeps the sum of such sums with what
// its additions round off, and so do warps and CTAs, which meet at the CTA that is done
// last, in an order that the sizes fix.  So the norm is off by two units of 2^-24 at most,
// one of them its own rounding.  (With 16 squares in a plain sum it was off by up to 7, for
// a large element beside small ones, and as fast from 0.5 GB of gradients on.  Every square
// by itself into the sum with its rest took 170 us for the gradients below.)
//
// Bound by HBM: 483 M bf16 gradients, 0.97 GB, in 142.6 us, 6.8 TB/s, the measured copy
// rate (with plain sums of 16: six CTAs an SM instead of eight 3 % more, four 20 %; one
// element a load 1506 us).  The tiny head's 1.2 M fp32 gradients take 5.2 us: the launch,
// the loads, and two small reductions with a counter between them (in fp64 6.6 us).
#include "optim_table.cuh"
#include "train_math.cuh"

namespace domino {
namespace optim {

namespace {

using train::add2;
using train::F2;
using train::f2;
using train::fma2;
using train::halves;
using train::mul2;

constexpr int kE = 16;
static_assert(kThreads * kE == kNormTile, "a tile is one vector of every thread");

// A running sum s with what its additions rounded off, c (an infinite or NaN s: c is
// not looked at).
struct Sum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(s, x), b = __fadd_rn(t, -s);
        c += __fadd_rn(s, -__fadd_rn(t, -b)) + __fadd_rn(x, -b);
        s = t;
    }
    __device__ __forceinline__ void add(float x, float xc) {
        add(x);
        c += xc;
    }
    __device__ __forceinline__ double value() const { return s < INFINITY ? (double)s + (double)c : (double)s; }
};

// The sum over the lanes' sums; lane 0 gets it.
template <int kLanes>
__device__ __forceinline__ Sum warp_sum(Sum a) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        a.add(__shfl_down_sync(0xffffffffu, a.s, o), __shfl_down_sync(0xffffffffu, a.c, o));
    return a;
}
// The sum over a CTA's threads; thread 0 gets it.
__device__ __forceinline__ Sum block_sum(Sum a) {
    __shared__ Sum part[kThreads / 32];
    a = warp_sum<32>(a);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = a;
    __syncthreads();
    if (threadIdx.x < 32) a = warp_sum<kThreads / 32>(threadIdx.x < kThreads / 32 ? part[threadIdx.x] : Sum());
    return a;
}

// A thread's sum of squares with what its additions round off: two of them, in packed
// operations.  Two (fp32) or four (bf16, whose squares are exact) squares are added
// before, with two roundings: 2^-23 of them at most, half of which is the norm's.
struct Squares {
    F2 s = f2(0.f, 0.f), c = f2(0.f, 0.f);
    __device__ __forceinline__ void add(F2 x) {
        const F2 minus = f2(-1.f, -1.f), t = add2(s, x), b = fma2(t, minus, s);  // b: minus what s grew by
        c = add2(c, add2(fma2(add2(t, b), minus, s), add2(x, b)));
        s = t;
    }
    template <typename G>
    __device__ __forceinline__ void add(const uint32_t* w) {
        const auto two = [&](int j) {
            const F2 g = f2(element<G>(w, j), element<G>(w, j + 1)), h = f2(element<G>(w, j + 2), element<G>(w, j + 3));
            return fma2(g, g, mul2(h, h));
        };
        constexpr int kStep = sizeof(G) == 2 ? 8 : 4;
#pragma unroll
        for (int j = 0; j < kE; j += kStep) add(kStep == 8 ? add2(two(j), two(j + 4)) : two(j));
    }
    __device__ __forceinline__ Sum sum() const {
        const float2 hs = halves(s), hc = halves(c);
        Sum r;
        r.s = hs.x;
        r.c = hc.x;
        r.add(hs.y, hc.y);
        return r;
    }
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 8) k_norm(const __grid_constant__ Table<NT> w, NormArgs a) {
    __shared__ bool is_last;
    Squares squares;
    int at = 0;
    pdl_wait();
#pragma unroll 1
    for (unsigned tile = blockIdx.x; tile < w.tiles; tile += gridDim.x) {
        at = find(w, tile, at);
        const Entry& e = w.e[at];
        const long long n = e.n & kElements, i = (long long)(tile - e.tile) * kNormTile + threadIdx.x * kE;
        if (i >= n) continue;
        uint32_t raw[kE];
        if (e.n & kGradBf16) {
            load_elements<__nv_bfloat16, kE>(raw, static_cast<const __nv_bfloat16*>(e.g), i, n);
            squares.template add<__nv_bfloat16>(raw);
        } else {
            load_elements<float, kE>(raw, static_cast<const float*>(e.g), i, n);
            squares.template add<float>(raw);
        }
    }
    Sum sum = block_sum(squares.sum());
    if (threadIdx.x == 0) {
        a.part[a.first + blockIdx.x] = make_float2(sum.s, sum.c);
        __threadfence();
        is_last = atomicInc(a.ticket, a.ctas - 1) == a.ctas - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    sum = Sum();
    for (unsigned i = threadIdx.x; i < a.ctas; i += kThreads) {
        const float2 one = __ldcg(a.part + i);
        sum.add(one.x, one.y);
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum.value());
        *a.norm = (float)norm;
        if (a.scale)
            *a.scale = (float)norm < INFINITY ? (float)fmin(1.0, a.max_norm / (norm + 1e-6))
                                              : __uint_as_float(0x7FC00000u);
    }
}

}  // namespace

unsigned norm_ctas(const domino_adamw_ctx* c, unsigned tiles) {
    const unsigned most = (unsigned)c->num_sms * 8;
    return tiles < most ? tiles : most;
}

cudaError_t launch_norm(const Work& w, const NormArgs& a, unsigned ctas, cudaStream_t st) {
    return of_size(w.tensors, [&](auto nt) {
        constexpr int kTensors = decltype(nt)::value;
        return launch_pdl(k_norm<kTensors>, dim3(ctas), dim3(kThreads), 0, st, table<kTensors>(w), a);
    });
}

}  // namespace optim
}  // namespace domino
