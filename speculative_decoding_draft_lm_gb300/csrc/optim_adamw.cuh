// One AdamW step over many tensors.
//
// Per element, with g' the scaled gradient:
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2,
//   p = p (1 - rate decay) - rate / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps).
// m and v are formed with every product and sum rounded by itself.  What is taken from
// p is formed by itself too, decay and update together, and subtracted once:
//   p = p - c (m / (..) + decay (1 - b1^t) p),   c = rate / (1 - b1^t).
// A factor 1 - rate decay would hold the decay to 2^-25 only: at a rate of 1e-6 and a
// decay of 0.01 it is 1, at 3e-6 it decays 2.6 times too fast.
#pragma once

#include "optim_table.cuh"
#include "train_math.cuh"

namespace domino {
namespace optim {

using train::F2;
using train::f2;
using train::fma2;
using train::halves;
using train::mul2;

constexpr int kBlock = DOMINO_ADAMW_BLOCK;

__device__ __forceinline__ F2 both(float x) { return f2(x, x); }
__device__ __forceinline__ F2 both(float2 x) { return f2(x.x, x.y); }

// The new moments, every product and sum rounded by itself.  The sums are written
// as fma with a factor of 1 that the compiler does not know (AdamArgs::one): a
// packed product and the packed sum behind it would become one fma, rounded once.
__device__ __forceinline__ F2 new_m(const AdamArgs& a, F2 m, F2 g) {
    return fma2(mul2(both(a.beta1), m), both(a.one), mul2(both(a.rest1), g));
}
__device__ __forceinline__ F2 new_v(const AdamArgs& a, F2 v, F2 g) {
    return fma2(mul2(both(a.beta2), v), both(a.one), mul2(mul2(both(a.rest2), g), g));
}
__device__ __forceinline__ float sqrt_fast(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the largest magnitude, NaN if any is
__device__ __forceinline__ float top_nan(float top, F2 v) {
    const float2 h = halves(v);
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top), "f"(fabsf(h.x)), "f"(fabsf(h.y)));
    return r;
}

__device__ __forceinline__ unsigned mix(unsigned h) {
    h = (h ^ (h >> 15)) * 0x6A09E667u;
    h = (h ^ (h >> 13)) * 0xBB67AE85u;
    return h ^ (h >> 16);
}

// The random word of the j-th position behind that whose sum is h0.  The factor is
// one that the compiler does not know (AdamArgs::golden), so that a multiplier forms
// the sum: the pipe of integer sums and logic is what these kernels wait for.
__device__ __forceinline__ unsigned word_of(const AdamArgs& a, unsigned h0, int j) {
    return mix(h0 + (unsigned)j * a.golden);
}

struct Coefficients {
    float scale, decay, rate, root;  // rate: of what is taken from p; decay: of p in it; root: of sqrt(v)
    unsigned key;
    bool skip;
};
__device__ __forceinline__ Coefficients coefficients(const AdamArgs& a) {
    Coefficients r;
    const long long t = *a.count + 1;
    const float lr = a.lr * (a.lr_factor ? *a.lr_factor : 1.f), tf = (float)t;
    r.scale = a.scale ? *a.scale : 1.f;
    r.skip = !(fabsf(r.scale) < INFINITY);
    const float seen = -expm1f(tf * a.log_beta1);
    r.decay = a.decay * seen;
    r.rate = lr / seen;
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

// two bf16 in a word from two fp32 words' upper halves
__device__ __forceinline__ uint32_t upper(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }
__device__ __forceinline__ uint32_t nearest(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// ---- e4m3 ------------------------------------------------------------------------

// two e4m3 codes, in a word's low or high half, as fp32
__device__ __forceinline__ F2 e4m3_values(uint32_t codes, bool high) {
    uint32_t h;
    if (high) asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, u;\n}" : "=r"(h) : "r"(codes));
    else asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(h) : "r"(codes));
    F2 r;
    asm("{\n .reg .b16 l, u;\n .reg .f32 a, b;\n mov.b32 {l, u}, %1;\n cvt.f32.f16 a, l;\n cvt.f32.f16 b, u;\n"
        " mov.b64 %0, {a, b};\n}"
        : "=l"(r.v)
        : "r"(h));
    return r;
}

// A block's scale and its reciprocal.
struct Scale {
    float s, inv;
};
__device__ __forceinline__ Scale scale_of(float top) {
    Scale r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r.s) : "f"(top * (1.f / 448.f)), "f"(0x1p-120f));
    r.inv = 1.f / r.s;
    return r;
}

// The fp32 words of a / s 2^-120.  From the rounded reciprocal one residual gives
// the rounded quotient (P. Markstein's division).  On the scale of 2^-120 an e4m3
// number's exponent field is fp32's, and its subnormals are fp32's: bits 20 to 26
// of the word are the code of the next e4m3 number towards zero, and the 20 bits
// below are the place between it and the one behind.
__device__ __forceinline__ uint2 places(F2 a, F2 inv, F2 minus_s) {
    const F2 q = mul2(a, inv);
    const F2 y = mul2(fma2(fma2(q, minus_s, a), inv, q), both(0x1p-120f));
    const float2 h = halves(y);
    return make_uint2(__float_as_uint(h.x), __float_as_uint(h.y));
}

// what the kinds of a launch's tensors are
template <typename P_, bool kMaster_, typename G_>
struct Kind {
    typedef P_ P;
    typedef G_ G;
    static constexpr bool kMaster = kMaster_;
    // the parameter is rounded stochastically
    static constexpr bool kLossy = sizeof(P) == 2 && !kMaster;
    static constexpr int kFrom = kMaster ? 4 : (int)sizeof(P);  // bytes of an element of what is updated
};

// two of the parameters that the step starts from
template <typename K>
__device__ __forceinline__ F2 before(const uint32_t* w, int j) {
    if (K::kFrom == 4) return f2(element<float>(w, 2 * j), element<float>(w, 2 * j + 1));
    return f2(element<typename K::P>(w, 2 * j), element<typename K::P>(w, 2 * j + 1));
}

// p after the step, from the new m and v
__device__ __forceinline__ F2 updated(const AdamArgs& a, const Coefficients& k, F2 p, F2 m, F2 v) {
    const float2 vf = halves(v);
    const float2 d = halves(fma2(f2(sqrt_fast(vf.x), sqrt_fast(vf.y)), both(k.root), both(a.eps)));
    return fma2(both(-k.rate), fma2(p, both(k.decay), mul2(m, f2(rcp_fast(d.x), rcp_fast(d.y)))), p);
}
// The word of what an element p becomes that `updated` makes NaN: an infinite one minus its
// infinite decay stays as it is, as long as m and v are finite.
__device__ __forceinline__ uint32_t of_nan(float p, float m, float v) {
    return fabsf(p) == INFINITY && fabsf(m) < INFINITY && v < INFINITY ? __float_as_uint(p) : 0x7FC00000u;
}

// Two fp32 values rounded to bf16, up where the 16 lower bits and the random ones
// carry.  Not for NaN, whose bits may all be set: the carry would reach the sign.
__device__ __forceinline__ uint32_t lossy(float2 q, unsigned r0_up12, unsigned r1_up12) {
    return upper(__float_as_uint(q.x) + (r0_up12 >> 16), __float_as_uint(q.y) + (r1_up12 >> 16));
}
// the fp32 number of the word x, NaN or infinite, as element j of the words w
template <typename K>
__device__ __forceinline__ void set_word(uint32_t* w, int j, uint32_t x) {
    if (K::kLossy) w[j / 2] = (w[j / 2] & (j % 2 ? 0xFFFFu : 0xFFFF0000u)) | x >> 16 << (j % 2 * 16);
    else w[j] = x;
}

// a thread's new parameters to memory, the exact ones too where they are held
template <typename K, int kE>
__device__ __forceinline__ void store_param(const Entry& e, float* master, long long pos, long long i, long long n,
                                            const uint32_t* w) {
    typedef typename K::P P;
    if (K::kMaster) {
        store_elements<float, kE>(master + (pos - i), i, n, w);
        uint32_t b[kE / 2];
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) b[j] = nearest(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        store_elements<P, kE>(static_cast<P*>(e.p), i, n, b);
    } else {
        store_elements<P, kE>(static_cast<P*>(e.p), i, n, w);
    }
}

// calls f(std::integral_constant of the table's size, Kind) for a launch
template <typename F>
cudaError_t of_kind(const Work& w, F&& f) {
    const auto sized = [&](auto kind) { return of_size(w.tensors, [&](auto nt) { return f(nt, kind); }); };
    const auto of = [&](auto grad) {
        typedef decltype(grad) G;
        if (w.kind & kMaster) return sized(Kind<__nv_bfloat16, true, G>());
        return w.kind & kParamBf16 ? sized(Kind<__nv_bfloat16, false, G>()) : sized(Kind<float, false, G>());
    };
    return w.kind & kGradBf16 ? of(__nv_bfloat16()) : of(float());
}

}  // namespace optim
}  // namespace domino
