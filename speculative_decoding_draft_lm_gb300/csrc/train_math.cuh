// Device helpers of the draft-head training operators: exponentials of scaled
// differences, running (maximum, sum) pairs and block reductions.
#pragma once

#include <float.h>

#include "common.cuh"

namespace domino {
namespace train {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x (the hardware's approximation, 2 ulp; results below 2^-126 become 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A set of values v seen through its maximum m and s = sum 2^((v - m) c).
// m starts at -FLT_MAX, not -inf, and never exceeds FLT_MAX, so that v - m is
// a number whenever v is one: -inf adds 0, a row whose every value is the
// type's lowest adds 1 each, +inf makes s infinite, NaN makes it NaN.
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum empty_set() { return {-FLT_MAX, 0.f}; }
__device__ __forceinline__ float clamp_max(float m, float v) { return fminf(fmaxf(m, v), FLT_MAX); }
__device__ __forceinline__ void add(MaxSum& a, float v, float c) {
    if (v > a.m) {
        const float m = clamp_max(a.m, v);
        a.s *= ex2((a.m - m) * c);
        a.m = m;
    }
    a.s += ex2((v - a.m) * c);
}
__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b, float c) {
    MaxSum r;
    r.m = fmaxf(a.m, b.m);
    r.s = a.s * ex2((a.m - r.m) * c) + b.s * ex2((b.m - r.m) * c);
    return r;
}

// ---- two fp32 values in one 64-bit register, one instruction for both -----------
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 halves(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 ex2x2(F2 a) {
    const float2 h = halves(a);
    return f2(ex2(h.x), ex2(h.y));
}

// ---- sixteen bytes of a row --------------------------------------------------------
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
    static constexpr int kElems = 4;
    uint4 q;
    __device__ __forceinline__ F2 pair(int i) const {
        return i == 0 ? f2(__uint_as_float(q.x), __uint_as_float(q.y)) : f2(__uint_as_float(q.z), __uint_as_float(q.w));
    }
    // the largest value; NaN only if all are
    __device__ __forceinline__ float top() const {
        return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
    // the largest value, NaN if any is
    __device__ __forceinline__ float top_nan() const {
        const float a = __uint_as_float(q.x), b = __uint_as_float(q.y), c = __uint_as_float(q.z), d = __uint_as_float(q.w);
        float r;
        asm("{\n .reg .f32 s, t;\n max.NaN.f32 s, %1, %2;\n max.NaN.f32 t, %3, %4;\n max.NaN.f32 %0, s, t;\n}"
            : "=f"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    }
    __device__ __forceinline__ void set(int i, F2 v) {
        const float2 h = halves(v);
        if (i == 0) {
            q.x = __float_as_uint(h.x);
            q.y = __float_as_uint(h.y);
        } else {
            q.z = __float_as_uint(h.x);
            q.w = __float_as_uint(h.y);
        }
    }
};
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int kElems = 8;
    uint4 q;
    __device__ __forceinline__ unsigned word(int i) const { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }
    __device__ __forceinline__ F2 pair(int i) const {
        const unsigned w = word(i);
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    __device__ __forceinline__ float top() const {
        auto h = [](unsigned w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(q.x), h(q.y)), __hmax2(h(q.z), h(q.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ float top_nan() const {
        auto h = [](unsigned w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(q.x), h(q.y)), __hmax2_nan(h(q.z), h(q.w)));
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__low2float(m)), "f"(__high2float(m)));
        return r;
    }
    __device__ __forceinline__ void set(int i, F2 v) {
        const float2 f = halves(v);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        const unsigned w = *reinterpret_cast<const unsigned*>(&b);
        if (i == 0) q.x = w;
        else if (i == 1) q.y = w;
        else if (i == 2) q.z = w;
        else q.w = w;
    }
};

// The largest value of U vectors (NaN only if all are), pairs of 16-bit values
// compared at once.
template <int U>
__device__ __forceinline__ float top_of(const Vec16<float>* v) {
    float m = v[0].top();
#pragma unroll
    for (int j = 1; j < U; ++j) m = fmaxf(m, v[j].top());
    return m;
}
template <int U>
__device__ __forceinline__ float top_of(const Vec16<__nv_bfloat16>* v) {
    auto h = [](unsigned w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m = __hmax2(__hmax2(h(v[0].q.x), h(v[0].q.y)), __hmax2(h(v[0].q.z), h(v[0].q.w)));
#pragma unroll
    for (int j = 1; j < U; ++j)
        m = __hmax2(m, __hmax2(__hmax2(h(v[j].q.x), h(v[j].q.y)), __hmax2(h(v[j].q.z), h(v[j].q.w))));
    return fmaxf(__low2float(m), __high2float(m));
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace train
}  // namespace domino
