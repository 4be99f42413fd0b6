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

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace train
}  // namespace domino
