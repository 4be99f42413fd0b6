// The tensors of a launch in the kernels' parameters, and vectors of their elements.
#pragma once

#include <type_traits>

#include "optim_internal.h"

namespace domino {
namespace optim {

constexpr int kThreads = 256;

// calls f(std::integral_constant of a table's size) with the smallest that holds so
// many tensors: parameters of 1, 4, 10 and 32 KB (a norm of 100 tensors takes 8 us in
// calls after one another, of 200 11.5, of 321 17)
template <typename F>
cudaError_t of_size(int tensors, F&& f) {
    if (tensors <= 32) return f(std::integral_constant<int, 32>());
    if (tensors <= 120) return f(std::integral_constant<int, 120>());
    if (tensors <= 320) return f(std::integral_constant<int, 320>());
    return f(std::integral_constant<int, kMaxPerLaunch>());
}

template <int NT>
struct Table {
    int tensors;
    unsigned tiles;
    Entry e[NT];
};
template <int NT>
Table<NT> table(const Work& w) {
    Table<NT> t;
    t.tensors = w.tensors;
    t.tiles = w.tiles;
    for (int i = 0; i < w.tensors; ++i) t.e[i] = w.entry[i];
    return t;
}

// the tensor of a tile, from entry `lo` on: the last one that does not begin behind it
template <int NT>
__device__ __forceinline__ int find(const Table<NT>& w, unsigned tile, int lo) {
    int hi = w.tensors;
    if (lo + 1 >= hi || w.e[lo + 1].tile > tile) return lo;  // mostly that of the CTA's last tile
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (w.e[mid].tile <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

// kWords 32-bit words in a row, 16 or 32 bytes a load (`wide`: on a 32-byte boundary, else on a 16-byte one)
template <int kWords>
__device__ __forceinline__ void load_words(uint32_t* w, const void* from, bool wide) {
    const char* a = static_cast<const char*>(from);
    if (kWords >= 8 && wide) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                           "=r"(w[i + 6]), "=r"(w[i + 7])
                         : "l"(a + 4 * i));
    } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "l"(a + 4 * i));
    }
}
template <int kWords>
__device__ __forceinline__ void store_words(void* to, const uint32_t* w, bool wide) {
    char* a = static_cast<char*>(to);
    if (kWords >= 8 && wide) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a + 4 * i), "r"(w[i]),
                         "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                         "r"(w[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(a + 4 * i), "r"(w[i]), "r"(w[i + 1]),
                         "r"(w[i + 2]), "r"(w[i + 3])
                         : "memory");
    }
}

// kE elements of a tensor of 2- or 4-byte elements from i on, as they lie in memory; 0 for those from n on.
template <typename T, int kE>
__device__ __forceinline__ void load_elements(uint32_t* w, const T* a, long long i, long long n) {
    constexpr int kWords = kE * (int)sizeof(T) / 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a);
    if ((at & 15) == 0 && i + kE <= n) {
        load_words<kWords>(w, a + i, (at & 31) == 0);
        return;
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0;
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        if (i + j >= n) continue;
        if (sizeof(T) == 4) w[j] = reinterpret_cast<const uint32_t*>(a)[i + j];
        else w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(a)[i + j] << (j % 2 * 16);
    }
}
template <typename T, int kE>
__device__ __forceinline__ void store_elements(T* a, long long i, long long n, const uint32_t* w) {
    constexpr int kWords = kE * (int)sizeof(T) / 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a);
    if ((at & 15) == 0 && i + kE <= n) {
        store_words<kWords>(a + i, w, (at & 31) == 0);
        return;
    }
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        if (i + j >= n) continue;
        if (sizeof(T) == 4) reinterpret_cast<uint32_t*>(a)[i + j] = w[j];
        else reinterpret_cast<uint16_t*>(a)[i + j] = (uint16_t)(w[j / 2] >> (j % 2 * 16));
    }
}

// element j of such words as fp32
template <typename T>
__device__ __forceinline__ float element(const uint32_t* w, int j);
template <>
__device__ __forceinline__ float element<float>(const uint32_t* w, int j) {
    return __uint_as_float(w[j]);
}
template <>
__device__ __forceinline__ float element<__nv_bfloat16>(const uint32_t* w, int j) {
    return __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
}

}  // namespace optim
}  // namespace domino
