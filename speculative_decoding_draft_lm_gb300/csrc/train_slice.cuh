// A row's slice in a CTA's shared memory.
#pragma once

#include "train_stream.cuh"

namespace domino {
namespace train {

// Before a CTA leaves although a wait gave up: what is still on its way into its
// shared memory may land, for 2 ms at most.
static __device__ __noinline__ void last_chance(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = tc::globaltimer();
    while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer() - t0 < 2000000ull) {
    }
}

// The slice of a row that a CTA holds: element i of the row is at data + i - v0,
// at the same place modulo 16 bytes as in memory.
template <typename T>
struct Slice {
    const T* src;   // element v0 of the row
    T* data;        // shared
    uint4* vec;     // the 16-byte vectors that cover it
    int v0, n, nvec;
    int head, body;  // elements before the first whole vector; elements of whole vectors

    __device__ Slice(const T* row, int V, int chunk, int rank, uint8_t* smem) {
        v0 = min(V, rank * chunk);
        n = min(V, v0 + chunk) - v0;
        src = row + v0;
        const int phase = (int)(reinterpret_cast<uintptr_t>(src) & 15);
        vec = reinterpret_cast<uint4*>(smem);
        data = reinterpret_cast<T*>(smem + phase);
        nvec = (phase + n * (int)sizeof(T) + 15) / 16;
        head = min(n, ((16 - phase) & 15) / (int)sizeof(T));
        body = (n - head) / (16 / (int)sizeof(T)) * (16 / (int)sizeof(T));
    }
    // fills what the copies leave of the first and last vectors: the row's own
    // elements, and -inf where there are none
    __device__ void load_edges() const {
        const int first = (int)(data - reinterpret_cast<T*>(vec)), per = 16 / (int)sizeof(T);
        const int t = (int)threadIdx.x;
        if (t < first) reinterpret_cast<T*>(vec)[t] = from_f32<T>(-INFINITY);
        if (t < head) data[t] = src[t];
        const int tail = n - head - body;
        if (t < tail) data[head + body + t] = src[head + body + t];
        const int end = first + n, pad = nvec * per - end;
        if (t < pad) reinterpret_cast<T*>(vec)[end + t] = from_f32<T>(-INFINITY);
    }
};

}  // namespace train
}  // namespace domino
