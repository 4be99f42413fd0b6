// Streaming of rows of any alignment through a CTA, and cluster helpers.
#pragma once

#include <type_traits>

#include "tc_common.cuh"
#include "train_math.cuh"

namespace domino {
namespace train {

constexpr int kMaxCluster = 16;  // non-portable size

// A slice of a row as whole 16-byte vectors [first, last) of memory and the
// elements beside them; vector i covers the elements 8 i - phase + {0..7} (4 i
// for fp32).
template <typename T>
struct Vectors {
    static constexpr int kPer = 16 / (int)sizeof(T);
    const T* src;
    int n, phase, first, last;
    __device__ Vectors(const T* src_, int n_) : src(src_), n(n_) {
        phase = (int)(reinterpret_cast<uintptr_t>(src) & 15) / (int)sizeof(T);
        first = phase ? 1 : 0;
        last = (phase + n) / kPer;
        if (last < first) last = first;
    }
    __device__ const uint4* vec() const { return reinterpret_cast<const uint4*>(src - phase); }
    // element j of those before the first vector or behind the last: its place, or n
    __device__ int beside(int j) const {
        const int head = min(n, (kPer - phase) % kPer);
        if (j < head) return j;
        const int at = max(head, last * kPer - phase) + (j - head);
        return j - head < kPer && at < n ? at : n;
    }
};

// elements of a row's slice when it is cut into `parts`
constexpr int slice_of(int V, int parts) { return ((V + parts - 1) / parts + 63) / 64 * 64; }

// The vectors [x.first, x.last) of this thread through a ring in shared memory
// that no other thread touches, filled by asynchronous copies kStages calls
// ahead (the first ones by the constructor): the bytes in flight cost no
// registers, and nothing waits on a barrier.  run(f) calls f(i, v, all) with
// kAhead vectors, i, i + kThreads, ...; `all` is a std::true_type where every
// thread has all of them, and v.q is -inf in every element of one past the end
// where it is not (the last call).
//
// kTogether: the vectors of a call are kAhead consecutive ones of each thread,
// from i on, in an order of the lane's own; a warp's copies are one piece of the
// ring and every lane reads what other lanes asked for.
template <int kThreads, int kAhead, int kStages, bool kTogether, typename T>
struct Streamer {
    static constexpr int kCall = kAhead * kThreads;
    static constexpr int kStep = kTogether ? 32 : kThreads;  // between a thread's copies of a call
    static_assert(!kTogether || kAhead == 4, "the order in which a lane reads is without bank conflicts for 4");
    uint4* ring;
    const uint4* src;  // of the next call to be filled
    int i, ahead, vectors, whole, calls, filled, fill_stage;

    __device__ __forceinline__ Streamer(const Vectors<T>& x, uint4* ring_) {
        const int t = (int)threadIdx.x, first = kTogether ? t / 32 * (32 * kAhead) + t % 32 : t;  // copy of a call
        ring = ring_ + first;
        src = x.vec() + x.first + first;
        i = x.first + (kTogether ? t * kAhead : t);
        vectors = x.last - x.first;
        whole = vectors / kCall;
        calls = (vectors + kCall - 1) / kCall;
        filled = fill_stage = 0;
        ahead = first;
#pragma unroll
        for (int g = 0; g < kStages; ++g) fill();
    }
    static __device__ __forceinline__ void copy(uint4* to, const uint4* from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(to)), "l"(from) : "memory");
    }
    __device__ __forceinline__ void fill() {
        uint4* slot = ring + fill_stage * kCall;
        if (filled < whole) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) copy(slot + j * kStep, src + j * kStep);
        } else if (filled < calls) {
            const unsigned inf = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
            const int left = vectors - filled * kCall - ahead;  // of this thread's first on
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (j * kStep < left) copy(slot + j * kStep, src + j * kStep);
                else slot[j * kStep] = make_uint4(inf, inf, inf, inf);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++filled;
        src += kCall;
        fill_stage = fill_stage + 1 == kStages ? 0 : fill_stage + 1;
    }
    template <typename F>
    __device__ __forceinline__ void run(F&& f) {
        int stage = 0;
        const auto take = [&](Vec16<T>* v) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint4* slot = ring + stage * kCall;
            if (kTogether) {
                // eight lanes' reads lie in different banks
                const int lane = (int)threadIdx.x % 32, turn = lane / 2 % 4;
                slot += lane * 3;  // of the warp's piece: lane * kAhead
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kAhead; ++j) v[j].q = slot[j ^ turn];
                __syncwarp();  // before the next copies over them
            } else {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) v[j].q = slot[j * kThreads];
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
        };
#pragma unroll 1
        for (int g = 0; g < whole; ++g, i += kCall) {
            Vec16<T> v[kAhead];
            take(v);
            f(i, v, std::true_type());
            fill();
        }
        if (calls > whole) {
            Vec16<T> v[kAhead];
            take(v);
            f(i, v, std::false_type());
        }
    }
};
template <int kThreads, int kAhead, int kStages, typename T, typename F>
__device__ __forceinline__ void stream(const Vectors<T>& x, uint4* ring, F&& f) {
    Streamer<kThreads, kAhead, kStages, false, T>(x, ring).run(f);
}

// the elements of a vector that `m` names set to -inf
__device__ __forceinline__ void strike(Vec16<float>& v, unsigned m) {
    const unsigned inf = 0xFF800000u;
    if (m & 1u) v.q.x = inf;
    if (m & 2u) v.q.y = inf;
    if (m & 4u) v.q.z = inf;
    if (m & 8u) v.q.w = inf;
}
__device__ __forceinline__ void strike(Vec16<__nv_bfloat16>& v, unsigned m) {
    auto word = [](unsigned w, unsigned two) {
        if (two & 1u) w = (w & 0xFFFF0000u) | 0xFF80u;
        if (two & 2u) w = (w & 0xFFFFu) | 0xFF800000u;
        return w;
    };
    v.q.x = word(v.q.x, m);
    v.q.y = word(v.q.y, m >> 2);
    v.q.z = word(v.q.z, m >> 4);
    v.q.w = word(v.q.w, m >> 6);
}

__device__ __forceinline__ float warp_max(float x) {
    return unord_f32(__reduce_max_sync(0xffffffffu, ord_f32(x)));
}
// All threads of the cluster, whole warps at a time.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A launch in clusters of `size` CTAs.
inline cudaLaunchConfig_t cluster_config(unsigned blocks, int threads, int size, size_t smem, cudaStream_t st,
                                         cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = size;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace train
}  // namespace domino
