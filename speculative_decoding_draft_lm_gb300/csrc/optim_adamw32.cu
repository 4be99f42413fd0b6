// AdamW with moments in fp32.
//
// A thread has 8 consecutive elements, 32 bytes of fp32 or 16 of bf16 a load; each is
// read and written once.  Bound by HBM: 319 M bf16 parameters with a master copy, 28
// bytes an element, 8.9 GB, in 1270 us, 7.0 TB/s, a little above the measured copy rate.
//
// Tiles go to the CTAs in up to 400 shares an SM, two or three tiles a CTA here: CTAs that
// take many tiles in turn drift apart and with them the places of memory that are open at
// one time (4 shares an SM, the resident CTAs', 1409 us, 30 1314, 100 1294, 150 1285, a
// CTA a tile 1274).  One element a load, a warp a block of 128: 2790 us.
#include "optim_adamw.cuh"

namespace domino {
namespace optim {

namespace {

constexpr int kE = 8;
static_assert(kThreads * kE == kTile32, "a tile is one vector of every thread");

template <int NT, typename K>
__global__ void __launch_bounds__(kThreads, 4) k_adamw32(const __grid_constant__ Table<NT> w, AdamArgs a) {
    typedef typename K::P P;
    typedef typename K::G G;
    pdl_wait();
    const Coefficients k = coefficients(a);
    int at = 0;
    for (unsigned tile = blockIdx.x; !k.skip && tile < w.tiles; tile += gridDim.x) {
        at = find(w, tile, at);
        const Entry& e = w.e[at];
        const long long n = e.n & kElements, i = (long long)(tile - e.tile) * kTile32 + threadIdx.x * kE;
        const long long pos = (long long)e.block * kBlock + i;
        if (i >= n) continue;
        float* const m32 = static_cast<float*>(a.m) + (pos - i);
        float* const v32 = static_cast<float*>(a.v) + (pos - i);
        uint32_t rg[kE * sizeof(G) / 4], rp[kE * K::kFrom / 4], rq[kE * K::kFrom / 4], rm[kE], rv[kE];
        float top_p = 0.f;
        load_elements<G, kE>(rg, static_cast<const G*>(e.g), i, n);
        if (K::kMaster) load_elements<float, kE>(rp, a.master + (pos - i), i, n);
        else load_elements<P, kE>(rp, static_cast<const P*>(e.p), i, n);
        load_elements<float, kE>(rm, m32, i, n);
        load_elements<float, kE>(rv, v32, i, n);
        const unsigned h0 = (unsigned)pos * 0x9E3779B9u + (unsigned)(pos >> 32) * 0x3C6EF373u + k.key;
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) {
            const F2 g = mul2(f2(element<G>(rg, 2 * j), element<G>(rg, 2 * j + 1)), both(k.scale));
            const F2 m = new_m(a, f2(element<float>(rm, 2 * j), element<float>(rm, 2 * j + 1)), g);
            const F2 v = new_v(a, f2(element<float>(rv, 2 * j), element<float>(rv, 2 * j + 1)), g);
            const F2 q = updated(a, k, before<K>(rp, j), m, v);
            const float2 mf = halves(m), vf = halves(v), qf = halves(q);
            rm[2 * j] = __float_as_uint(mf.x);
            rm[2 * j + 1] = __float_as_uint(mf.y);
            rv[2 * j] = __float_as_uint(vf.x);
            rv[2 * j + 1] = __float_as_uint(vf.y);
            top_p = top_nan(top_p, q);
            if (K::kLossy) {
                rq[j] = lossy(qf, word_of(a, h0, 2 * j) << 12, word_of(a, h0, 2 * j + 1) << 12);
            } else {
                rq[2 * j] = __float_as_uint(qf.x);
                rq[2 * j + 1] = __float_as_uint(qf.y);
            }
        }
        if (top_p != top_p) {
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const float2 ps = halves(before<K>(rp, j / 2));
                const float p = j % 2 ? ps.y : ps.x, m = element<float>(rm, j), v = element<float>(rv, j);
                const float q = halves(updated(a, k, both(p), both(m), both(v))).x;
                if (q != q) set_word<K>(rq, j, of_nan(p, m, v));
            }
        }
        store_param<K, kE>(e, a.master, pos, i, n, rq);
        store_elements<float, kE>(m32, i, n, rm);
        store_elements<float, kE>(v32, i, n, rv);
    }
    done(a, k.skip);
}

template <int NT, typename K>
cudaError_t launch_kind(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    const unsigned most = (unsigned)c->num_sms * 400;
    return launch_pdl(k_adamw32<NT, K>, dim3(w.tiles < 1 ? 1 : w.tiles < most ? w.tiles : most), dim3(kThreads), 0, st,
                      table<NT>(w), a);
}

}  // namespace

cudaError_t launch_adamw32(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    return of_kind(
        w, [&](auto nt, auto kind) { return launch_kind<decltype(nt)::value, decltype(kind)>(c, w, a, st); });
}

}  // namespace optim
}  // namespace domino
