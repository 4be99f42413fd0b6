// AdamW with moments in e4m3, a scale for every 128 of them.
//
// A thread has 16 consecutive elements, eight threads a block: the largest
// magnitudes of a block meet by shuffles, so each element is read and written once.
//
// At 10 bytes an element (bf16) the instructions weigh as much as the bytes: 54 an
// element, which alone would take 470 us for 319 M elements where the bytes take 475
// at the measured copy rate.  They take 562 us, 5.7 TB/s, 0.85 of that rate.  What
// brought it there, in us: one element a load, branches in the conversions 4949;
// vectors, codes by integer places 839; constants in pairs, no branch an element 726;
// the ends of the codes' range looked at once a thread 657; the parameter's update
// behind the block's maxima, so that a random word is used as soon as it is formed
// and four CTAs fit an SM, 572 (three: 605, five: 688 with spills); nothing held over a
// thread's four words of codes for what is rare (their ends, NaN) 562.
//
// Tiles go to the CTAs in 30 shares an SM: with one share a resident CTA the SMs end
// apart (654 against 632 when that was measured).  Prefetches of the next tile into L2,
// threads by 128 or the random words' shifts as upper halves of products gained nothing.
// A ring of asynchronous copies a tile ahead took 593: the issue slots were as full as
// without it, with more instructions to issue.
#include "optim_adamw.cuh"

namespace domino {
namespace optim {

namespace {

constexpr int kThreads8 = kTile8 / 16, kE = 16, kLanes = kBlock / kE;
static_assert(kThreads8 * kE == kTile8, "a tile is one vector of every thread");

// Four codes in the bytes of a word, from words of places with their random bits
// added: the code is in bits 20 to 26.  The halves are shifted by products, which the
// pipe of shifts and logic does not take.
__device__ __forceinline__ uint32_t codes(const uint32_t* x, uint32_t* signs) {
    const uint32_t a = upper(x[0], x[1]), b = upper(x[2], x[3]);
    *signs = __byte_perm(a, b, 0x7531);
    return __byte_perm(a * 16u, b * 16u, 0x7531);
}
constexpr uint32_t kOnes = 0x01010101u, kTops = 0x80808080u;

// CTAs an SM: as many as leave the raw elements in registers, none of them spilled
template <typename K>
constexpr int kPerSm = K::kFrom == 2 && sizeof(typename K::G) == 2 ? 4 : 3;

template <int NT, typename K>
__global__ void __launch_bounds__(kThreads8, kPerSm<K>) k_adamw8(const __grid_constant__ Table<NT> w, AdamArgs a) {
    typedef typename K::P P;
    typedef typename K::G G;
    pdl_wait();
    const Coefficients k = coefficients(a);
    int at = 0;
    for (unsigned tile = blockIdx.x; !k.skip && tile < w.tiles; tile += gridDim.x) {
        at = find(w, tile, at);
        const Entry& e = w.e[at];
        const long long n = e.n & kElements, i = (long long)(tile - e.tile) * kTile8 + threadIdx.x * kE;
        const long long block = (long long)e.block + i / kBlock, pos = (long long)e.block * kBlock + i;
        uint32_t rg[kE * sizeof(G) / 4], rp[kE * K::kFrom / 4], rm[4], rv[4];
        load_elements<G, kE>(rg, static_cast<const G*>(e.g), i, n);
        if (K::kMaster) load_elements<float, kE>(rp, a.master + (pos - i), i, n);
        else load_elements<P, kE>(rp, static_cast<const P*>(e.p), i, n);
        uint8_t* const m8 = static_cast<uint8_t*>(a.m) + pos;
        uint8_t* const v8 = static_cast<uint8_t*>(a.v) + pos;
        float sm = 0.f, sv = 0.f;
        if (i + kE <= n) {
            load_words<4>(rm, m8, false);
            load_words<4>(rv, v8, false);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) rm[j] = rv[j] = 0;
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                if (i + j >= n) continue;
                rm[j / 4] |= (uint32_t)m8[j] << (j % 4 * 8);
                rv[j / 4] |= (uint32_t)v8[j] << (j % 4 * 8);
            }
        }
        if (i < n) {
            sm = a.m_scale[block];
            sv = a.v_scale[block];
        }
        const unsigned h0 = (unsigned)pos * 0x9E3779B9u + (unsigned)(pos >> 32) * 0x3C6EF373u + k.key;
        F2 m[kE / 2], v[kE / 2];
        float top_m = 0.f, top_v = 0.f, top_p = 0.f;
#pragma unroll
        for (int j = 0; j < kE / 2; ++j) {
            const F2 g = mul2(f2(element<G>(rg, 2 * j), element<G>(rg, 2 * j + 1)), both(k.scale));
            m[j] = new_m(a, mul2(e4m3_values(rm[j / 2], j % 2), both(sm)), g);
            v[j] = new_v(a, mul2(e4m3_values(rv[j / 2], j % 2), both(sv)), g);
            top_m = top_nan(top_m, m[j]);
            top_v = top_nan(top_v, v[j]);
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, top_m, o), ov = __shfl_xor_sync(0xffffffffu, top_v, o);
            top_m = top_nan(top_m, f2(om, om));
            top_v = top_nan(top_v, f2(ov, ov));
        }
        const Scale zm = scale_of(top_m), zv = scale_of(top_v);
        // everything that takes an element's random word, so that it need not be held
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t xm[4], xv[4], signs, none;
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                const int at2 = 2 * j + l;
                const unsigned r0 = word_of(a, h0, 2 * at2), r1 = word_of(a, h0, 2 * at2 + 1);
                const unsigned u0 = r0 * a.up12, u1 = r1 * a.up12;
                const F2 q = updated(a, k, before<K>(rp, at2), m[at2], v[at2]);
                const float2 qf = halves(q);
                top_p = top_nan(top_p, q);
                if (K::kLossy) {
                    rp[at2] = lossy(qf, u0, u1);
                } else {
                    rp[2 * at2] = __float_as_uint(qf.x);
                    rp[2 * at2 + 1] = __float_as_uint(qf.y);
                }
                const uint2 ym = places(m[at2], both(zm.inv), both(-zm.s));
                const uint2 yv = places(v[at2], both(zv.inv), both(-zv.s));
                xm[2 * l] = ym.x + (u0 >> 12);
                xm[2 * l + 1] = ym.y + (u1 >> 12);
                xv[2 * l] = yv.x + (r0 >> 12);
                xv[2 * l + 1] = yv.y + (r1 >> 12);
            }
            const uint32_t cm = codes(xm, &signs);
            rv[j] = codes(xv, &none);
            rm[j] = cm | (signs & kTops);
            if (((cm + kOnes) | (rv[j] + kOnes) | (rv[j] - kOnes)) & kTops) {  // a code of 127 or, of v, of 0
                // a quotient by a rounded scale can pass the largest number, 126, by its last bits;
                // and a v that is not 0 does not become 0
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const float2 vf = halves(v[2 * j + l / 2]);
                    const uint32_t one = 1u << (l * 8);
                    if ((rm[j] & 0x7Fu * one) == 0x7Fu * one) rm[j] -= one;
                    if ((rv[j] & 0x7Fu * one) == 0x7Fu * one) rv[j] -= one;
                    if ((l % 2 ? vf.y : vf.x) != 0.f && !(rv[j] & 0x7Fu * one)) rv[j] |= one;
                }
            }
        }
        if (top_p != top_p) {
            // each element from memory once more, so that no register is held for this (from registers, and with the
            // codes' fix behind all of them, 92 bytes a thread were spilled)
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                if (i + j >= n) continue;
                const F2 g = mul2(both(to_f32(static_cast<const G*>(e.g)[i + j])), both(k.scale));
                const F2 m1 = new_m(a, mul2(e4m3_values(m8[j], false), both(sm)), g);
                const F2 v1 = new_v(a, mul2(e4m3_values(v8[j], false), both(sv)), g);
                const float p = K::kMaster ? a.master[pos + j] : to_f32(static_cast<const P*>(e.p)[i + j]);
                const float q = halves(updated(a, k, both(p), m1, v1)).x;
                if (q != q) set_word<K>(rp, j, of_nan(p, halves(m1).x, halves(v1).x));
            }
        }
        store_param<K, kE>(e, a.master, pos, i, n, rp);
        if (i + kE <= n) {
            store_words<4>(m8, rm, false);
            store_words<4>(v8, rv, false);
        } else {
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                if (i + j >= n) continue;
                m8[j] = (uint8_t)(rm[j / 4] >> (j % 4 * 8));
                v8[j] = (uint8_t)(rv[j / 4] >> (j % 4 * 8));
            }
        }
        if (threadIdx.x % kLanes == 0 && i < n) {
            a.m_scale[block] = zm.s;
            a.v_scale[block] = zv.s;
        }
    }
    done(a, k.skip);
}

template <int NT, typename K>
cudaError_t launch_kind(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    const unsigned most = (unsigned)c->num_sms * 30;
    return launch_pdl(k_adamw8<NT, K>, dim3(w.tiles < 1 ? 1 : w.tiles < most ? w.tiles : most), dim3(kThreads8), 0, st,
                      table<NT>(w), a);
}

}  // namespace

cudaError_t launch_adamw8(const domino_adamw_ctx* c, const Work& w, const AdamArgs& a, cudaStream_t st) {
    return of_kind(
        w, [&](auto nt, auto kind) { return launch_kind<decltype(nt)::value, decltype(kind)>(c, w, a, st); });
}

}  // namespace optim
}  // namespace domino
