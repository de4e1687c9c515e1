// norm_rotate.cuh -- what the norm and rotation of queries and keys share with their gradients: how a
// row lies in a group of lanes, a token's angles, the scale of a row.
//
//   xh = x s,  s = 1 / sqrt(c sum(x^2) + eps)  (c = 1/d: rms, c = 1: unit length; s = 1 without a norm)
//   u = xh * weight,   y = u with each rotated pair (u_a, u_b) turned by position * freq of its pair
//
// A group of LPR lanes takes a token and goes through a range of the heads of q or of k, so that the sines
// are computed once for all of them.  A lane holds CP pairs of chunks of VEC values, chosen so that both
// values of a rotated pair are in it: with pairs (e, e + r) ("halves", r pairs) the chunks at VEC c and
// r + VEC c, and neighbours behind the 2 r rotated values; with pairs (2 e, 2 e + 1) ("adjacent") neighbours.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_device.cuh"
#include "la_internal.h"
#include "tc_ptx.cuh"

namespace la {
namespace {

constexpr int kMostVec = 4;   // values of a chunk: the row's sums and sines over twice as many lanes as with 16-byte chunks of
                             // bf16, and half the registers of each (gradients 293 us, with chunks of 8 343; the forward 4% faster)
// A row whose squares sum to more than kRotBig (or to no number) is summed again with its values times kRotDown, one whose
// squares sum to less than kRotSmall, if eps is below that too, with its values times kRotUp: float32 holds squares below
// 2^-126 with fewer and fewer bits.
constexpr float kRotBig = 1e37f, kRotDown = 0x1p-70f, kRotSmall = 0x1p-90f, kRotUp = 0x1p70f;

// VEC values of T as they lie in memory.
template <typename T, int VEC> struct Chunk;
template <> struct Chunk<__nv_bfloat16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ void get(const Raw &r, float (&x)[4]) {
        x[0] = tc::bf16_lo_f(r.x);
        x[1] = tc::bf16_hi_f(r.x);
        x[2] = tc::bf16_lo_f(r.y);
        x[3] = tc::bf16_hi_f(r.y);
    }
    static __device__ __forceinline__ Raw put(const float (&x)[4]) {
        return make_uint2(tc::pack_bf16x2(x[0], x[1]), tc::pack_bf16x2(x[2], x[3]));
    }
};
template <> struct Chunk<__nv_bfloat16, 2> {
    using Raw = uint32_t;
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ void get(Raw r, float (&x)[2]) {
        x[0] = tc::bf16_lo_f(r);
        x[1] = tc::bf16_hi_f(r);
    }
    static __device__ __forceinline__ Raw put(const float (&x)[2]) { return tc::pack_bf16x2(x[0], x[1]); }
};
template <> struct Chunk<__nv_bfloat16, 1> {
    using Raw = __nv_bfloat16;
    static __device__ __forceinline__ Raw zero() { return __float2bfloat16_rn(0.f); }
    static __device__ __forceinline__ void get(Raw r, float (&x)[1]) { x[0] = __bfloat162float(r); }
    static __device__ __forceinline__ Raw put(const float (&x)[1]) { return __float2bfloat16_rn(x[0]); }
};
template <> struct Chunk<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void get(const Raw &r, float (&x)[4]) {
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    }
    static __device__ __forceinline__ Raw put(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <> struct Chunk<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw zero() { return 0.f; }
    static __device__ __forceinline__ void get(Raw r, float (&x)[1]) { x[0] = r; }
    static __device__ __forceinline__ Raw put(const float (&x)[1]) { return x[0]; }
};

__device__ __forceinline__ bool sum_holds(float ss, float least) { return ss <= kRotBig && ss >= least; }
__device__ __forceinline__ float rescale(float ss, float least) { return !(ss <= kRotBig) ? kRotDown : ss >= least ? 1.f : kRotUp; }

// One of q and k.
struct RotSide {
    HeadsView x, g, y;      // input; gradient of the output (gradients only); output or the input's gradient
    const float *weight;    // nullable
    int heads, parts;       // its heads, the ranges that they are cut into
};
struct RotParams {
    RotSide side[2];
    long long tokens;       // B N
    int N, d, r;            // r: rotated pairs
    int span;               // heads of a range
    int blocks;             // CTAs along the tokens
    float c, eps;           // c = 0: no norm
    float least;            // kRotSmall, or 0 where eps makes up for what small squares lose
    const double *freq;
    const long long *positions;   // nullable (the token's index)
    long long pos_batch;          // its stride from one sequence to the next
    float *partials;              // gradients: sums of the weights' gradients, a row for each CTA
};

// Pairs of chunks c = lane + LPR i of a row: offsets of both chunks.
template <int VEC, bool ADJ> __device__ __forceinline__ void chunk_at(int c, int r, int &a, int &b) {
    const int rc = r / VEC;   // ADJ == false: r is a multiple of VEC
    if (ADJ || c >= rc) {
        a = ADJ ? 2 * c * VEC : 2 * r + 2 * (c - rc) * VEC;
        b = a + VEC;
    } else {
        a = c * VEC;
        b = r + a;
    }
}

// Angles are fractions of a turn in units of 2^-64: the frequency becomes such a fraction, and position times it drops
// whole turns by the overflow.  With the frequency's bits m, m / (2 pi) is a product with 2^66 / (2 pi) cut to an integer,
// shifted to its exponent.  An angle is off by less than |position| (2^-64 + |freq| 2^-66) turns: 2^-30 turns for positions
// below kNear and frequencies below 2^kSlow.
constexpr long long kNear = 1ll << 32;
constexpr int kSlow = 3;   // the exponent of 8
struct FreqBits {   // no comparison in 64-bit floating point, which the chip is slow at (10 us became 13 for 3,093 tokens)
    uint64_t m;   // |freq| = m 2^(e - 63)
    int e;
    bool negative;
    __device__ __forceinline__ explicit FreqBits(double freq) {
        const uint64_t bits = (uint64_t)__double_as_longlong(freq);
        e = (int)((bits >> 52) & 0x7FF) - 1023;
        m = ((bits & 0xFFFFFFFFFFFFFull) | (1ull << 52)) << 11;
        negative = bits >> 63;
    }
    __device__ __forceinline__ bool none() const { return e <= -1023 || e >= 64; }   // zero and what is next to it; no angle
};
constexpr uint64_t kInv2Pi = 0xA2F9836E4E441529ull, kInv2PiLow = 0xFC2757D1F534DDC0ull;   // 2^130 / (2 pi), upper and lower half
// `ok` is false for what has no angle: 2^64 and more, infinities, NaN; `fast` is set for 2^kSlow and more.
__device__ __forceinline__ uint64_t turn_fraction(double freq, bool &ok, bool &fast) {
    const FreqBits f(freq);
    ok = f.e < 64;
    fast |= f.e >= kSlow;
    if (f.none()) return 0ull;
    const uint64_t hi = __umul64hi(f.m, kInv2Pi), lo = f.m * kInv2Pi;   // turns 2^(129 - e)
    const int s = 65 - f.e;
    uint64_t t;
    if (s >= 128) t = 0ull;
    else if (s >= 64) t = hi >> (s - 64);
    else t = (hi << (64 - s)) | (lo >> s);
    return f.negative ? 0ull - t : t;
}
// The angle of any position and frequency that has one: the same with fractions in units of 2^-128 and 1 / (2 pi) in 130 bits, off
// by less than |position| (2^-128 + |freq| 2^-130) turns, 2^-27 for frequencies below 2^40 and every position.  It costs the
// forward 5% where every token takes it.
__device__ __forceinline__ uint64_t far_angle(double freq, long long pos) {
    const FreqBits f(freq);
    if (f.none()) return 0ull;
    const uint64_t p0 = f.m * kInv2PiLow, mid = f.m * kInv2Pi, p1 = mid + __umul64hi(f.m, kInv2PiLow),
                   p2 = __umul64hi(f.m, kInv2Pi) + (p1 < mid);
    const int s = 65 - f.e, w = s >> 6, b = s & 63;   // turns 2^(193 - e); s >= 2
    const uint64_t x0 = w == 0 ? p0 : w == 1 ? p1 : w == 2 ? p2 : 0ull, x1 = w == 0 ? p1 : w == 1 ? p2 : 0ull, x2 = w == 0 ? p2 : 0ull;
    const uint64_t lo = b ? (x0 >> b) | (x1 << (64 - b)) : x0, hi = b ? (x1 >> b) | (x2 << (64 - b)) : x1;
    const uint64_t n = pos < 0 ? 0ull - (uint64_t)pos : (uint64_t)pos, at = hi * n + __umul64hi(lo, n);
    return (pos < 0) != f.negative ? 0ull - at : at;
}
__device__ __forceinline__ void sine_of(uint64_t angle, bool ok, float &cs, float &sn) {
    sincospif(__ll2float_rn((long long)angle) * 0x1p-63f, &sn, &cs);
    if (!ok) cs = sn = __int_as_float(0x7FFFFFFF);
}

template <int LPR> __device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a lane knows of its token and chunks.
template <int VEC, int CP, bool ADJ> struct Place {
    int a[CP], b[CP];          // offsets of its chunks
    bool live[CP];
    uint64_t turn[CP][VEC];    // of the pairs of both chunks
    unsigned rot[CP];          // which of them are rotated (ADJ = false: all or none)
    unsigned bad[CP];          // and have no angle
    bool fast;                 // one of its frequencies is 2^kSlow or more
    float cs[CP][VEC], sn[CP][VEC];

    template <int LPR> __device__ __forceinline__ void init(const RotParams &p, int gl) {
        fast = false;
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            const int c = gl + LPR * i;
            live[i] = 2 * c * VEC < p.d;
            chunk_at<VEC, ADJ>(live[i] ? c : 0, p.r, a[i], b[i]);
            rot[i] = bad[i] = 0;
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                bool ok = true;
                turn[i][t] = 0ull;
                if (pair(i, t) < p.r) {
                    rot[i] |= 1u << t;
                    turn[i][t] = turn_fraction(p.freq[pair(i, t)], ok, fast);
                    if (!ok) bad[i] |= 1u << t;
                }
            }
        }
    }
    __device__ __forceinline__ int pair(int i, int t) const { return ADJ ? a[i] / 2 + t : a[i] + t; }   // ADJ: VEC/2 of each chunk, in order
    __device__ __forceinline__ void at(const RotParams &p, long long pos) {
        uint64_t angle[CP][VEC];
#pragma unroll
        for (int i = 0; i < CP; ++i)
#pragma unroll
            for (int t = 0; t < VEC; ++t) angle[i][t] = turn[i][t] * (uint64_t)pos;
        if (fast || pos >= kNear || pos <= -kNear) {
#pragma unroll
            for (int i = 0; i < CP; ++i)
#pragma unroll
                for (int t = 0; t < VEC; ++t)
                    if (rot[i] >> t & 1) angle[i][t] = far_angle(p.freq[pair(i, t)], pos);
        }
#pragma unroll
        for (int i = 0; i < CP; ++i)
            if (ADJ || rot[i])
#pragma unroll
                for (int t = 0; t < VEC; ++t) sine_of(angle[i][t], !(bad[i] >> t & 1), cs[i][t], sn[i][t]);
    }
    // Turns the pairs of chunk pair i, backwards with sign = -1.
    __device__ __forceinline__ void rotate(int i, float (&x)[VEC], float (&y)[VEC], float sign) const {
        if (ADJ && VEC > 1) {
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                float &u = t < VEC / 2 ? x[2 * t % VEC] : y[2 * t % VEC], &v = t < VEC / 2 ? x[(2 * t + 1) % VEC] : y[(2 * t + 1) % VEC];
                if (rot[i] >> t & 1) turn_pair(u, v, i, t, sign);   // what is not rotated does not meet its neighbour
            }
        } else if (rot[i]) {
#pragma unroll
            for (int t = 0; t < VEC; ++t) turn_pair(x[t], y[t], i, t, sign);
        }
    }

  private:
    __device__ __forceinline__ void turn_pair(float &u, float &v, int i, int t, float sign) const {
        const float s = sign * sn[i][t], u1 = fmaf(u, cs[i][t], -v * s);
        v = fmaf(v, cs[i][t], u * s);
        u = u1;
    }
};

// Sizes that a launch is built for, and which of them a call takes: VEC by what the row width, the number of pairs
// and every address and stride are multiples of.
struct RotShape {
    int vec, cls;   // cls: d <= 64, 128, 256
};
inline RotShape rot_shape(const NormRotateArgs &a) {
    const int es = a.dt == LA_DTYPE_BF16 ? 2 : 4;
    auto fits = [&](int vec) {
        if (a.d % (2 * vec) || (a.pairs == LA_PAIRS_HALVES && a.r % vec)) return false;
        const HeadsView *v[6] = {&a.q, &a.k, &a.gq, &a.gk, &a.yq, &a.yk};
        for (int i = 0; i < 6; ++i) {
            if (!v[i]->p) continue;
            if (reinterpret_cast<uintptr_t>(v[i]->p) % (vec * es)) return false;
            if (v[i]->b % vec || v[i]->h % vec || v[i]->t % vec) return false;
        }
        return true;
    };
    RotShape s;
    s.vec = fits(kMostVec) ? kMostVec : es == 2 && fits(2) ? 2 : 1;
    s.cls = a.d <= 64 ? 0 : a.d <= 128 ? 1 : 2;
    return s;
}
// Lanes of a row and chunk pairs of a lane.
template <int VEC, int CLS> struct RotLanes {
    static constexpr int chunks = (32 << CLS) / VEC;   // pairs of chunks of the widest row
    static constexpr int LPR = chunks < 32 ? chunks : 32, CP = chunks / LPR;
};

inline RotParams rot_params(const NormRotateArgs &a) {
    RotParams p{};
    p.side[0] = {a.q, a.gq, a.yq, a.wq, a.Hq, 0};
    p.side[1] = {a.k, a.gk, a.yk, a.wk, a.Hk, 0};
    p.tokens = (long long)a.B * a.N;
    p.N = a.N; p.d = a.d; p.r = a.r;
    p.c = a.norm == LA_NORM_RMS ? 1.f / a.d : a.norm == LA_NORM_L2 ? 1.f : 0.f;
    p.eps = a.eps;
    p.least = a.eps < kRotSmall ? kRotSmall : 0.f;
    p.freq = a.freq;
    p.positions = a.positions;
    p.pos_batch = a.pos_batch;
    p.partials = a.partials;
    return p;
}

inline int rot_sms() {
    int dev = 0, n = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

// Cuts the heads of both sides into ranges: as few as give `want` groups of lanes their token and range.
inline void rot_ranges(RotParams &p, long long want) {
    const int most = p.side[0].heads > p.side[1].heads ? p.side[0].heads : p.side[1].heads;
    p.span = most;
    auto parts = [&](int heads) { return (heads + p.span - 1) / p.span; };
    while (p.span > 1 && p.tokens * (parts(p.side[0].heads) + parts(p.side[1].heads)) < want) p.span = (p.span + 1) / 2;
    p.side[0].parts = parts(p.side[0].heads);
    p.side[1].parts = parts(p.side[1].heads);
}

// K::run<T, VEC, CLS, ADJ>(a) for the sizes that a call takes.
template <typename K, typename T, int VEC> cudaError_t rot_sized(const NormRotateArgs &a, int cls) {
    const bool adj = a.pairs == LA_PAIRS_ADJACENT;
    switch (cls) {
    case 0: return adj ? K::template run<T, VEC, 0, true>(a) : K::template run<T, VEC, 0, false>(a);
    case 1: return adj ? K::template run<T, VEC, 1, true>(a) : K::template run<T, VEC, 1, false>(a);
    default: return adj ? K::template run<T, VEC, 2, true>(a) : K::template run<T, VEC, 2, false>(a);
    }
}
template <typename K> cudaError_t rot_launch(const NormRotateArgs &a) {
    const RotShape s = rot_shape(a);
    if (a.dt == LA_DTYPE_F32) return s.vec == 4 ? rot_sized<K, float, 4>(a, s.cls) : rot_sized<K, float, 1>(a, s.cls);
    return s.vec == 4   ? rot_sized<K, __nv_bfloat16, 4>(a, s.cls)
           : s.vec == 2 ? rot_sized<K, __nv_bfloat16, 2>(a, s.cls)
                        : rot_sized<K, __nv_bfloat16, 1>(a, s.cls);
}

}  // namespace
}  // namespace la
