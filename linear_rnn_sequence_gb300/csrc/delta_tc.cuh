// delta_tc.cuh -- what the tensor-core kernels of the gated delta rule share:
// float32 values as bf16 pieces, a block's gates, the inverse of its unit
// triangular matrix, MMA sequences, tensor maps.
#pragma once

#include "delta_common.cuh"
#include "tc_common.cuh"

namespace la {
namespace {

constexpr int kDC = kDeltaC;   // tokens of a block
constexpr int kStages = 3;     // K and Q tiles in flight
constexpr int kChain = 256, kInner = 64, kOut = 128;   // threads: chain; each T group; P and y
constexpr int kBarChain = 1, kBarInner = 2;   // kBarInner + 1: the second T group; + 2: P and y
constexpr int kBarEnd = kBarInner + 3;
constexpr int kAP = kDC + 4;   // floats of a row of A: rows four banks apart

struct Gates {   // of one block
    float c[kDC], w[kDC], b[kDC], hi[kDC], lo[kDC];
    float f[kDC];   // b_j / c_j (reverse pass: 1 / c_j), for blocks whose c stays above 2^-60 (`fast`)
    float cC, fast, pad[2];
};
// Three pieces of a pair: words of the high, middle and low bf16 halves.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &h, uint32_t &m, uint32_t &l) {
    const uint32_t a0 = f2u(x0), a1 = f2u(x1);
    h = __byte_perm(a0, a1, 0x7632);
    float r0, r1;
    f2unpack(f2sub(f2pack(x0, x1), f2pack(u2f(a0 & 0xFFFF0000u), u2f(a1 & 0xFFFF0000u))), r0, r1);
    const uint32_t b0 = f2u(r0), b1 = f2u(r1);
    m = __byte_perm(b0, b1, 0x7632);
    f2unpack(f2sub(f2pack(r0, r1), f2pack(u2f(b0 & 0xFFFF0000u), u2f(b1 & 0xFFFF0000u))), r0, r1);
    l = __byte_perm(f2u(r0), f2u(r1), 0x7632);
}
// Two pieces, each rounded to nearest: at most 2^-17 of x is left.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &h, uint32_t &m) {
    h = pack_bf16x2(x0, x1);
    float r0, r1;
    f2unpack(f2sub(f2pack(x0, x1), f2pack(bf16_lo_f(h), bf16_hi_f(h))), r0, r1);
    m = pack_bf16x2(r0, r1);
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
constexpr float kMost = 3.3895314e38f;   // bf16's largest; what is larger, or no number, counts as not finite
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= kMost; }
__device__ __forceinline__ float nan_f() { return u2f(0x7FFFFFFFu); }
// Zeroes x from its first value that is not finite on, whose index (x[0]'s: j0) `first` becomes; all of x where
// an earlier one is known.
__device__ __forceinline__ void cut16(float (&x)[16], int j0, int &first) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if (j0 + j < first && !finite(x[j])) first = j0 + j;
        if (j0 + j >= first) x[j] = 0.f;
    }
}
__device__ __forceinline__ void load16(const float *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4 *>(x + i) = *reinterpret_cast<const float4 *>(p + i);
}

// The gates of a block: running log2 sums as pairs hi + lo (differences of two of
// them keep their precision behind a nearly closed gate), c, w = D_Cj b_j, b, f; w and f without
// b_j for the reverse pass.  One warp; two tokens a lane.
template <bool REV> __device__ __forceinline__ void block_gates(Gates &g, const float (&b)[2], const float (&lg)[2], int lane) {
    constexpr float kL = 1.44269502f, kLl = 1.92596299e-8f;   // log2(e) in two floats
    F2 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // 2^-14427 is 0; keeps -inf out
        const float v = lg[i] < -1e4f ? -1e4f : lg[i], h = __fmul_rn(v, kL);
        x[i] = {h, fmaf(v, kL, -h) + v * kLl};
    }
    x[1] = f2sum2(x[0], x[1]);
    F2 s = x[1];
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const F2 y = {__shfl_up_sync(0xffffffffu, s.h, o), __shfl_up_sync(0xffffffffu, s.l, o)};
        if (lane >= o) s = f2sum2(y, s);
    }
    F2 before = {__shfl_up_sync(0xffffffffu, s.h, 1), __shfl_up_sync(0xffffffffu, s.l, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const F2 last = {__shfl_sync(0xffffffffu, s.h, 31), __shfl_sync(0xffffffffu, s.l, 31)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = 2 * lane + i;
        const F2 y = f2sum2(before, x[i]);
        g.hi[j] = y.h;
        g.lo[j] = y.l;
        g.c[j] = ex2_ftz(y.h) * fmaf(y.l, 0.693147f, 1.f);
        g.w[j] = ex2_ftz((last.h - y.h) + (last.l - y.l)) * (REV ? 1.f : b[i]);
        g.b[j] = b[i];
        g.f[j] = (REV ? 1.f : b[i]) * (ex2_ftz(-y.h) * fmaf(y.l, -0.693147f, 1.f));
    }
    // sums of logs of gates <= 1 fall; any other order of a block's sums takes the general path
    const bool fast = __all_sync(0xffffffffu, lg[0] <= 0.f && lg[1] <= 0.f && last.h > -60.f);
    if (lane == 31) g.fast = fast ? 1.f : 0.f;
    if (lane == 31) g.cC = ex2_ftz(last.h) * fmaf(last.l, 0.693147f, 1.f);
}

// T = (I + A)^-1 in place, for A [64][64] strictly lower triangular with zeros above (row pitch
// kAP), by the 64 threads of a T group: the four diagonal blocks of 16 by forward substitution, a
// thread for each column, then twice [[T1, 0], [-T2 A21 T1, T2]].  In the second merge a warp has
// half of the product's columns (with T1 on the right), then half of its rows (with T2 on the left), and
// leaves out the terms that are zero for all of them.  The zeros above T2's diagonal meet rows of A21 T1
// that come later: with CARE, those that are not finite are zeroed, and *bad becomes the first of them, from
// which on T is not what it should be.  (What is not finite in T1 or T2 stays in its row and later ones by itself.)
template <int SZ, bool CARE> __device__ __forceinline__ void merge_blocks(float *A, int t, int bar, int *bad) {
    constexpr int RT = SZ / 8, PER = SZ * SZ / 4 / RT;   // rows of a thread (x 4 columns), threads a pair
    const int pair = t / PER, q = t % PER, half = SZ == 32 ? q >> 5 : 0;
    float *T1 = A + pair * 2 * SZ * (kAP + 1), *A21 = T1 + SZ * kAP, *T2 = A21 + SZ;
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {   // A21 <- A21 T1, then A21 <- -T2 A21
        const bool by_col = SZ == 32 && step == 0;
        const int r = by_col ? q % 8 : q / (SZ / 4) * RT, rs = by_col ? 8 * kAP : kAP;   // first row, row stride
        const int c = by_col ? q / 8 * 4 : q % (SZ / 4) * 4;
        const int m0 = by_col ? half * 16 : 0, m1 = SZ == 32 && step == 1 ? half * 16 + 16 : SZ;
        const float *L = (step ? T2 : A21) + r * kAP, *Rm = (step ? A21 : T1) + c;
        uint64_t acc[RT][2];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = 0ull;
#pragma unroll 2
        for (int m = m0; m < m1; m += 4) {
            float l[RT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
                *reinterpret_cast<float4 *>(l[i]) = *reinterpret_cast<const float4 *>(L + i * rs + m);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(Rm + (m + k) * kAP);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const uint64_t l2 = f2pack(l[i][k], l[i][k]);
                    acc[i][0] = f2fma(l2, x.x, acc[i][0]);
                    acc[i][1] = f2fma(l2, x.y, acc[i][1]);
                }
            }
        }
        named_bar(bar, kInner);
        const float sg = step ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            float y[4];
            f2unpack(acc[i][0], y[0], y[1]);
            f2unpack(acc[i][1], y[2], y[3]);
            if (CARE && step == 0 && !(finite(y[0]) && finite(y[1]) && finite(y[2]) && finite(y[3]))) {
                atomicMin(bad, pair * 2 * SZ + SZ + r + i * (rs / kAP));
                y[0] = y[1] = y[2] = y[3] = 0.f;
            }
            *reinterpret_cast<float4 *>(A21 + r * kAP + i * rs + c) =
                make_float4(sg * y[0], sg * y[1], sg * y[2], sg * y[3]);
        }
        named_bar(bar, kInner);
    }
}
template <bool CARE> __device__ __forceinline__ void invert_unit_lower(float *A, int t, int bar, int *bad) {
    float *blk = A + (t >> 4) * 16 * (kAP + 1);
    const int c = t & 15;
    float x[16] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        uint64_t v = 0ull;   // of even and of odd j; A_ii is zero
#pragma unroll
        for (int j = 0; j < i; j += 4) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(blk + i * kAP + j);
            v = f2fma(a.x, f2pack(x[j], x[j + 1]), v);
            if (j + 2 < i) v = f2fma(a.y, f2pack(x[j + 2], x[j + 3]), v);
        }
        x[i] = (i == c ? 1.f : 0.f) - f2sum(v);
    }
    named_bar(bar, kInner);
#pragma unroll
    for (int i = 0; i < 16; ++i) blk[i * kAP + c] = x[i];
    named_bar(bar, kInner);
    merge_blocks<16, CARE>(A, t, bar, bad);
    merge_blocks<32, CARE>(A, t, bar, bad);
}

// x <- a x and x <- a x + b, by pairs.
__device__ __forceinline__ void mul16(float (&x)[16], const uint32_t (&a)[16]) {
#pragma unroll
    for (int j = 0; j < 16; j += 2)
        f2unpack(f2mul(f2pack(x[j], x[j + 1]), f2pack(u2f(a[j]), u2f(a[j + 1]))), x[j], x[j + 1]);
}
__device__ __forceinline__ void fma16(float (&x)[16], const uint32_t (&a)[16], const float (&b)[16]) {
#pragma unroll
    for (int j = 0; j < 16; j += 2)
        f2unpack(f2fma(f2pack(x[j], x[j + 1]), f2pack(u2f(a[j]), u2f(a[j + 1])), f2pack(b[j], b[j + 1])), x[j],
                 x[j + 1]);
}

// x_j = D_ij b_j s_j (REV: D_ij s_j) for 16 columns j0.. of row i (s: 16 scores; LD: still in flight from TMEM).
template <bool LD, bool REV>
__device__ __forceinline__ void decayed16(const Gates &G, int i, int j0, const uint32_t (&s)[16], float (&x)[16]) {
    if (G.fast != 0.f) {   // c_i (b_j / c_j)
        const float c = G.c[i];
        load16(&G.f[j0], x);
        if (LD) tmem_wait_ld();
        const uint64_t c2 = f2pack(c, c);
#pragma unroll
        for (int j = 0; j < 16; j += 2)
            f2unpack(f2mul(f2mul(c2, f2pack(x[j], x[j + 1])), f2pack(u2f(s[j]), u2f(s[j + 1]))), x[j], x[j + 1]);
    } else {
        const float hi = G.hi[i], lo = G.lo[i];
        float y[16];
        load16(&G.hi[j0], x);
        load16(&G.lo[j0], y);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = ex2_ftz((hi - x[j]) + (lo - y[j]));
        load16(&G.b[j0], y);
        if (LD) tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = x[j] * (REV ? 1.f : y[j]) * u2f(s[j]);
    }
}

__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return smem_desc(addr, 16, 1024, kSwizzle128B); }

// d (+)= A B^T over K = 16 N values: A in TMEM from column `a` on, B token- or row-major (K
// contiguous) in 64-value slabs SLAB bytes apart.
template <int N, int SLAB>
__device__ __forceinline__ void mma_rows(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         bool add) {
    const uint64_t base = desc_k(b);
#pragma unroll
    for (int ks = 0; ks < N; ++ks)
        mma_ts_if(leader, d, a + ks * 8, base + (uint32_t)(((ks >> 2) * SLAB + (ks & 3) * 32) >> 4), idesc,
                  add || ks > 0);
}

// Map over a token tensor of `heads` heads of width w: (feature, token, head, batch), boxes of 64
// features x `rows` tokens.
bool encode_tokens(CUtensorMap *m, const void *base, int layout, int B, int heads, int N, int w, int rows = kDC) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t tok = layout == LA_LAYOUT_BNHD ? (cuuint64_t)heads * w : w;
    const cuuint64_t hd = layout == LA_LAYOUT_BNHD ? w : (cuuint64_t)N * w;
    const cuuint64_t dims[4] = {(cuuint64_t)w, (cuuint64_t)N, (cuuint64_t)heads, (cuuint64_t)B};
    const cuuint64_t strides[3] = {2 * tok, 2 * hd, 2 * (cuuint64_t)heads * N * w};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace la
