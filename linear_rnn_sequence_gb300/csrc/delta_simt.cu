// delta_simt.cu -- the gated delta rule on the CUDA cores, in float32: the
// forward and the two recurrent passes of the gradients, token by token.
//
// The columns of S are independent of one another, so a CTA owns 16 columns
// of one head and walks the sequence alone: eight threads share a column,
// each holding d/8 rows of it in registers (rows 32 i + 4 part + r, so that
// the eight float4 reads of a key from shared memory make one 128-byte row),
// as packed pairs.  Bound by the serial part of a token, k . S with its three
// shuffles, as long as there are fewer CTAs than the SMs take; one warp to a
// scheduler (16 columns rather than 32), the decay beside that chain rather
// than in it, four tokens unrolled and the next tile on its way keep it short:
// 0.11 us a token (B1 H2 N256 d32: 36 us; 61 without these).  It serves float32
// inputs and widths of 32, and bf16 sequences of fewer than 32 tokens.
#include "delta_common.cuh"
#include "tc_common.cuh"

namespace la {
namespace {

constexpr int kCols = 16;      // columns of a CTA
constexpr int kThr = 8 * kCols;
constexpr int kTile = 16;      // tokens staged in shared memory at a time
constexpr int kUnroll = 4;     // tokens in flight

struct DeltaSimt {
    const void *q, *k, *v, *dy;
    void *y;
    const float *beta, *lg;
    int H, Hk, N, dv, layout;
    const float *S_in;
    float *S_out;
    float *S_ck, *G_ck, *e, *du;   // backward workspace (DeltaBwdWs)
    const float *dS_out;
    float *dS_in;
};

// Packed float32 pairs.
__device__ __forceinline__ uint64_t pk(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float pk_sum(uint64_t v) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return a + b;
}
__device__ __forceinline__ void pk_get(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t pk_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pk_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// This thread's rows of a staged vector, and sum of products over them.
template <int D> __device__ __forceinline__ void rows_of(const float *v, int part, uint64_t (&x)[D / 16]) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(v + i * 32 + part * 4);
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
    }
}
template <int P> __device__ __forceinline__ float dot(const uint64_t (&a)[P], const uint64_t (&b)[P]) {
    uint64_t s0 = pk_mul(a[0], b[0]), s1 = pk_mul(a[1], b[1]);
#pragma unroll
    for (int i = 2; i < P; i += 2) {
        s0 = pk_fma(a[i], b[i], s0);
        s1 = pk_fma(a[i + 1], b[i + 1], s1);
    }
    return pk_sum(s0) + pk_sum(s1);
}

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}

// One tile's inputs on their way from memory to shared memory: loaded into registers while the tile
// before is worked on, stored as floats when its buffer is free.  Zeros (gate 1) past token N.
template <int D, typename T, bool QUERY> struct Tile {
    static constexpr int kVec = 16 / (int)sizeof(T), kRow = D / kVec;   // values of a vector, vectors of a row
    static constexpr int NV = (kTile * kRow + kThr - 1) / kThr, NC = kTile * kCols / kThr;
    uint4 k[NV], q[QUERY ? NV : 1];
    T c[NC];
    float b, a;
    __device__ __forceinline__ void load(const T *kp, const T *qp, const T *cp, const float *beta, const float *lg,
                                         TokenRows rk, TokenRows rv, TokenRows rs, int c0, int t0, int N) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = j * kThr + threadIdx.x, t = i / kRow, f = i % kRow * kVec;
            const bool in = t < kTile && t0 + t < N;
            k[j] = in ? __ldg(reinterpret_cast<const uint4 *>(kp + rk.at(t0 + t) + f)) : make_uint4(0u, 0u, 0u, 0u);
            if (QUERY)
                q[j] = in ? __ldg(reinterpret_cast<const uint4 *>(qp + rk.at(t0 + t) + f)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int i = j * kThr + threadIdx.x, t = i / kCols;
            c[j] = t0 + t < N ? cp[rv.at(t0 + t) + c0 + i % kCols] : from_f<T>(0.f);
        }
        if (threadIdx.x < kTile) {
            const int t = t0 + threadIdx.x;
            b = t < N ? beta[rs.at(t)] : 0.f;
            a = t < N && lg ? lg[rs.at(t)] : 0.f;
        }
    }
    static __device__ __forceinline__ void put(float (*dst)[D], int j, uint4 v) {
        const int i = j * kThr + threadIdx.x, t = i / kRow, f = i % kRow * kVec;
        if (t >= kTile) return;
        const unsigned u[4] = {v.x, v.y, v.z, v.w};
        float x[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            x[e] = sizeof(T) == 4 ? __uint_as_float(u[e & 3])
                                  : __uint_as_float(e & 1 ? u[e >> 1] & 0xFFFF0000u : u[e >> 1] << 16);
#pragma unroll
        for (int e = 0; e < kVec; e += 4)
            *reinterpret_cast<float4 *>(&dst[t][f + e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
    __device__ __forceinline__ void store(float (*ks)[D], float (*qs)[D], float (*cs)[kCols], float *bs, float *as) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            put(ks, j, k[j]);
            if (QUERY) put(qs, j, q[j]);
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) cs[(j * kThr + threadIdx.x) / kCols][threadIdx.x % kCols] = to_f(c[j]);
        if (threadIdx.x < kTile) {
            bs[threadIdx.x] = b;
            as[threadIdx.x] = expf(a);
        }
    }
};

// SAVE: for the gradients; writes e of every token and the states before each block instead of y.
template <int D, typename T, bool SAVE>
__global__ void __launch_bounds__(kThr) delta_forward_kernel(const DeltaSimt p) {
    constexpr int R = D / 8, P = R / 2;
    __shared__ __align__(16) float ks[2][kTile][D], qs[2][SAVE ? 1 : kTile][D];
    __shared__ float vs[2][kTile][kCols], os[2][kTile][kCols], bs[2][kTile], as[2][kTile];
    if (SAVE) griddep_launch_dependents();   // the reverse pass, which needs nothing of this one
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * kCols;
    const int tid = threadIdx.x, col = tid >> 3, part = tid & 7;
    const TokenRows rk = token_rows(p.layout, b, h / (p.H / p.Hk), p.Hk, p.N, D);
    const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, p.dv);
    const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
    const T *q = (const T *)p.q, *k = (const T *)p.k, *v = (const T *)p.v;
    const size_t st = (size_t)D * p.dv;
    const int nc = delta_blocks(p.N);

    auto row = [&](int r) { return (r >> 2) * 32 + part * 4 + (r & 3); };
    uint64_t S[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float *src = p.S_in + bh * st + c0 + col;
        S[i] = p.S_in ? pk(src[(size_t)row(2 * i) * p.dv], src[(size_t)row(2 * i + 1) * p.dv]) : 0ull;
    }
    auto keep = [&](float *dst) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            pk_get(S[i], lo, hi);
            dst[(size_t)row(2 * i) * p.dv + c0 + col] = lo;
            dst[(size_t)row(2 * i + 1) * p.dv + c0 + col] = hi;
        }
    };

    Tile<D, T, !SAVE> tile;
    tile.load(k, q, v, p.beta, p.lg, rk, rv, rs, c0, 0, p.N);
    // a tile's results, once the barrier behind it has passed
    auto write_out = [&](int t0, int bf) {
        for (int i = tid; i < min(kTile, p.N - t0) * kCols; i += kThr) {
            const int t = i / kCols, c = i % kCols;
            if (SAVE)
                p.e[((size_t)bh * p.N + t0 + t) * p.dv + c0 + c] = os[bf][t][c];
            else
                ((T *)p.y)[rv.at(t0 + t) + c0 + c] = from_f<T>(os[bf][t][c]);
        }
    };
    int bf = 0;
    for (int t0 = 0; t0 < p.N; t0 += kTile, bf ^= 1) {
        if (SAVE && t0 % kDeltaC == 0) keep(p.S_ck + ((size_t)bh * (nc + 1) + t0 / kDeltaC) * st);
        tile.store(ks[bf], reinterpret_cast<float(*)[D]>(qs[bf]), vs[bf], bs[bf], as[bf]);
        __syncthreads();   // this tile is there; the other buffers have been read, the last results written
        if (t0 + kTile < p.N) tile.load(k, q, v, p.beta, p.lg, rk, rv, rs, c0, t0 + kTile, p.N);
        if (t0 > 0) write_out(t0 - kTile, bf ^ 1);
        const int n = min(kTile, p.N - t0);
        // tokens behind the last have k = 0, b = 0 and a = 1: they change nothing
#pragma unroll 1
        for (int t1 = 0; t1 < n; t1 += kUnroll) {
            float out[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int t = t1 + i;
                const float a = as[bf][t];
                uint64_t kk[P];
                rows_of<D>(ks[bf][t], part, kk);
                const float e = fmaf(-a, sum8(dot<P>(kk, S)), vs[bf][t][col]);
                const float u = bs[bf][t] * e;
                const uint64_t a2 = pk(a, a), u2 = pk(u, u);
#pragma unroll
                for (int r = 0; r < P; ++r) S[r] = pk_fma(kk[r], u2, pk_mul(a2, S[r]));
                if (SAVE) {
                    out[i] = e;
                } else {
                    uint64_t qq[P];
                    rows_of<D>(qs[bf][t], part, qq);
                    out[i] = sum8(dot<P>(qq, S));
                }
            }
            if (part == 0)
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) os[bf][t1 + i][col] = out[i];
        }
    }
    __syncthreads();
    if (p.N > 0) write_out((p.N - 1) / kTile * kTile, bf ^ 1);
    if (SAVE) keep(p.S_ck + ((size_t)bh * (nc + 1) + nc) * st);
    if (!SAVE && p.S_out) keep(p.S_out + bh * st);
}

// Backwards through the tokens: G <- a (I - b k k^T)(G + q dy^T), du = (G + q dy^T)^T k.
template <int D, typename T>
__global__ void __launch_bounds__(kThr) delta_reverse_kernel(const DeltaSimt p) {
    constexpr int R = D / 8, P = R / 2;
    __shared__ __align__(16) float ks[2][kTile][D], qs[2][kTile][D];
    __shared__ float ys[2][kTile][kCols], os[2][kTile][kCols], bs[2][kTile], as[2][kTile];
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * kCols;
    const int tid = threadIdx.x, col = tid >> 3, part = tid & 7;
    const TokenRows rk = token_rows(p.layout, b, h / (p.H / p.Hk), p.Hk, p.N, D);
    const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, p.dv);
    const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
    const T *q = (const T *)p.q, *k = (const T *)p.k, *dy = (const T *)p.dy;
    const size_t st = (size_t)D * p.dv;
    const int nc = delta_blocks(p.N);

    auto row = [&](int r) { return (r >> 2) * 32 + part * 4 + (r & 3); };
    uint64_t G[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float *src = p.dS_out + bh * st + c0 + col;
        G[i] = p.dS_out ? pk(src[(size_t)row(2 * i) * p.dv], src[(size_t)row(2 * i + 1) * p.dv]) : 0ull;
    }
    auto keep = [&](float *dst) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float lo, hi;
            pk_get(G[i], lo, hi);
            dst[(size_t)row(2 * i) * p.dv + c0 + col] = lo;
            dst[(size_t)row(2 * i + 1) * p.dv + c0 + col] = hi;
        }
    };

    const int last = (p.N - 1) / kTile * kTile;
    Tile<D, T, true> tile;
    tile.load(k, q, dy, p.beta, p.lg, rk, rv, rs, c0, last, p.N);
    auto write_out = [&](int t0, int bf) {
        for (int i = tid; i < min(kTile, p.N - t0) * kCols; i += kThr)
            p.du[((size_t)bh * p.N + t0 + i / kCols) * p.dv + c0 + i % kCols] = os[bf][i / kCols][i % kCols];
    };
    int bf = 0;
    for (int t0 = last; t0 >= 0; t0 -= kTile, bf ^= 1) {
        const int n = min(kTile, p.N - t0);
        if ((t0 + n) % kDeltaC == 0 || t0 + n == p.N)
            keep(p.G_ck + ((size_t)bh * nc + t0 / kDeltaC) * st);
        tile.store(ks[bf], qs[bf], ys[bf], bs[bf], as[bf]);
        __syncthreads();   // this tile is there; the other buffers have been read, the last results written
        if (t0 > 0) tile.load(k, q, dy, p.beta, p.lg, rk, rv, rs, c0, t0 - kTile, p.N);
        if (t0 < last) write_out(t0 + kTile, bf ^ 1);
        // tokens behind the last have k = q = 0, b = 0 and a = 1: they change nothing
#pragma unroll 1
        for (int t1 = (n - 1) / kUnroll * kUnroll; t1 >= 0; t1 -= kUnroll) {
            float out[kUnroll];
#pragma unroll
            for (int i = kUnroll - 1; i >= 0; --i) {
                const int t = t1 + i;
                const float a = as[bf][t], y = ys[bf][t][col], ab = a * bs[bf][t];
                uint64_t kk[P], qq[P];
                rows_of<D>(ks[bf][t], part, kk);
                rows_of<D>(qs[bf][t], part, qq);
                const uint64_t y2 = pk(y, y), a2 = pk(a, a);
#pragma unroll
                for (int r = 0; r < P; ++r) G[r] = pk_fma(qq[r], y2, G[r]);
                const float du = sum8(dot<P>(kk, G)), w = -ab * du;
                const uint64_t w2 = pk(w, w);
#pragma unroll
                for (int r = 0; r < P; ++r) G[r] = pk_fma(kk[r], w2, pk_mul(a2, G[r]));
                out[i] = du;
            }
            if (part == 0)
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) os[bf][t1 + i][col] = out[i];
        }
    }
    __syncthreads();
    write_out(0, bf ^ 1);
    if (p.dS_in) keep(p.dS_in + bh * st);
    griddep_wait();   // what follows in the stream waits for this kernel, and so for the states' pass beside it
}

DeltaSimt params(const DeltaArgs &a) {
    DeltaSimt p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.dy = a.dy;
    p.y = a.y;
    p.beta = a.beta; p.lg = a.log_gate;
    p.H = a.H; p.Hk = a.Hk; p.N = a.N; p.dv = a.dv; p.layout = a.layout;
    p.S_in = a.S_in; p.S_out = a.S_out;
    p.dS_out = a.dS_out; p.dS_in = a.dS_in;
    return p;
}

template <int D, typename T>
cudaError_t launch_d(const DeltaArgs &a, int what) {
    DeltaSimt p = params(a);
    const dim3 grid(a.B * a.H, a.dv / kCols);
    if (what) {
        const DeltaBwdWs w = delta_bwd_ws(a);
        p.S_ck = w.S; p.G_ck = w.G; p.e = w.e; p.du = w.du;
    }
    if (what == 0) delta_forward_kernel<D, T, false><<<grid, kThr, 0, a.stream>>>(p);
    if (what == 1) delta_forward_kernel<D, T, true><<<grid, kThr, 0, a.stream>>>(p);
    // Beside the states' pass where both fit the SMs, one CTA each (B2 H4 N777 d64, 32 CTAs: 156 us for the
    // gradients, 237 one after the other).  Where they share SMs the second pass's CTAs crowd on the
    // emptier ones: 128 CTAs of d = 128, 2048 tokens: 1516 us, 1080 one after the other.
    if (what == 2 && 2 * (long long)grid.x * grid.y <= num_sms())
        return launch_overlapped(delta_reverse_kernel<D, T>, grid, dim3(kThr), 0, a.stream, p);
    if (what == 2) delta_reverse_kernel<D, T><<<grid, kThr, 0, a.stream>>>(p);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_t(const DeltaArgs &a, int what) {
    switch (a.d) {
    case 32: return launch_d<32, T>(a, what);
    case 64: return launch_d<64, T>(a, what);
    case 128: return launch_d<128, T>(a, what);
    }
    return cudaErrorInvalidValue;
}
cudaError_t launch(const DeltaArgs &a, int what) {
    return a.dt == LA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, what) : launch_t<float>(a, what);
}

}  // namespace

cudaError_t launch_delta_forward_simt(const DeltaArgs &a) { return launch(a, 0); }
cudaError_t launch_delta_states_simt(const DeltaArgs &a) { return launch(a, 1); }
cudaError_t launch_delta_reverse_simt(const DeltaArgs &a) { return launch(a, 2); }

}  // namespace la
