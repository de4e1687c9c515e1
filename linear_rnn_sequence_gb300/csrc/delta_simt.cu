// delta_simt.cu -- the gated delta rule on the CUDA cores, in float32: the
// forward and the two recurrent passes of the gradients, token by token.
//
// The columns of S are independent of one another, so a CTA owns 32 columns
// of one head and walks the sequence alone: eight threads share a column,
// each holding d/8 rows of it in registers (rows 32 i + 4 part + r, so that
// the eight float4 reads of a key from shared memory make one 128-byte row).
// A token costs each thread 4 d/8 FMAs; its serial part is the dot product
// k . S with three shuffles, which bounds the kernel at about 0.1 us a token
// whatever the number of heads below the SM count.  It serves float32 inputs
// and widths of 32.
#include "delta_common.cuh"

namespace la {
namespace {

constexpr int kCols = 32;      // columns of a CTA
constexpr int kThr = 256;
constexpr int kTile = 16;      // tokens staged in shared memory at a time

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

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}

// The kTile x D values from token t0 on, as floats in shared memory (zeros past N).
template <int D, typename T>
__device__ __forceinline__ void stage_rows(float (*dst)[D], const T *src, TokenRows r, int t0, int N) {
    for (int i = threadIdx.x; i < kTile * D / 8; i += kThr) {
        const int t = i / (D / 8), c = (i % (D / 8)) * 8;
        float x[8];
        if (t0 + t < N) {
            load_vec<8>(src + r.at(t0 + t) + c, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.f;
        }
        *reinterpret_cast<float4 *>(&dst[t][c]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(&dst[t][c + 4]) = make_float4(x[4], x[5], x[6], x[7]);
    }
}
template <typename T>
__device__ __forceinline__ void stage_cols(float (*dst)[kCols], const T *src, TokenRows r, int c0, int t0,
                                           int N) {
    for (int i = threadIdx.x; i < kTile * kCols; i += kThr) {
        const int t = i / kCols, c = i % kCols;
        dst[t][c] = t0 + t < N ? to_f(src[r.at(t0 + t) + c0 + c]) : 0.f;
    }
}

// SAVE: for the gradients; writes e of every token and the states before each block instead of y.
template <int D, typename T, bool SAVE>
__global__ void __launch_bounds__(kThr) delta_forward_kernel(const DeltaSimt p) {
    constexpr int R = D / 8;
    __shared__ __align__(16) float ks[kTile][D], qs[SAVE ? 1 : kTile][D];
    __shared__ float vs[kTile][kCols], os[kTile][kCols], bs[kTile], as[kTile];
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * kCols;
    const int tid = threadIdx.x, col = tid >> 3, part = tid & 7;
    const TokenRows rk = token_rows(p.layout, b, h / (p.H / p.Hk), p.Hk, p.N, D);
    const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, p.dv);
    const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
    const T *q = (const T *)p.q, *k = (const T *)p.k, *v = (const T *)p.v;
    const size_t st = (size_t)D * p.dv;
    const int nc = delta_blocks(p.N);

    auto row = [&](int r) { return (r >> 2) * 32 + part * 4 + (r & 3); };
    float S[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        S[r] = p.S_in ? p.S_in[bh * st + (size_t)row(r) * p.dv + c0 + col] : 0.f;
    auto keep = [&](float *dst) {
#pragma unroll
        for (int r = 0; r < R; ++r) dst[(size_t)row(r) * p.dv + c0 + col] = S[r];
    };

    for (int t0 = 0; t0 < p.N; t0 += kTile) {
        if (SAVE && t0 % kDeltaC == 0) keep(p.S_ck + ((size_t)bh * (nc + 1) + t0 / kDeltaC) * st);
        __syncthreads();
        stage_rows<D, T>(ks, k, rk, t0, p.N);
        if (!SAVE) stage_rows<D, T>(reinterpret_cast<float(*)[D]>(qs), q, rk, t0, p.N);
        stage_cols<T>(vs, v, rv, c0, t0, p.N);
        if (tid < kTile) {
            const bool in = t0 + tid < p.N;
            bs[tid] = in ? p.beta[rs.at(t0 + tid)] : 0.f;
            as[tid] = in && p.lg ? expf(p.lg[rs.at(t0 + tid)]) : 1.f;
        }
        __syncthreads();
        const int n = min(kTile, p.N - t0);
        for (int t = 0; t < n; ++t) {
            const float a = as[t];
            float kk[R], dot = 0.f;
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&ks[t][row(r)]);
                kk[r] = x.x; kk[r + 1] = x.y; kk[r + 2] = x.z; kk[r + 3] = x.w;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                S[r] *= a;
                dot = fmaf(kk[r], S[r], dot);
            }
            const float e = vs[t][col] - sum8(dot);
            const float u = bs[t] * e;
#pragma unroll
            for (int r = 0; r < R; ++r) S[r] = fmaf(kk[r], u, S[r]);
            if (SAVE) {
                if (part == 0) os[t][col] = e;
            } else {
                float o = 0.f;
#pragma unroll
                for (int r = 0; r < R; r += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&qs[t][row(r)]);
                    o = fmaf(x.x, S[r], fmaf(x.y, S[r + 1], fmaf(x.z, S[r + 2], fmaf(x.w, S[r + 3], o))));
                }
                o = sum8(o);
                if (part == 0) os[t][col] = o;
            }
        }
        __syncthreads();
        for (int i = tid; i < n * kCols; i += kThr) {
            const int t = i / kCols, c = i % kCols;
            if (SAVE)
                p.e[((size_t)bh * p.N + t0 + t) * p.dv + c0 + c] = os[t][c];
            else
                ((T *)p.y)[rv.at(t0 + t) + c0 + c] = from_f<T>(os[t][c]);
        }
    }
    if (SAVE) keep(p.S_ck + ((size_t)bh * (nc + 1) + nc) * st);
    if (!SAVE && p.S_out) keep(p.S_out + bh * st);
}

// Backwards through the tokens: G <- a (I - b k k^T)(G + q dy^T), du = (G + q dy^T)^T k.
template <int D, typename T>
__global__ void __launch_bounds__(kThr) delta_reverse_kernel(const DeltaSimt p) {
    constexpr int R = D / 8;
    __shared__ __align__(16) float ks[kTile][D], qs[kTile][D];
    __shared__ float ys[kTile][kCols], os[kTile][kCols], bs[kTile], as[kTile];
    const int bh = blockIdx.x, b = bh / p.H, h = bh % p.H, c0 = blockIdx.y * kCols;
    const int tid = threadIdx.x, col = tid >> 3, part = tid & 7;
    const TokenRows rk = token_rows(p.layout, b, h / (p.H / p.Hk), p.Hk, p.N, D);
    const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, p.dv);
    const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
    const T *q = (const T *)p.q, *k = (const T *)p.k, *dy = (const T *)p.dy;
    const size_t st = (size_t)D * p.dv;
    const int nc = delta_blocks(p.N);

    auto row = [&](int r) { return (r >> 2) * 32 + part * 4 + (r & 3); };
    float G[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        G[r] = p.dS_out ? p.dS_out[bh * st + (size_t)row(r) * p.dv + c0 + col] : 0.f;
    auto keep = [&](float *dst) {
#pragma unroll
        for (int r = 0; r < R; ++r) dst[(size_t)row(r) * p.dv + c0 + col] = G[r];
    };

    for (int t0 = (p.N - 1) / kTile * kTile; t0 >= 0; t0 -= kTile) {
        const int n = min(kTile, p.N - t0);
        if ((t0 + n) % kDeltaC == 0 || t0 + n == p.N)
            keep(p.G_ck + ((size_t)bh * nc + t0 / kDeltaC) * st);
        __syncthreads();
        stage_rows<D, T>(ks, k, rk, t0, p.N);
        stage_rows<D, T>(qs, q, rk, t0, p.N);
        stage_cols<T>(ys, dy, rv, c0, t0, p.N);
        if (tid < kTile) {
            const bool in = t0 + tid < p.N;
            bs[tid] = in ? p.beta[rs.at(t0 + tid)] : 0.f;
            as[tid] = in && p.lg ? expf(p.lg[rs.at(t0 + tid)]) : 1.f;
        }
        __syncthreads();
        for (int t = n - 1; t >= 0; --t) {
            const float a = as[t], dyc = ys[t][col];
            float kk[R], dot = 0.f;
#pragma unroll
            for (int r = 0; r < R; r += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(&ks[t][row(r)]);
                kk[r] = x.x; kk[r + 1] = x.y; kk[r + 2] = x.z; kk[r + 3] = x.w;
                const float4 z = *reinterpret_cast<const float4 *>(&qs[t][row(r)]);
                G[r] = fmaf(z.x, dyc, G[r]);
                G[r + 1] = fmaf(z.y, dyc, G[r + 1]);
                G[r + 2] = fmaf(z.z, dyc, G[r + 2]);
                G[r + 3] = fmaf(z.w, dyc, G[r + 3]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) dot = fmaf(kk[r], G[r], dot);
            const float du = sum8(dot), dvv = bs[t] * du;
#pragma unroll
            for (int r = 0; r < R; ++r) G[r] = a * fmaf(-kk[r], dvv, G[r]);
            if (part == 0) os[t][col] = du;
        }
        __syncthreads();
        for (int i = tid; i < n * kCols; i += kThr) {
            const int t = i / kCols, c = i % kCols;
            p.du[((size_t)bh * p.N + t0 + t) * p.dv + c0 + c] = os[t][c];
        }
    }
    if (p.dS_in) keep(p.dS_in + bh * st);
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
