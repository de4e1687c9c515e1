// layer_norm.cu -- layer norm over rows, forward and gradients.
//
// Bound by HBM: each value is read once and written once; a row stays in
// registers between its statistics and its result, and the variance is taken
// about the mean (a second pass over registers) rather than as a difference of
// squares.  G threads share a row (16, 32, or a whole CTA for long rows) and
// load 16-byte vectors, or single values where the row length or a pointer is
// not a multiple of 16 bytes.
//
// The gradient kernel keeps the column sums of dy xh and dy of all its rows in
// registers (a thread owns the same columns of every row), writes them once
// per CTA, and a second kernel adds the CTAs' sums in their order.
#include "delta_common.cuh"
#include "tc_ptx.cuh"

namespace la {
namespace {

// E elements of T moved at once.
template <typename T, int E> struct Vec;
template <typename T> struct Vec<T, 1> {
    static __device__ __forceinline__ void load(const T *p, float (&x)[1]) { x[0] = to_f(*p); }
    static __device__ __forceinline__ void store(T *p, const float (&x)[1]) { *p = from_f<T>(x[0]); }
};
template <> struct Vec<float, 4> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[4]) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Vec<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = tc::bf16_lo_f(u[j]);
            x[2 * j + 1] = tc::bf16_hi_f(u[j]);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(tc::pack_bf16x2(x[0], x[1]), tc::pack_bf16x2(x[2], x[3]),
                       tc::pack_bf16x2(x[4], x[5]), tc::pack_bf16x2(x[6], x[7]));
    }
};

// Sum over the G threads of a row: shuffles within a warp, then shared memory.
// A row takes two sums through two `red` arrays in turn, so that the barrier
// of one also orders the other's reads before its next writes.
template <int G> __device__ __forceinline__ float row_sum(float x, float *red) {
    constexpr int W = G < 32 ? G : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (G > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) x += red[w];
    }
    return x;
}

struct LnParams {
    const void *x, *dy;
    void *y;               // y or dx
    const float *weight, *bias;
    float *mean, *rstd;
    float *partials;       // gradients: [CTAs][2][D], or null
    long long rows;
    int D;
    float eps;
};

// V vectors of E elements per thread; column of element j of vector i: (i * G + lane) * E + j.
template <typename T, int E, int V, int G, int THR>
__global__ void __launch_bounds__(THR) layer_norm_kernel(const LnParams p) {
    constexpr int RPB = THR / G;
    __shared__ float red[2][32];
    const int lane = threadIdx.x % G, D = p.D;
    const float invD = 1.f / (float)D;
    const T *x = (const T *)p.x;
    T *y = (T *)p.y;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const long long r = r0 + threadIdx.x / G;
        const bool in = r < p.rows;
        float v[V][E];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * G + lane) * E;
            if (in && c < D) {
                Vec<T, E>::load(x + r * D + c, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) v[i][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < E; ++j) sum += v[i][j];
        }
        const float mean = row_sum<G>(sum, red[0]) * invD;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if ((i * G + lane) * E < D)
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float d = v[i][j] - mean;
                    sq = fmaf(d, d, sq);
                }
        const float var = row_sum<G>(sq, red[1]) * invD;
        const float rstd = 1.f / sqrtf(var + p.eps);
        if (in && lane == 0 && p.mean) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * G + lane) * E;
            if (!in || c >= D) continue;
            float o[E];
#pragma unroll
            for (int j = 0; j < E; ++j) {
                o[j] = (v[i][j] - mean) * rstd;
                if (p.weight) o[j] *= p.weight[c + j];
                if (p.bias) o[j] += p.bias[c + j];
            }
            Vec<T, E>::store(y + r * D + c, o);
        }
    }
}

template <typename T, int E, int V, int G, int THR>
__global__ void __launch_bounds__(THR) layer_norm_backward_kernel(const LnParams p) {
    constexpr int RPB = THR / G;
    __shared__ float red[2][32];
    extern __shared__ float cols[];   // RPB > 1: the row groups' column sums, joined at the end
    const int lane = threadIdx.x % G, D = p.D;
    const float invD = 1.f / (float)D;
    const T *x = (const T *)p.x, *dy = (const T *)p.dy;
    T *dx = (T *)p.y;
    float aw[V][E], ab[V][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) aw[i][j] = ab[i][j] = 0.f;
    for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
        const long long r = r0 + threadIdx.x / G;
        const bool in = r < p.rows;
        const float mean = in ? p.mean[r] : 0.f, rstd = in ? p.rstd[r] : 0.f;
        float xh[V][E], g[V][E], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * G + lane) * E;
            if (in && c < D) {
                Vec<T, E>::load(x + r * D + c, xh[i]);
                Vec<T, E>::load(dy + r * D + c, g[i]);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    xh[i][j] = (xh[i][j] - mean) * rstd;
                    aw[i][j] = fmaf(g[i][j], xh[i][j], aw[i][j]);
                    ab[i][j] += g[i][j];
                    if (p.weight) g[i][j] *= p.weight[c + j];
                    s1 += g[i][j];
                    s2 = fmaf(g[i][j], xh[i][j], s2);
                }
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) xh[i][j] = g[i][j] = 0.f;
            }
        }
        s1 = row_sum<G>(s1, red[0]) * invD;
        s2 = row_sum<G>(s2, red[1]) * invD;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (i * G + lane) * E;
            if (!in || c >= D) continue;
            float o[E];
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = (g[i][j] - s1 - xh[i][j] * s2) * rstd;
            Vec<T, E>::store(dx + r * D + c, o);
        }
    }
    if (!p.partials) return;
    float *out = p.partials + (size_t)blockIdx.x * 2 * D;
    if (RPB == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = (i * G + lane) * E + j;
                if (c < D) { out[c] = aw[i][j]; out[D + c] = ab[i][j]; }
            }
        return;
    }
    // row groups in their order
    constexpr int WID = V * G * E;
    float *mine = cols + (size_t)(threadIdx.x / G) * 2 * WID;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const int c = (i * G + lane) * E + j;
            mine[c] = aw[i][j];
            mine[WID + c] = ab[i][j];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += THR) {
        float a = 0.f, b = 0.f;
        for (int g = 0; g < RPB; ++g) {
            a += cols[(size_t)g * 2 * WID + c];
            b += cols[(size_t)g * 2 * WID + WID + c];
        }
        out[c] = a;
        out[D + c] = b;
    }
}

// Column sums over the CTAs' partial sums; 32 columns x 8 slices of the CTAs.
__global__ void __launch_bounds__(256)
layer_norm_columns_kernel(const float *__restrict__ part, int n, int D, float *dw, float *db) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5, which = blockIdx.y;
    float *out = which ? db : dw;
    if (!out) return;
    float x = 0.f;
    if (c < D)
        for (int i = sl; i < n; i += 8) x += part[(size_t)i * 2 * D + (size_t)which * D + c];
    s[sl][threadIdx.x & 31] = x;
    __syncthreads();
    if (sl == 0 && c < D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x];
        out[c] = t;
    }
}

int sm_count() {
    int dev = 0, n = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n;
}

// Gradient CTAs: enough to fill the GPU, and no more than there are row groups.
int backward_ctas(long long rows, int rows_per_cta) {
    const long long need = (rows + rows_per_cta - 1) / rows_per_cta, most = 4LL * sm_count();
    return (int)(need < most ? (need > 0 ? need : 1) : most);
}

bool vec16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int E, int V, int G, int THR>
cudaError_t go(const LayerNormArgs &a, bool backward) {
    LnParams p{a.x, a.dy, backward ? a.dx : a.y, a.weight, a.bias, a.mean, a.rstd, nullptr, a.rows, a.D,
               a.eps};
    constexpr int RPB = THR / G;
    if (!backward) {
        const long long need = (a.rows + RPB - 1) / RPB, most = 16LL * sm_count();
        layer_norm_kernel<T, E, V, G, THR><<<(unsigned)(need < most ? need : most), THR, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
    p.partials = a.dweight || a.dbias ? a.partials : nullptr;
    const int ctas = backward_ctas(a.rows, RPB);
    const size_t smem = RPB > 1 && p.partials ? sizeof(float) * RPB * 2 * V * G * E : 0;
    layer_norm_backward_kernel<T, E, V, G, THR><<<ctas, THR, smem, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partials) return e;
    layer_norm_columns_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, a.stream>>>(a.partials, ctas, a.D,
                                                                            a.dweight, a.dbias);
    return cudaGetLastError();
}

// The threads of a row and the vectors of a thread, by the number n of vectors in a row; f is called
// with them as template arguments.
template <typename T, int E> cudaError_t shape(const LayerNormArgs &a, bool bwd) {
    const int n = (a.D + E - 1) / E;
    if (E == 1) {
        if (n <= 128) return go<T, E, 4, 32, 256>(a, bwd);
        if (n <= 1024) return go<T, E, 4, 256, 256>(a, bwd);
        if (n <= 4096) return go<T, E, 16, 256, 256>(a, bwd);
        return go<T, E, 16, 1024, 1024>(a, bwd);
    }
    if (n <= 16) return go<T, E, 1, 16, 256>(a, bwd);
    if (n <= 32) return go<T, E, 1, 32, 256>(a, bwd);
    if (n <= 64) return go<T, E, 2, 32, 256>(a, bwd);
    if (n <= 256) return go<T, E, 1, 256, 256>(a, bwd);
    if (n <= 512) return go<T, E, 2, 256, 256>(a, bwd);
    if (n <= 1024) return go<T, E, 4, 256, 256>(a, bwd);
    if (n <= 2048) return go<T, E, 2, 1024, 1024>(a, bwd);
    return go<T, E, 4, 1024, 1024>(a, bwd);
}

template <typename T> cudaError_t run(const LayerNormArgs &a, bool bwd) {
    constexpr int E = 16 / (int)sizeof(T);
    const bool wide = a.D % E == 0 && vec16(a.x) && (bwd ? vec16(a.dy) && vec16(a.dx) : vec16(a.y));
    return wide ? shape<T, E>(a, bwd) : shape<T, 1>(a, bwd);
}

cudaError_t dispatch(const LayerNormArgs &a, bool bwd) {
    return a.dt == LA_DTYPE_BF16 ? run<__nv_bfloat16>(a, bwd) : run<float>(a, bwd);
}

}  // namespace

size_t layer_norm_partials(long long rows, int D, la_dtype) {
    return (size_t)backward_ctas(rows, 1) * 2 * D;   // at most one CTA per row
}
cudaError_t launch_layer_norm(const LayerNormArgs &a) { return dispatch(a, false); }
cudaError_t launch_layer_norm_backward(const LayerNormArgs &a) { return dispatch(a, true); }

}  // namespace la
