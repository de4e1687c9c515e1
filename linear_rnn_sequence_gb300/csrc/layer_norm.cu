// layer_norm.cu -- layer norm over rows, forward and gradients.
//
// Bound by HBM: each value is read once and written once; a row stays in
// registers between its statistics and its result, and the variance is taken
// about the mean (a second pass over registers) rather than as a difference of
// squares.  G threads share a row (16, 32, or a whole CTA for long rows) and
// load 16-byte vectors, or two values or one where the row length or a pointer is
// not a multiple of 16 bytes or of two values.  1048576 x 128 bf16: 93 us, 5.8 TB/s of the 6.8
// that a copy reaches; gradients at 65536 x 2048: 154 us, 5.2 TB/s.
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
    using Raw = T;
    static __device__ __forceinline__ Raw load(const T *p) { return *p; }
    static __device__ __forceinline__ Raw zero() { return from_f<T>(0.f); }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[1]) { x[0] = to_f(r); }
    static __device__ __forceinline__ void store(T *p, const float (&x)[1]) { *p = from_f<T>(x[0]); }
};
template <> struct Vec<float, 2> {
    using Raw = float2;
    static __device__ __forceinline__ Raw load(const float *p) { return *reinterpret_cast<const float2 *>(p); }
    static __device__ __forceinline__ Raw zero() { return make_float2(0.f, 0.f); }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[2]) { x[0] = r.x; x[1] = r.y; }
    static __device__ __forceinline__ void store(float *p, const float (&x)[2]) {
        *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    }
};
template <> struct Vec<__nv_bfloat16, 2> {
    using Raw = unsigned;
    static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p) { return *reinterpret_cast<const unsigned *>(p); }
    static __device__ __forceinline__ Raw zero() { return 0u; }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[2]) {
        x[0] = tc::bf16_lo_f(r);
        x[1] = tc::bf16_hi_f(r);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[2]) {
        *reinterpret_cast<unsigned *>(p) = tc::pack_bf16x2(x[0], x[1]);
    }
};
template <> struct Vec<float, 4> {
    using Raw = float4;
    static __device__ __forceinline__ Raw load(const float *p) { return *reinterpret_cast<const float4 *>(p); }
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ void unpack(Raw r, float (&x)[4]) {
        x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }
    static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
    static __device__ __forceinline__ void unpack(Raw w, float (&x)[8]) {
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

// Sums over the G threads of a row, for RW rows at once: shuffles within a
// warp, then shared memory.  `red` alternates between two places, so that one
// barrier a sum is enough.
template <int G, int RW> __device__ __forceinline__ void row_sums(float (&x)[RW], float (*red)[RW]) {
    constexpr int W = G < 32 ? G : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < RW; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    if (G > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < RW; ++i) red[threadIdx.x >> 5][i] = x[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RW; ++i) x[i] = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w)
#pragma unroll
            for (int i = 0; i < RW; ++i) x[i] += red[w][i];
    }
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

// G threads share a row and have V vectors of E elements of it; column of element j of vector i:
// (i * G + lane) * E + j.  RW rows of each group are in flight at once.
template <typename T, int E, int V, int G, int RW, int THR>
__global__ void __launch_bounds__(THR) layer_norm_kernel(const LnParams p) {
    constexpr int RPB = THR / G;
    constexpr bool kKeep = V * E <= 16;   // weight and bias stay in registers
    __shared__ float red[2][32][RW];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, D = p.D;
    const float invD = 1.f / (float)D;
    const T *x = (const T *)p.x;
    T *y = (T *)p.y;
    float w[kKeep ? V : 1][E], bi[kKeep ? V : 1][E];
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = (i * G + lane) * E + j;
                w[i][j] = p.weight && c < D ? p.weight[c] : 1.f;
                bi[i][j] = p.bias && c < D ? p.bias[c] : 0.f;
            }
    }
    auto fetch = [&](long long r0, typename Vec<T, E>::Raw (&raw)[RW][V]) {
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const long long r = r0 + k * RPB + grp;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * G + lane) * E;
                raw[k][i] = r < p.rows && c < D ? Vec<T, E>::load(x + r * D + c) : Vec<T, E>::zero();
            }
        }
    };
    typename Vec<T, E>::Raw raw[RW][V], ahead[RW][V];
    const long long step = (long long)gridDim.x * RPB * RW;
    fetch((long long)blockIdx.x * RPB * RW, ahead);
    for (long long r0 = (long long)blockIdx.x * RPB * RW; r0 < p.rows; r0 += step) {
        float s[RW], mean[RW];
#pragma unroll
        for (int k = 0; k < RW; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) raw[k][i] = ahead[k][i];
        fetch(r0 + step, ahead);   // in flight through this step's sums
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            s[k] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v[E];
                Vec<T, E>::unpack(raw[k][i], v);
#pragma unroll
                for (int j = 0; j < E; ++j) s[k] += v[j];
            }
        }
        row_sums<G, RW>(s, red[0]);
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            mean[k] = s[k] * invD;
            s[k] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((i * G + lane) * E < D) {
                    float v[E];
                    Vec<T, E>::unpack(raw[k][i], v);
#pragma unroll
                    for (int j = 0; j < E; ++j) s[k] = fmaf(v[j] - mean[k], v[j] - mean[k], s[k]);
                }
        }
        row_sums<G, RW>(s, red[1]);
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const long long r = r0 + k * RPB + grp;
            if (r >= p.rows) continue;
            const float rstd = 1.f / sqrtf(fmaf(s[k], invD, p.eps));
            if (lane == 0 && p.mean) {
                p.mean[r] = mean[k];
                p.rstd[r] = rstd;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * G + lane) * E;
                if (c >= D) continue;
                float v[E];
                Vec<T, E>::unpack(raw[k][i], v);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    v[j] = (v[j] - mean[k]) * rstd;
                    if (kKeep) {
                        v[j] = fmaf(v[j], w[i][j], bi[i][j]);
                    } else {
                        if (p.weight) v[j] *= p.weight[c + j];
                        if (p.bias) v[j] += p.bias[c + j];
                    }
                }
                Vec<T, E>::store(y + r * D + c, v);
            }
        }
    }
}

template <typename T, int E, int V, int G, int RW, int THR>
__global__ void __launch_bounds__(THR) layer_norm_backward_kernel(const LnParams p) {
    constexpr int RPB = THR / G;
    constexpr bool kKeep = V * E <= 16;
    __shared__ float red[2][32][2 * RW];
    extern __shared__ float cols[];   // RPB > 1: the row groups' column sums, joined at the end
    const int lane = threadIdx.x % G, grp = threadIdx.x / G, D = p.D;
    const float invD = 1.f / (float)D;
    const T *x = (const T *)p.x, *dy = (const T *)p.dy;
    T *dx = (T *)p.y;
    float aw[V][E], ab[V][E], w[kKeep ? V : 1][E];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            aw[i][j] = ab[i][j] = 0.f;
            const int c = (i * G + lane) * E + j;
            if (kKeep) w[i][j] = p.weight && c < D ? p.weight[c] : 1.f;
        }
    int turn = 0;
    typename Vec<T, E>::Raw rx[RW][V], ry[RW][V], ax[RW][V], ay[RW][V];
    float mean[RW], rstd[RW], am[RW], ar[RW];
    auto fetch = [&](long long r0) {
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const long long r = r0 + k * RPB + grp;
            const bool in = r < p.rows;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * G + lane) * E;
                ax[k][i] = in && c < D ? Vec<T, E>::load(x + r * D + c) : Vec<T, E>::zero();
                ay[k][i] = in && c < D ? Vec<T, E>::load(dy + r * D + c) : Vec<T, E>::zero();
            }
            am[k] = in ? p.mean[r] : 0.f;
            ar[k] = in ? p.rstd[r] : 0.f;
        }
    };
    const long long step = (long long)gridDim.x * RPB * RW;
    fetch((long long)blockIdx.x * RPB * RW);
    for (long long r0 = (long long)blockIdx.x * RPB * RW; r0 < p.rows; r0 += step) {
        float s[2 * RW];
#pragma unroll
        for (int k = 0; k < RW; ++k) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                rx[k][i] = ax[k][i];
                ry[k][i] = ay[k][i];
            }
            mean[k] = am[k];
            rstd[k] = ar[k];
        }
        fetch(r0 + step);   // in flight through this step's sums
        // xh and g = dy weight of one vector; what lies behind the row or the last row adds nothing
        // (dy = 0 there)
        auto values = [&](int k, int i, float (&xh)[E], float (&g)[E], float (&d)[E]) {
            Vec<T, E>::unpack(rx[k][i], xh);
            Vec<T, E>::unpack(ry[k][i], d);
            const int c = (i * G + lane) * E;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                xh[j] = (xh[j] - mean[k]) * rstd[k];
                g[j] = kKeep ? d[j] * w[i][j] : p.weight && c + j < D ? d[j] * p.weight[c + j] : d[j];
            }
        };
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            s[2 * k] = s[2 * k + 1] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float xh[E], g[E], d[E];
                values(k, i, xh, g, d);
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    s[2 * k] += g[j];
                    s[2 * k + 1] = fmaf(g[j], xh[j], s[2 * k + 1]);
                    aw[i][j] = fmaf(d[j], xh[j], aw[i][j]);
                    ab[i][j] += d[j];
                }
            }
        }
        row_sums<G, 2 * RW>(s, red[turn]);
        turn ^= 1;
#pragma unroll
        for (int k = 0; k < RW; ++k) {
            const long long r = r0 + k * RPB + grp;
            if (r >= p.rows) continue;
            const float s1 = s[2 * k] * invD, s2 = s[2 * k + 1] * invD;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (i * G + lane) * E;
                if (c >= D) continue;
                float xh[E], g[E], d[E];
                values(k, i, xh, g, d);
#pragma unroll
                for (int j = 0; j < E; ++j) d[j] = (g[j] - s1 - xh[j] * s2) * rstd[k];
                Vec<T, E>::store(dx + r * D + c, d);
            }
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
    float *mine = cols + (size_t)grp * 2 * WID;
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

// Gradient CTAs: two an SM, whose rows in flight fill the memory's queues (more of them measured no
// faster, and leave more partial sums), and no more than there are row groups.
int backward_ctas(long long rows, int rows_per_cta) {
    const long long need = (rows + rows_per_cta - 1) / rows_per_cta, most = 2LL * sm_count();
    return (int)(need < most ? (need > 0 ? need : 1) : most);
}

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

template <typename T, int E, int V, int G, int RW, int THR>
cudaError_t go(const LayerNormArgs &a, bool backward) {
    LnParams p{a.x, a.dy, backward ? a.dx : a.y, a.weight, a.bias, a.mean, a.rstd, nullptr, a.rows, a.D,
               a.eps};
    constexpr int RPB = THR / G;
    if (!backward) {
        const long long need = (a.rows + RPB * RW - 1) / (RPB * RW), most = (RPB > 1 ? 6LL : 4LL) * sm_count();
        layer_norm_kernel<T, E, V, G, RW, THR><<<(unsigned)(need < most ? need : most), THR, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
    p.partials = a.dweight || a.dbias ? a.partials : nullptr;
    const int ctas = backward_ctas(a.rows, RPB * RW);
    const size_t smem = RPB > 1 && p.partials ? sizeof(float) * RPB * 2 * V * G * E : 0;
    layer_norm_backward_kernel<T, E, V, G, RW, THR><<<ctas, THR, smem, a.stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partials) return e;
    layer_norm_columns_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, a.stream>>>(a.partials, ctas, a.D,
                                                                            a.dweight, a.dbias);
    return cudaGetLastError();
}

// The threads of a row, the vectors of a thread and the rows in flight, by the number n of vectors in
// a row.  Two rows of a group at once, beside the next two on their way, where a thread has at most eight
// values of a row, or four of those that go by pairs or one by one (1048576 x 128 bf16: 93 us, 101 without the
// next ones, 121 with four rows and without; gradients of 16384 x 4096 float32: 134 us, 152 by one row), but not
// with 1024 threads, whose 64 registers do not hold them (gradients of 13107 x 5120 float32: 184 us, 440 by
// two); one row where it has more, and for few rows, which want threads rather than rows in flight.
// Pairs and single values: a warp to a row as far as its registers go, and threads that fit the row beyond
// (gradients, 61688 x 158 float32: 36 us, 127 with 256 threads a row; 13550 x 2090 bf16: 60 us, 135 by single values).
template <typename T, int E, int V, int G, int THR>
cudaError_t rows_in_flight(const LayerNormArgs &a, bool bwd) {
    constexpr int RW = V * E <= (E > 2 ? 8 : 4) && THR < 1024 ? 2 : 1;
    if (RW == 1 || a.rows >= 4LL * RW * sm_count() * (THR / G)) return go<T, E, V, G, RW, THR>(a, bwd);
    return go<T, E, V, G, 1, THR>(a, bwd);
}
template <typename T, int E> cudaError_t shape(const LayerNormArgs &a, bool bwd) {
    const int n = (a.D + E - 1) / E;   // up to 16384 / E
    if (n <= 16) return rows_in_flight<T, E, 1, 16, 256>(a, bwd);
    if (n <= 32) return rows_in_flight<T, E, 1, 32, 256>(a, bwd);
    if (n <= 64) return rows_in_flight<T, E, 2, 32, 256>(a, bwd);
    if constexpr (E <= 2) {   // rows that start anywhere: a warp takes up to 512 values
        if (n <= 128) return rows_in_flight<T, E, 4, 32, 256>(a, bwd);
        if (n <= 256) return rows_in_flight<T, E, 8, 32, 256>(a, bwd);
        if (E == 1 && n <= 512) return rows_in_flight<T, E, 16 / E, 32, 256>(a, bwd);
        if (n <= 1024) return rows_in_flight<T, E, 4, 256, 256>(a, bwd);
        if (n <= 2048) return rows_in_flight<T, E, 8, 256, 256>(a, bwd);
        if (n <= 4096) return rows_in_flight<T, E, 8, 512, 512>(a, bwd);
        if (n <= 8192) return rows_in_flight<T, E, 8, 1024, 1024>(a, bwd);
        return rows_in_flight<T, E, 16 / E, 1024, 1024>(a, bwd);
    } else {
        if (n <= 256) return rows_in_flight<T, E, 1, 256, 256>(a, bwd);
        if (n <= 512) return rows_in_flight<T, E, 2, 256, 256>(a, bwd);
        if (n <= 1024) return rows_in_flight<T, E, 2, 512, 512>(a, bwd);
        if (E == 8 || n <= 2048) return rows_in_flight<T, E, 2, 1024, 1024>(a, bwd);
        return rows_in_flight<T, E, E == 8 ? 2 : 4, 1024, 1024>(a, bwd);
    }
}

template <typename T> cudaError_t run(const LayerNormArgs &a, bool bwd) {
    constexpr int E = 16 / (int)sizeof(T);
    auto by = [&](int e) {
        const size_t n = e * sizeof(T);
        return a.D % e == 0 && aligned(a.x, n) && (bwd ? aligned(a.dy, n) && aligned(a.dx, n) : aligned(a.y, n));
    };
    if (by(E)) return shape<T, E>(a, bwd);
    return by(2) ? shape<T, 2>(a, bwd) : shape<T, 1>(a, bwd);
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
