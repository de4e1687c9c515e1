// retention_simt.cu -- retention on the CUDA cores, in float32: blocks of 64 tokens in three launches.
//
//   1. each block's own sum of k_j v_j^T, at the weights of its end (a CTA a block);
//   2. the states before the blocks, one after another over the sums (a thread for four of a state's values);
//   3. each block's y from its state (a CTA a block): scores, their product with v, the state's part.
// Every block of 1 and 3 runs at once, so a long sequence of few heads fills the GPU as well as many short ones
// do.  The gradients take the states of both directions in one pass of 1 and 2, and all three of them in 3 (two launches if
// d and dv differ).  Bound by the float32 multiplications, (4 d + 64) dv + 64 d of them for a token of a head, and by
// the states' way through memory, 16 d dv bytes a block; small calls by the three launches.
// It serves float32 inputs and widths of 32.
#include "retention.cuh"
#include "tc_common.cuh"

namespace la {
namespace {

using namespace tc;

constexpr int kRC = 64;       // tokens of a block
constexpr int kRThr = 256;    // 16 x 16 threads
constexpr int kScanThr = 128;
constexpr int kPad = 4;       // floats behind a row of Q, K and P: rows four banks apart

// One retention, or one of its gradients; their state arrays are [head][block][d][dv], or, to a job with `trans`,
// [head][block][dv][d].
struct Job {
    const void *q, *k, *v;
    void *y;
    const float *S_in;
    float *S_out, *states;
    bool rev, trans;
};
struct RetainSimt {
    Job job[3];
    const float *gamma;
    int H, N, layout, nblk, heads;
    int tokens;               // of a block of the scan
};

// Rows t0.. of a head as floats into dst (rows LD floats apart), zeros from token n on.
template <int W, int LD, typename T>
__device__ __forceinline__ void stage(float *dst, const T *src, TokenRows r, int t0, int n) {
    constexpr int V = 16 / (int)sizeof(T), ROW = W / V;
    for (int e = threadIdx.x; e < kRC * ROW; e += kRThr) {
        const int t = e / ROW, f = e % ROW * V;
        float x[V];
        if (t < n) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src + r.at(t0 + t) + f));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < V; ++i)
                x[i] = V == 4 ? __uint_as_float(w[i & 3]) : __uint_as_float(i & 1 ? w[i >> 1 & 3] & 0xFFFF0000u : w[i >> 1 & 3] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(dst + t * LD + f + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}

// A thread's columns of a row of W values: groups of G, 16 G apart.
template <int W> struct Cols {
    static constexpr int G = W / 16 < 4 ? W / 16 : 4, NG = W / 16 / G, N = G * NG;
    static __device__ __forceinline__ void load(const float *row, int tx, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const float *p = row + i * 16 * G + tx * G;
            if (G == 4) {
                const float4 t = *reinterpret_cast<const float4 *>(p);
                x[i * G] = t.x; x[i * G + 1 % G] = t.y; x[i * G + 2 % G] = t.z; x[i * G + 3 % G] = t.w;
            } else {
                const float2 t = *reinterpret_cast<const float2 *>(p);
                x[i * G] = t.x; x[i * G + 1 % G] = t.y;
            }
        }
    }
    static __device__ __forceinline__ int at(int tx, int c) { return c / G * 16 * G + tx * G + c % G; }
};

template <int D, int DV, typename T>
__global__ void __launch_bounds__(kRThr) retain_sums_kernel(const RetainSimt p) {
    extern __shared__ float sm[];
    float *K = sm, *V = K + kRC * D;
    __shared__ float w[kRC];
    griddep_launch_dependents();   // the scan, which waits for this grid's end
    const int unit = blockIdx.x % (p.heads * p.nblk), bh = unit / p.nblk, blk = unit % p.nblk, b = bh / p.H, h = bh % p.H;
    const int t0 = blk * kRC, n = min(kRC, p.N - t0);
    const Job &jb = p.job[blockIdx.x / (p.heads * p.nblk)];
    if (threadIdx.x < kRC) w[threadIdx.x] = (int)threadIdx.x < n ? gamma_power(p.gamma[h], key_exp(jb.rev, threadIdx.x, n)) : 0.f;
    stage<D, D>(K, (const T *)jb.k, token_rows(p.layout, b, h, p.H, p.N, D), t0, n);
    stage<DV, DV>(V, (const T *)jb.v, token_rows(p.layout, b, h, p.H, p.N, DV), t0, n);
    __syncthreads();
    using CA = Cols<D>;
    using CC = Cols<DV>;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[CA::N][CC::N];
#pragma unroll
    for (int a = 0; a < CA::N; ++a)
#pragma unroll
        for (int c = 0; c < CC::N; ++c) acc[a][c] = 0.f;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        float x[CA::N], y[CC::N];
        CA::load(K + j * D, ty, x);
        CC::load(V + j * DV, tx, y);
        const float g = w[j];
#pragma unroll
        for (int a = 0; a < CA::N; ++a) {
            x[a] *= g;
#pragma unroll
            for (int c = 0; c < CC::N; ++c) acc[a][c] = fmaf(x[a], y[c], acc[a][c]);
        }
    }
    float *out = jb.states + (size_t)unit * D * DV;
#pragma unroll
    for (int a = 0; a < CA::N; ++a)
#pragma unroll
        for (int c = 0; c < CC::N; ++c) out[CA::at(ty, a) * DV + CC::at(tx, c)] = acc[a][c];
}

// The sums become the states before their blocks.
__global__ void __launch_bounds__(kScanThr) retain_scan_kernel(const RetainSimt p, int D, int DV) {
    const int st = D * DV, parts = st / 4 / kScanThr;
    const int unit = blockIdx.x / parts, bh = unit % p.heads, at = (blockIdx.x % parts * kScanThr + threadIdx.x) * 4;
    const Job &jb = p.job[unit / p.heads];
    const bool rev = jb.rev, trans = jb.trans;
    const float g = p.gamma[bh % p.H], whole = gamma_power(g, p.tokens), last = gamma_power(g, p.N - (p.nblk - 1) * p.tokens);
    float4 *s = reinterpret_cast<float4 *>(jb.states + (size_t)bh * p.nblk * st + at);
    const int step = st / 4;
    griddep_launch_dependents();   // what takes the states: it waits for this grid's end in turn
    griddep_wait();
    // of a state's values in their order here; a transposed state's lie DV apart
    auto where = [&](int i) { return trans ? (size_t)((at + i) % DV) * D + (at + i) / DV : (size_t)at + i; };
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (jb.S_in)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = jb.S_in[(size_t)bh * st + where(i)];
    constexpr int U = 8;
    for (int k0 = 0; k0 < p.nblk; k0 += U) {
        float4 u[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (k0 + i < p.nblk) u[i] = s[(size_t)(rev ? p.nblk - 1 - k0 - i : k0 + i) * step];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (k0 + i < p.nblk) {
                const int blk = rev ? p.nblk - 1 - k0 - i : k0 + i;
                const float f = blk == p.nblk - 1 ? last : whole;
                s[(size_t)blk * step] = make_float4(x[0], x[1], x[2], x[3]);
                x[0] = fmaf(f, x[0], u[i].x);
                x[1] = fmaf(f, x[1], u[i].y);
                x[2] = fmaf(f, x[2], u[i].z);
                x[3] = fmaf(f, x[3], u[i].w);
            }
    }
    if (jb.S_out)
#pragma unroll
        for (int i = 0; i < 4; ++i) jb.S_out[(size_t)bh * st + where(i)] = x[i];
}

// acc[4][C] += sum over 4 j of p[4][4] v[4][C]; DIAG: only where row r may see j.
template <int N, bool DIAG> __device__ __forceinline__ void four(float (&acc)[4][N], const float *P, int ldp, const float *V, int ldv, int tx, bool rev) {
    float pr[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float4 t = *reinterpret_cast<const float4 *>(P + r * ldp);
        pr[r][0] = t.x; pr[r][1] = t.y; pr[r][2] = t.z; pr[r][3] = t.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[N];
        Cols<N * 16>::load(V + j * ldv, tx, v);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (DIAG && (rev ? j < r : j > r)) continue;   // a value that is not finite meets no zero
#pragma unroll
            for (int c = 0; c < N; ++c) acc[r][c] = fmaf(pr[r][j], v[c], acc[r][c]);
        }
    }
}

template <int D, int DV, typename T> struct OutLay {
    static constexpr int LQ = D + kPad, LP = kRC + kPad, SR = 32;   // SR: rows of the state at a time
    static constexpr int over = LP * kRC + SR * DV, k = kRC * LQ > over ? kRC * LQ : over;   // K, then P and rows of S
    static constexpr int bytes = 4 * (kRC * LQ + k + kRC * DV);
};

template <int D, int DV, typename T>
__global__ void __launch_bounds__(kRThr, 2) retain_out_kernel(const RetainSimt p) {
    using L = OutLay<D, DV, T>;
    using CC = Cols<DV>;
    constexpr int C = CC::N;
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + kRC * L::LQ, *V = K + L::k, *P = K, *S = P + L::LP * kRC;
    __shared__ float pw[kRC + 1];
    const int unit = blockIdx.x % (p.heads * p.nblk), bh = unit / p.nblk, blk = unit % p.nblk, b = bh / p.H, h = bh % p.H;
    const int t0 = blk * kRC, n = min(kRC, p.N - t0);
    const Job &jb = p.job[blockIdx.x / (p.heads * p.nblk)];
    const bool rev = jb.rev, trans = jb.trans;
    if (threadIdx.x <= kRC) pw[threadIdx.x] = gamma_power(p.gamma[h], threadIdx.x);
    const TokenRows rk = token_rows(p.layout, b, h, p.H, p.N, D), rv = token_rows(p.layout, b, h, p.H, p.N, DV);
    stage<D, L::LQ>(Q, (const T *)jb.q, rk, t0, n);
    stage<D, L::LQ>(K, (const T *)jb.k, rk, t0, n);
    stage<DV, DV>(V, (const T *)jb.v, rv, t0, n);
    __syncthreads();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;   // rows 4 ty ..; scores of columns tx + 16 c
    float s[4][4] = {};
#pragma unroll 2
    for (int a = 0; a < D; a += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4 *>(Q + (4 * ty + r) * L::LQ + a);
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const float4 *>(K + (tx + 16 * c) * L::LQ + a);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                s[r][c] = fmaf(x[r].x, y[c].x, fmaf(x[r].y, y[c].y, fmaf(x[r].z, y[c].z, fmaf(x[r].w, y[c].w, s[r][c]))));
    }
    __syncthreads();   // K has been read
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 4 * ty + r, j = tx + 16 * c, e = rev ? j - i : i - j;
            P[i * L::LP + j] = e >= 0 ? s[r][c] * pw[e] : 0.f;
        }
    griddep_wait();   // the states
    // the state's part, rows of S staged where K was
    const float *S0 = jb.states ? jb.states + (size_t)unit * D * DV : jb.S_in ? jb.S_in + (size_t)bh * D * DV : nullptr;
    float acc[4][C];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = 0.f;
    if (S0) {
#pragma unroll 1
        for (int a0 = 0; a0 < D; a0 += L::SR) {
            __syncthreads();
            for (int e = threadIdx.x; e < L::SR * DV; e += kRThr)
                S[e] = trans ? S0[(size_t)(e % DV) * D + a0 + e / DV] : S0[(size_t)a0 * DV + e];
            __syncthreads();
#pragma unroll 2
            for (int a = 0; a < L::SR; a += 4) four<C, false>(acc, Q + 4 * ty * L::LQ + a0 + a, L::LQ, S + a * DV, DV, tx, rev);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int e = inter_exp(rev, 4 * ty + r, n);
            const float f = e >= 0 ? pw[e] : 0.f;   // none: behind the last token
#pragma unroll
            for (int c = 0; c < C; ++c) acc[r][c] *= f;
        }
    }
    __syncthreads();
    const int d0 = 4 * ty;   // the four columns on the diagonal
#pragma unroll 2
    for (int j = rev ? d0 + 4 : 0; j < (rev ? kRC : d0); j += 4) four<C, false>(acc, P + d0 * L::LP + j, L::LP, V + j * DV, DV, tx, rev);
    if (rev) four<C, true>(acc, P + d0 * L::LP + d0, L::LP, V + d0 * DV, DV, tx, true);
    else four<C, true>(acc, P + d0 * L::LP + d0, L::LP, V + d0 * DV, DV, tx, false);
    T *y = (T *)jb.y;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * ty + r < n)
#pragma unroll
            for (int c = 0; c < C; ++c) y[rv.at(t0 + 4 * ty + r) + CC::at(tx, c)] = from_f<T>(acc[r][c]);
}

int blocks_of(int N) { return (N + kRC - 1) / kRC; }
// One block, and no final state asked for: y comes from S_in itself.
bool needs_states(const RetainArgs &a) { return a.N > kRC || a.S_out; }

RetainSimt simt_params(const RetainArgs &a) {
    RetainSimt p{};
    p.gamma = a.gamma; p.H = a.H; p.N = a.N; p.layout = a.layout; p.nblk = blocks_of(a.N); p.heads = a.B * a.H;
    p.tokens = kRC;
    return p;
}

// Launches of `jobs` jobs; their units are fewer than tokens, which fit 31 bits.
template <int D, int DV, typename T> struct Launch {
    static cudaError_t sums(const RetainSimt &p, int jobs, cudaStream_t s) {
        constexpr int smem = 4 * kRC * (D + DV);
        cudaError_t e = cudaFuncSetAttribute(retain_sums_kernel<D, DV, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        retain_sums_kernel<D, DV, T><<<(unsigned)jobs * p.heads * p.nblk, kRThr, smem, s>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        return launch_overlapped(retain_scan_kernel, dim3((unsigned)jobs * p.heads * (D * DV / 4 / kScanThr)), dim3(kScanThr), 0, s, p, D, DV);
    }
    // behind: launched right behind the scan, and so early
    static cudaError_t out(const RetainSimt &p, int jobs, bool behind, cudaStream_t s) {
        constexpr int smem = OutLay<D, DV, T>::bytes;
        cudaError_t e = cudaFuncSetAttribute(retain_out_kernel<D, DV, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        const dim3 grid((unsigned)jobs * p.heads * p.nblk);
        if (behind) return launch_overlapped(retain_out_kernel<D, DV, T>, grid, dim3(kRThr), smem, s, p);
        retain_out_kernel<D, DV, T><<<grid, kRThr, smem, s>>>(p);
        return cudaGetLastError();
    }
};

struct Forward {
    template <int D, int DV, typename T> static cudaError_t run(const RetainArgs &a, const RetainGrads &) {
        RetainSimt p = simt_params(a);
        Job &jb = p.job[0];
        jb = {a.q, a.k, a.v, a.y, a.S_in, a.S_out, nullptr, false, false};
        if (needs_states(a)) {
            jb.states = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
            const cudaError_t e = Launch<D, DV, T>::sums(p, 1, a.stream);
            if (e != cudaSuccess) return e;
        }
        return Launch<D, DV, T>::out(p, 1, jb.states != nullptr, a.stream);
    }
};

// The states S (for grad_q) and, from behind, G (for grad_k and grad_v) together, then the three gradients: those whose
// rows are d wide, and grad_v, in one launch if d = dv.
struct Grads {
    template <int D, int DV, typename T> static cudaError_t run(const RetainArgs &a, const RetainGrads &g) {
        RetainSimt p = simt_params(a);
        float *S = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader)), *G = S + (size_t)p.heads * p.nblk * D * DV;
        p.job[0] = {nullptr, a.k, a.v, nullptr, a.S_in, nullptr, S, false, false};
        p.job[1] = {nullptr, a.q, g.dy, nullptr, g.dS_out, g.dS_in, G, true, false};
        cudaError_t e = Launch<D, DV, T>::sums(p, 2, a.stream);
        if (e != cudaSuccess) return e;
        p.job[0] = {g.dy, a.v, a.k, g.dq, nullptr, nullptr, S, false, true};
        p.job[1] = {a.v, g.dy, a.q, g.dk, nullptr, nullptr, G, true, true};
        p.job[2] = {a.k, a.q, g.dy, g.dv, nullptr, nullptr, G, true, false};
        if (D == DV) return Launch<DV, D, T>::out(p, 3, true, a.stream);
        if ((e = Launch<DV, D, T>::out(p, 2, true, a.stream)) != cudaSuccess) return e;
        p.job[0] = p.job[2];
        return Launch<D, DV, T>::out(p, 1, false, a.stream);
    }
};

template <typename K, int D, typename T> cudaError_t by_dv(const RetainArgs &a, const RetainGrads &g) {
    switch (a.dv) {
    case 32: return K::template run<D, 32, T>(a, g);
    case 64: return K::template run<D, 64, T>(a, g);
    case 128: return K::template run<D, 128, T>(a, g);
    }
    return cudaErrorInvalidValue;
}
template <typename K, typename T> cudaError_t by_d(const RetainArgs &a, const RetainGrads &g) {
    switch (a.d) {
    case 32: return by_dv<K, 32, T>(a, g);
    case 64: return by_dv<K, 64, T>(a, g);
    case 128: return by_dv<K, 128, T>(a, g);
    }
    return cudaErrorInvalidValue;
}
template <typename K> cudaError_t by_type(const RetainArgs &a, const RetainGrads &g) {
    return a.dt == LA_DTYPE_BF16 ? by_d<K, __nv_bfloat16>(a, g) : by_d<K, float>(a, g);
}

}  // namespace

size_t retain_simt_workspace(const RetainArgs &a, bool grads) {
    const size_t one = (size_t)a.B * a.H * blocks_of(a.N) * a.d * a.dv * 4;
    return grads ? 2 * one : needs_states(a) ? one : 0;
}
cudaError_t launch_retain_scan(const RetainArgs &a, float *states, int blocks, int tokens) {
    RetainSimt p = simt_params(a);
    p.job[0] = {nullptr, nullptr, nullptr, nullptr, a.S_in, a.S_out, states, a.rev, a.trans};
    p.nblk = blocks; p.tokens = tokens;
    return launch_overlapped(retain_scan_kernel, dim3((unsigned)p.heads * (a.d * a.dv / 4 / kScanThr)), dim3(kScanThr), 0, a.stream, p,
                             a.d, a.dv);
}
cudaError_t launch_retain_simt(const RetainArgs &a) { return by_type<Forward>(a, RetainGrads{}); }
cudaError_t launch_retain_grads_simt(const RetainArgs &a, const RetainGrads &g) { return by_type<Grads>(a, g); }

}  // namespace la
