// delta_step.cu -- one token of the gated delta rule per head, on the float32 state.
//
//   u = b (v - a S^T k),  S' = a S + k u^T,  y = S'^T q = a S^T q + (k . q) u
//
// Bound by HBM: S is read once and written once (8 d dv bytes a head), and
// the second form of y needs no second pass over it.  The CTA, its rows and
// columns are those of the linear-attention step (decode.cu): 8 warps own d/8
// rows each, a lane dv/32 contiguous columns; all loads of a warp are in
// flight before the first is used, S stays in registers between the two
// column sums (S^T k and S^T q, joined through shared memory) and the update.
#include "delta_common.cuh"

namespace la {
namespace {

constexpr int kWarps = 8;

template <int VEC> struct Row;
template <> struct Row<1> { float x[1]; };
template <> struct Row<2> { float x[2]; };
template <> struct Row<4> { float x[4]; };
__device__ __forceinline__ void ld(Row<1> &r, const float *p) { r.x[0] = __ldcs(p); }
__device__ __forceinline__ void ld(Row<2> &r, const float *p) {
    const float2 t = __ldcs(reinterpret_cast<const float2 *>(p));
    r.x[0] = t.x; r.x[1] = t.y;
}
__device__ __forceinline__ void ld(Row<4> &r, const float *p) {
    const float4 t = __ldcs(reinterpret_cast<const float4 *>(p));
    r.x[0] = t.x; r.x[1] = t.y; r.x[2] = t.z; r.x[3] = t.w;
}
__device__ __forceinline__ void stv(const Row<1> &r, float *p) { __stcs(p, r.x[0]); }
__device__ __forceinline__ void stv(const Row<2> &r, float *p) {
    __stcs(reinterpret_cast<float2 *>(p), make_float2(r.x[0], r.x[1]));
}
__device__ __forceinline__ void stv(const Row<4> &r, float *p) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(r.x[0], r.x[1], r.x[2], r.x[3]));
}

// S_in and S_out may be the same buffer: a head's rows are read before they are written, by the
// same threads.
template <int D, int DV, typename T>
__global__ void __launch_bounds__(kWarps * 32)
delta_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                  T *__restrict__ y, const float *__restrict__ beta, const float *__restrict__ lg,
                  const float *S_in, float *S_out, int H, int Hk) {
    constexpr int RPW = D / kWarps, VEC = DV / 32;
    __shared__ float qs[D], ks[D];
    __shared__ float pk[kWarps][DV], pq[kWarps][DV];
    const int bh = blockIdx.x, key = bh / H * Hk + (bh % H) / (H / Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float *src = S_in + ((size_t)bh * D + warp * RPW) * DV + lane * VEC;
    float *dst = S_out + ((size_t)bh * D + warp * RPW) * DV + lane * VEC;

    Row<VEC> s[RPW];
#pragma unroll
    for (int r = 0; r < RPW; ++r) ld(s[r], src + (size_t)r * DV);
    if (tid < D) {
        qs[tid] = to_f(q[(size_t)key * D + tid]);
        ks[tid] = to_f(k[(size_t)key * D + tid]);
    }
    const float a = lg ? expf(lg[bh]) : 1.f, b = beta[bh];
    float vv[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) vv[c] = to_f(v[(size_t)bh * DV + lane * VEC + c]);
    __syncthreads();

    float ak[VEC], aq[VEC], kq = 0.f;
#pragma unroll
    for (int c = 0; c < VEC; ++c) ak[c] = aq[c] = 0.f;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const float kr = ks[warp * RPW + r], qr = qs[warp * RPW + r];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            s[r].x[c] *= a;
            ak[c] = fmaf(kr, s[r].x[c], ak[c]);
            aq[c] = fmaf(qr, s[r].x[c], aq[c]);
        }
    }
    for (int i = lane; i < D; i += 32) kq = fmaf(ks[i], qs[i], kq);
    kq = warp_sum(kq);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        pk[warp][lane * VEC + c] = ak[c];
        pq[warp][lane * VEC + c] = aq[c];
    }
    __syncthreads();
    float u[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += pk[w][lane * VEC + c];
        u[c] = b * (vv[c] - x);
    }
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const float kr = ks[warp * RPW + r];
#pragma unroll
        for (int c = 0; c < VEC; ++c) s[r].x[c] = fmaf(kr, u[c], s[r].x[c]);
        stv(s[r], dst + (size_t)r * DV);
    }
    if (warp == 0) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x += pq[w][lane * VEC + c];
            y[(size_t)bh * DV + lane * VEC + c] = from_f<T>(fmaf(kq, u[c], x));
        }
    }
}

template <int D, int DV, typename T> cudaError_t launch_t(const DeltaArgs &a) {
    delta_step_kernel<D, DV, T><<<a.B * a.H, kWarps * 32, 0, a.stream>>>(
        (const T *)a.q, (const T *)a.k, (const T *)a.v, (T *)a.y, a.beta, a.log_gate, a.S_in, a.S_out,
        a.H, a.Hk);
    return cudaGetLastError();
}
template <int D, typename T> cudaError_t launch_d(const DeltaArgs &a) {
    switch (a.dv) {
    case 32: return launch_t<D, 32, T>(a);
    case 64: return launch_t<D, 64, T>(a);
    case 128: return launch_t<D, 128, T>(a);
    }
    return cudaErrorInvalidValue;
}
template <typename T> cudaError_t launch(const DeltaArgs &a) {
    switch (a.d) {
    case 32: return launch_d<32, T>(a);
    case 64: return launch_d<64, T>(a);
    case 128: return launch_d<128, T>(a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a) {
    return a.dt == LA_DTYPE_BF16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace la
