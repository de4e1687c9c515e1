// retention_step.cu -- one token of retention per head, on the float32 state.
//
//   S' = gamma S + k v^T,   y = S'^T q
//
// Bound by HBM: S is read once and written once (8 d dv bytes a head).  The CTA, its rows and columns are
// those of the delta rule's step: 8 warps own d/8 rows each, a lane dv/32 contiguous columns, all loads of
// a warp in flight before the first is used; the column sums of y are joined through shared memory.
#include "retention.cuh"

namespace la {
namespace {

constexpr int kWarps = 8;

template <int VEC> struct Lane {   // VEC contiguous floats
    float x[VEC];
    __device__ __forceinline__ void load(const float *p) {
        if (VEC == 4) {
            const float4 t = __ldcs(reinterpret_cast<const float4 *>(p));
            x[0] = t.x; x[1 % VEC] = t.y; x[2 % VEC] = t.z; x[3 % VEC] = t.w;
        } else if (VEC == 2) {
            const float2 t = __ldcs(reinterpret_cast<const float2 *>(p));
            x[0] = t.x; x[1 % VEC] = t.y;
        } else {
            x[0] = __ldcs(p);
        }
    }
    __device__ __forceinline__ void store(float *p) const {
        if (VEC == 4) __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1 % VEC], x[2 % VEC], x[3 % VEC]));
        else if (VEC == 2) __stcs(reinterpret_cast<float2 *>(p), make_float2(x[0], x[1 % VEC]));
        else __stcs(p, x[0]);
    }
};

// S_in and S_out may be the same buffer: a head's rows are read before they are written, by the
// same threads.
template <int D, int DV, typename T>
__global__ void __launch_bounds__(kWarps * 32)
retain_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, T *__restrict__ y,
                   const float *__restrict__ gamma, const float *S_in, float *S_out, int H) {
    constexpr int RPW = D / kWarps, VEC = DV / 32;
    __shared__ float qs[D], ks[D];
    __shared__ float part[kWarps][DV];
    const int bh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t at = ((size_t)bh * D + warp * RPW) * DV + lane * VEC;
    Lane<VEC> s[RPW];
#pragma unroll
    for (int r = 0; r < RPW; ++r) s[r].load(S_in + at + (size_t)r * DV);
    if (tid < D) {
        qs[tid] = to_f(q[(size_t)bh * D + tid]);
        ks[tid] = to_f(k[(size_t)bh * D + tid]);
    }
    const float g = gamma[bh % H];
    float vv[VEC], sum[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
        vv[c] = to_f(v[(size_t)bh * DV + lane * VEC + c]);
        sum[c] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        const float kr = ks[warp * RPW + r], qr = qs[warp * RPW + r];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
            s[r].x[c] = fmaf(g, s[r].x[c], kr * vv[c]);
            sum[c] = fmaf(qr, s[r].x[c], sum[c]);
        }
        s[r].store(S_out + at + (size_t)r * DV);
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) part[warp][lane * VEC + c] = sum[c];
    __syncthreads();
    if (tid < DV) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += part[w][tid];
        y[(size_t)bh * DV + tid] = from_f<T>(x);
    }
}

template <int D, int DV, typename T> cudaError_t launch_t(const RetainArgs &a) {
    retain_step_kernel<D, DV, T><<<a.B * a.H, kWarps * 32, 0, a.stream>>>(
        (const T *)a.q, (const T *)a.k, (const T *)a.v, (T *)a.y, a.gamma, a.S_in, a.S_out, a.H);
    return cudaGetLastError();
}
template <int D, typename T> cudaError_t launch_d(const RetainArgs &a) {
    switch (a.dv) {
    case 32: return launch_t<D, 32, T>(a);
    case 64: return launch_t<D, 64, T>(a);
    case 128: return launch_t<D, 128, T>(a);
    }
    return cudaErrorInvalidValue;
}
template <typename T> cudaError_t launch(const RetainArgs &a) {
    switch (a.d) {
    case 32: return launch_d<32, T>(a);
    case 64: return launch_d<64, T>(a);
    case 128: return launch_d<128, T>(a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_retain_step(const RetainArgs &a) {
    return a.dt == LA_DTYPE_BF16 ? launch<__nv_bfloat16>(a) : launch<float>(a);
}

}  // namespace la
