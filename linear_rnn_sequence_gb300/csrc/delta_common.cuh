// delta_common.cuh -- what the kernels of the gated delta rule share.
//
// The recurrence, per head, with the state S [d, dv] in float32:
//   e_t = v_t - a_t S_{t-1}^T k_t,   S_t = a_t S_{t-1} + k_t (b_t e_t)^T,   y_t = S_t^T q_t
// (a_t = exp(log_gate_t); the same update as a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_device.cuh"
#include "la_internal.h"

namespace la {

constexpr int kDeltaC = 64;   // tokens of a block: the distance of the states the backward keeps

// Token rows of one head: row t starts at base + t * step (elements).
struct TokenRows {
    size_t base, step;
    __device__ __forceinline__ size_t at(int t) const { return base + (size_t)t * step; }
};
__host__ __device__ __forceinline__ TokenRows token_rows(int layout, int b, int h, int heads, int N,
                                                         int w) {
    if (layout == LA_LAYOUT_BNHD)
        return {((size_t)b * N * heads + h) * w, (size_t)heads * w};
    return {((size_t)b * heads + h) * N * w, (size_t)w};
}

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// A float32 pair h + l, |l| at most half a step of h: sums keep about 46 bits.  The _rn forms are not
// contracted: where h is a product, a fused multiply-add would bring its low part in a second time.
struct F2 {
    float h, l;
};
__device__ __forceinline__ F2 f2sum2(F2 a, F2 b) {
    const float s = __fadd_rn(a.h, b.h), t = __fsub_rn(s, a.h);
    const float l = __fadd_rn(__fadd_rn(__fsub_rn(a.h, __fsub_rn(s, t)), __fsub_rn(b.h, t)), __fadd_rn(a.l, b.l));
    const float h = __fadd_rn(s, l);
    return {h, __fsub_rn(l, __fsub_rn(h, s))};
}

// Workspace of the gradients, in floats behind the status header: the states before each block and
// the final one, their gradients after each block, e and du of every token (head-major), and what
// a split of the sequence takes.
struct DeltaBwdWs {
    float *S, *G, *e, *du, *split;
};
__host__ __device__ __forceinline__ int delta_blocks(int N) { return (N + kDeltaC - 1) / kDeltaC; }
inline DeltaBwdWs delta_bwd_ws(const DeltaArgs &a) {
    const size_t BH = (size_t)a.B * a.H, nc = delta_blocks(a.N), st = (size_t)a.d * a.dv;
    DeltaBwdWs w;
    w.S = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
    w.G = w.S + BH * (nc + 1) * st;
    w.e = w.G + BH * nc * st;
    w.du = w.e + BH * a.N * a.dv;
    w.split = w.du + BH * a.N * a.dv;
    return w;
}

}  // namespace la
