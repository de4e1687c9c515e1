// retention.cuh -- what the kernels of retention share.
//
//   S_t = gamma S_{t-1} + k_t v_t^T,   y_t = S_t^T q_t     (per head, S [d, dv] in float32)
//
// by blocks of tokens, S the state before a block of L tokens:
//   y_i = sum_{j <= i} gamma^(i-j) (q_i . k_j) v_j + gamma^(i+1) S^T q_i,
//   S'  = gamma^L S + sum_j gamma^(L-1-j) k_j v_j^T.
// From behind (rev), with the state G behind a block already decayed up to it:
//   y_i = sum_{j >= i} gamma^(j-i) (q_i . k_j) v_j + gamma^(L-1-i) G^T q_i,
//   G'  = gamma^L G + sum_j gamma^(j+1) k_j v_j^T.
#pragma once

#include "delta_common.cuh"

namespace la {

// Exponents of the state's part of y_i and of key j's part of the next state.
__host__ __device__ __forceinline__ int inter_exp(bool rev, int i, int L) { return rev ? L - 1 - i : i + 1; }
__host__ __device__ __forceinline__ int key_exp(bool rev, int j, int L) { return rev ? j + 1 : L - 1 - j; }

// gamma^n (n >= 0) by squarings of float32 pairs, so that a power is off by little more than its one
// rounding; 1 for n = 0, gamma = 0 among them.
__device__ __forceinline__ F2 f2prod(F2 a, F2 b) {
    const float p = __fmul_rn(a.h, b.h), e = fmaf(a.h, b.h, -p);
    const float l = fmaf(a.h, b.l, fmaf(a.l, b.h, e)), h = __fadd_rn(p, l);
    return {h, __fsub_rn(l, __fsub_rn(h, p))};
}
__device__ __forceinline__ float gamma_power(float gamma, int n) {
    F2 r = {1.f, 0.f}, x = {gamma, 0.f};
    for (; n > 0; n >>= 1) {
        if (n & 1) r = f2prod(r, x);
        x = f2prod(x, x);
    }
    return r.h;
}

}  // namespace la
