// delta_grad.cu -- gradients of the gated delta rule: what follows the two
// recurrent passes, all blocks of 64 tokens at once, in float32.
//
// With the state S before a block and its gradient G after it, e and du of
// its tokens (from the recurrent passes), c_i the product of the block's
// gates up to token i and D_ij = c_i / c_j, u_j = b_j e_j:
//   dq_i = c_i S dy_i + sum_{j<=i} D_ij (dy_i . u_j) k_j
//   dk_j = D_Cj G u_j - b_j c_j S du_j + sum_{i>=j} D_ij (dy_i . u_j) q_i
//          - sum_{i>j} b_i D_ij (du_i . u_j) k_i - sum_{i<j} b_j D_ji (du_j . u_i) k_i
//   dv_j = b_j du_j,   db_j = du_j . e_j
//   dlog a_j = <G, S'> + sum_{i>=j} (q_i . dq_i - v_i . dv_i)
// (S' the state after the block; the last line holds because scaling the
// state after token j scales what every later token reads of it, and what
// the block hands on).
//
// A CTA takes one block of one key head, sums over that head's value heads
// in registers and writes dq and dk once.  512 threads, a warp for each 4 tokens
// (its factors of the products are broadcasts), lanes along the features: bound
// by the latency of the staged slices, which 16 warps cover better than 8
// (B8 H16 N512 d64 float32: 473 us for the gradients, 568 with 256 threads; at d = 128 up to 152 bytes a thread spill).  The
// gates' sums run as float32 pairs in one warp: 64-bit additions by one thread
// were a quarter of the kernel's time.
#include "delta_common.cuh"

namespace la {
namespace {

constexpr int kThr = 512;
constexpr int kSl = 16;        // dv slice staged at a time
constexpr int kP = kDeltaC + 4;   // padded row of the transposed stages

struct GradParams {
    const void *q, *k, *v, *dy;
    const float *beta, *lg;
    void *dq, *dk, *dvg;
    float *dbeta, *dlg;
    const float *S_ck, *G_ck, *e, *du;
    int H, Hk, N, dv, layout;
};

template <int D> struct GradSmem {
    // transposed stages of a dv slice: [slice][token] and [slice][feature]
    float dyT[kSl][kP], eT[kSl][kP], duT[kSl][kP];
    float ST[kSl][D + 4], GT[kSl][D + 4];
    float P[kDeltaC][kDeltaC + 1];    // D_ij (dy_i . u_j), j <= i
    float F[kDeltaC][kDeltaC + 1];    // -b_i D_ij (du_i . u_j), j < i, mirrored
    float rows[kSl][D + 4], rows2[kSl][D + 4];
    float c[kDeltaC], cC[kDeltaC], b[kDeltaC], hi[kDeltaC], lo[kDeltaC];
    float qdq[kDeltaC], vdv[kDeltaC], db[kDeltaC];
    float red[kThr / 32];
};

template <int D, typename T>
__global__ void __launch_bounds__(kThr, D == 32 ? 2 : 1) delta_grad_kernel(const GradParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<D> &s = *reinterpret_cast<GradSmem<D> *>(raw);
    constexpr int CW = D / 32;   // features of a thread: 4 tokens x CW
    const int tid = threadIdx.x, ti = tid >> 5, tj = tid & 31;   // tokens 4 ti.., features tj + 32 j
    const int nc = delta_blocks(p.N), blk = blockIdx.x % nc, t0 = blk * kDeltaC;
    const int bk = blockIdx.x / nc, b = bk / p.Hk, hk = bk % p.Hk, group = p.H / p.Hk;
    const int n = min(kDeltaC, p.N - t0);
    const size_t st = (size_t)D * p.dv;
    const TokenRows rk = token_rows(p.layout, b, hk, p.Hk, p.N, D);
    const T *q = (const T *)p.q, *k = (const T *)p.k, *v = (const T *)p.v, *dy = (const T *)p.dy;

    float dq[4][CW], dk[4][CW];   // sums over the value heads
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < CW; ++j) dq[i][j] = dk[i][j] = 0.f;

    for (int g = 0; g < group; ++g) {
        const int h = hk * group + g;
        const size_t bh = (size_t)b * p.H + h;
        const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, p.dv);
        const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
        const float *S0 = p.S_ck + (bh * (nc + 1) + blk) * st, *S1 = S0 + st;
        const float *G1 = p.G_ck + (bh * nc + blk) * st;
        __syncthreads();
        // running sums of the log gates as pairs hi + lo, so that differences of two of them keep
        // their precision behind a nearly closed gate; one warp, two tokens a lane
        if (tid < 32) {
            F2 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // exp(-1e4) is 0; keeps -inf out
                const int t = 2 * tid + i;
                const float v = t < n && p.lg ? p.lg[rs.at(t0 + t)] : 0.f;
                x[i] = {v < -1e4f ? -1e4f : v, 0.f};
            }
            x[1] = f2sum2(x[0], x[1]);
            F2 sum = x[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const F2 y = {__shfl_up_sync(0xffffffffu, sum.h, o), __shfl_up_sync(0xffffffffu, sum.l, o)};
                if (tid >= o) sum = f2sum2(y, sum);
            }
            F2 before = {__shfl_up_sync(0xffffffffu, sum.h, 1), __shfl_up_sync(0xffffffffu, sum.l, 1)};
            if (tid == 0) before = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const F2 y = f2sum2(before, x[i]);
                s.hi[2 * tid + i] = y.h;
                s.lo[2 * tid + i] = y.l;
            }
        }
        if (tid < kDeltaC) {
            s.b[tid] = tid < n ? p.beta[rs.at(t0 + tid)] : 0.f;
            s.vdv[tid] = s.db[tid] = 0.f;
        }
        __syncthreads();
        auto decay = [&](int i, int j) { return expf((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j])); };
        if (tid < kDeltaC) {
            s.c[tid] = expf(s.hi[tid] + s.lo[tid]);
            s.cC[tid] = decay(n - 1, tid);
        }

        float P[4][2], F[4][2], aq[4][CW], ak[4][CW], as[4][CW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) P[i][j] = F[i][j] = 0.f;
#pragma unroll
            for (int j = 0; j < CW; ++j) aq[i][j] = ak[i][j] = as[i][j] = 0.f;
        }
        float gs = 0.f;   // <G, S'>
        for (int c0 = 0; c0 < p.dv; c0 += kSl) {
            __syncthreads();
            for (int i = tid; i < kDeltaC * kSl; i += kThr) {
                const int t = i / kSl, c = i % kSl;
                float x = 0.f, e = 0.f, du = 0.f;
                if (t < n) {
                    x = to_f(dy[rv.at(t0 + t) + c0 + c]);
                    e = p.e[(bh * p.N + t0 + t) * p.dv + c0 + c];
                    du = p.du[(bh * p.N + t0 + t) * p.dv + c0 + c];
                }
                s.dyT[c][t] = x; s.eT[c][t] = e; s.duT[c][t] = du;
                if (t < n) ((T *)p.dvg)[rv.at(t0 + t) + c0 + c] = from_f<T>(s.b[t] * du);
                float db = e * du;
                float vd = t < n && p.lg ? s.b[t] * du * to_f(v[rv.at(t0 + t) + c0 + c]) : 0.f;
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    db += __shfl_xor_sync(0xffffffffu, db, o);
                    vd += __shfl_xor_sync(0xffffffffu, vd, o);
                }
                if (c == 0) { s.db[t] += db; s.vdv[t] += vd; }
            }
            for (int i = tid; i < D * kSl; i += kThr) {
                const int r = i / kSl, c = i % kSl;
                const size_t o = (size_t)r * p.dv + c0 + c;
                const float gg = G1[o];
                s.ST[c][r] = S0[o];
                s.GT[c][r] = gg;
                if (p.lg) gs = fmaf(gg, S1[o], gs);
            }
            __syncthreads();
#pragma unroll 4
            for (int c = 0; c < kSl; ++c) {
                const float4 y4 = *reinterpret_cast<const float4 *>(&s.dyT[c][4 * ti]);
                const float4 d4 = *reinterpret_cast<const float4 *>(&s.duT[c][4 * ti]);
                const float4 e4 = *reinterpret_cast<const float4 *>(&s.eT[c][4 * ti]);
                const float2 f2 = *reinterpret_cast<const float2 *>(&s.eT[c][2 * tj]);
                const float yi[4] = {y4.x, y4.y, y4.z, y4.w}, di[4] = {d4.x, d4.y, d4.z, d4.w};
                const float ei[4] = {e4.x, e4.y, e4.z, e4.w}, ej[2] = {f2.x, f2.y};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        P[i][j] = fmaf(yi[i], ej[j], P[i][j]);
                        F[i][j] = fmaf(di[i], ej[j], F[i][j]);
                    }
#pragma unroll
                for (int j = 0; j < CW; ++j) {
                    const float S = s.ST[c][tj + 32 * j], G = s.GT[c][tj + 32 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        aq[i][j] = fmaf(yi[i], S, aq[i][j]);
                        ak[i][j] = fmaf(ei[i], G, ak[i][j]);
                        as[i][j] = fmaf(di[i], S, as[i][j]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ii = 4 * ti + i;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int jj = 2 * tj + j;
                const float w = jj <= ii ? decay(ii, jj) * s.b[jj] : 0.f;
                s.P[ii][jj] = w * P[i][j];
                if (jj <= ii) {
                    const float f = jj < ii ? -s.b[ii] * w * F[i][j] : 0.f;
                    s.F[ii][jj] = f;
                    s.F[jj][ii] = f;
                }
            }
            const float c = s.c[ii], ce = s.cC[ii] * s.b[ii], cs = -s.b[ii] * c;
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                aq[i][j] *= c;
                dk[i][j] += fmaf(ce, ak[i][j], cs * as[i][j]);
            }
        }
        // dq += P K, dk += P^T Q + F K over the block's tokens, a slice of them at a time
        for (int j0 = 0; j0 < kDeltaC; j0 += kSl) {
            __syncthreads();
            for (int i = tid; i < kSl * D; i += kThr) {
                const int t = i / D, f = i % D;
                const bool in = j0 + t < n;
                s.rows[t][f] = in ? to_f(k[rk.at(t0 + j0 + t) + f]) : 0.f;
                s.rows2[t][f] = in ? to_f(q[rk.at(t0 + j0 + t) + f]) : 0.f;
            }
            __syncthreads();
#pragma unroll 4
            for (int t = 0; t < kSl; ++t) {
                float a0[4], a1[4], a2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a0[i] = s.P[4 * ti + i][j0 + t];
                    a1[i] = s.P[j0 + t][4 * ti + i];
                    a2[i] = s.F[4 * ti + i][j0 + t];
                }
#pragma unroll
                for (int j = 0; j < CW; ++j) {
                    const float kx = s.rows[t][tj + 32 * j], qx = s.rows2[t][tj + 32 * j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        aq[i][j] = fmaf(a0[i], kx, aq[i][j]);
                        dk[i][j] = fmaf(a1[i], qx, fmaf(a2[i], kx, dk[i][j]));
                    }
                }
            }
        }
        if (p.lg) {   // q . dq of this value head, <G, S'>
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + 4 * ti + i;
                float x = 0.f;
                if (t < p.N)
#pragma unroll
                    for (int j = 0; j < CW; ++j) x = fmaf(to_f(q[rk.at(t) + tj + 32 * j]), aq[i][j], x);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (tj == 0) s.qdq[4 * ti + i] = x;
            }
            gs = warp_sum(gs);
            if ((tid & 31) == 0) s.red[tid >> 5] = gs;
        }
        __syncthreads();
        if (tid < n) p.dbeta[rs.at(t0 + tid)] = s.db[tid];
        if (p.lg && tid < 32) {   // running sums from the block's end, two tokens a lane
            F2 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // q . dq - v . dv, exactly
                const int t = 2 * tid + i;
                const float qd = t < n ? s.qdq[t] : 0.f, vd = t < n ? s.vdv[t] : 0.f, d = qd - vd, z = d - qd;
                x[i] = {d, (qd - (d - z)) - (vd + z)};
            }
            const float e = warp_sum(tid < kThr / 32 ? s.red[tid] : 0.f);
            x[0] = f2sum2(x[0], x[1]);
            F2 sum = x[0];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const F2 y = {__shfl_down_sync(0xffffffffu, sum.h, o), __shfl_down_sync(0xffffffffu, sum.l, o)};
                if (tid + o < 32) sum = f2sum2(sum, y);
            }
            F2 after = {__shfl_down_sync(0xffffffffu, sum.h, 1), __shfl_down_sync(0xffffffffu, sum.l, 1)};
            if (tid == 31) after = {0.f, 0.f};
            const F2 end = {e, 0.f}, first = f2sum2(end, sum), second = f2sum2(end, f2sum2(after, x[1]));
            if (2 * tid < n) p.dlg[rs.at(t0 + 2 * tid)] = first.h + first.l;
            if (2 * tid + 1 < n) p.dlg[rs.at(t0 + 2 * tid + 1)] = second.h + second.l;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CW; ++j) dq[i][j] += aq[i][j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * ti + i;
        if (t >= n) continue;
#pragma unroll
        for (int j = 0; j < CW; ++j) {
            ((T *)p.dq)[rk.at(t0 + t) + tj + 32 * j] = from_f<T>(dq[i][j]);
            ((T *)p.dk)[rk.at(t0 + t) + tj + 32 * j] = from_f<T>(dk[i][j]);
        }
    }
}

template <int D, typename T> cudaError_t launch_grad(const DeltaArgs &a) {
    const DeltaBwdWs w = delta_bwd_ws(a);
    const GradParams p{a.q, a.k, a.v, a.dy, a.beta, a.log_gate, a.dq, a.dk, a.dv_grad, a.dbeta, a.dlog_gate,
                       w.S, w.G, w.e, w.du, a.H, a.Hk, a.N, a.dv, (int)a.layout};
    const size_t smem = sizeof(GradSmem<D>);
    cudaError_t e = cudaFuncSetAttribute(delta_grad_kernel<D, T>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    delta_grad_kernel<D, T><<<(unsigned)delta_blocks(a.N) * a.B * a.Hk, kThr, smem, a.stream>>>(p);
    return cudaGetLastError();
}
template <typename T> cudaError_t launch_grad_t(const DeltaArgs &a) {
    switch (a.d) {
    case 32: return launch_grad<32, T>(a);
    case 64: return launch_grad<64, T>(a);
    case 128: return launch_grad<128, T>(a);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

size_t delta_backward_workspace(const DeltaArgs &a) {
    const size_t BH = (size_t)a.B * a.H, nc = delta_blocks(a.N), st = (size_t)a.d * a.dv;
    return sizeof(WsHeader) + 4 * (BH * (2 * nc + 1) * st + 2 * BH * a.N * a.dv +
                                   (delta_tc_supported(a) ? delta_tc_split_floats(a) : 0));
}

cudaError_t launch_delta_backward(const DeltaArgs &a) {
    if (delta_tc_supported(a)) {
        const cudaError_t e = launch_delta_passes_tc(a);
        return e == cudaSuccess ? launch_delta_grad_tc(a) : e;
    }
    cudaError_t e = launch_delta_states_simt(a);
    if (e == cudaSuccess) e = launch_delta_reverse_simt(a);
    if (e != cudaSuccess) return e;
    return a.dt == LA_DTYPE_BF16 ? launch_grad_t<__nv_bfloat16>(a) : launch_grad_t<float>(a);
}

}  // namespace la
