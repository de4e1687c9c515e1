// norm_rotate.cu -- queries and keys normed by head, weighted and rotated by position, in one pass
// (norm_rotate.cuh says how a row lies in the lanes).
//
// Bound by HBM: each value is read once and written once, and stays in registers between.
#include "norm_rotate.cuh"

namespace la {
namespace {

template <typename T, int VEC, int LPR, int CP, bool ADJ>
__global__ void __launch_bounds__(kRotThreads) norm_rotate_kernel(const RotParams p) {
    using Ch = Chunk<T, VEC>;
    using Raw = typename Ch::Raw;
    constexpr int U = CP > 1 ? 2 : 4;   // heads in flight
    const int gl = threadIdx.x % LPR, part = blockIdx.y;
    const long long at = (long long)blockIdx.x * (kRotThreads / LPR) + threadIdx.x / LPR;
    const bool live = at < p.tokens;
    const long long tok = live ? at : p.tokens - 1;
    const bool second = part >= p.side[0].parts;
    const RotSide sd = second ? p.side[1] : p.side[0];
    const int h0 = (second ? part - p.side[0].parts : part) * p.span, h1 = min(sd.heads, h0 + p.span);
    const long long b = tok / p.N;
    const int n = (int)(tok - b * p.N);

    Place<VEC, CP, ADJ> pl;
    pl.template init<LPR>(p, gl);
    const T *x = static_cast<const T *>(sd.x.p) + b * sd.x.b + n * sd.x.t;
    T *y = static_cast<T *>(sd.y.p) + b * sd.y.b + n * sd.y.t;
    Raw ra[U][CP], rb[U][CP];
    auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                ra[u][i] = rb[u][i] = Ch::zero();
                if (pl.live[i] && h + u < h1) {
                    ra[u][i] = *reinterpret_cast<const Raw *>(x + (h + u) * sd.x.h + pl.a[i]);
                    rb[u][i] = *reinterpret_cast<const Raw *>(x + (h + u) * sd.x.h + pl.b[i]);
                }
            }
    };
    load(h0);   // on their way while the sines are computed
    float wa[CP][VEC], wb[CP][VEC];
#pragma unroll
    for (int i = 0; i < CP; ++i)
#pragma unroll
        for (int t = 0; t < VEC; ++t) {
            wa[i][t] = sd.weight ? sd.weight[pl.a[i] + t] : 1.f;
            wb[i][t] = sd.weight ? sd.weight[pl.b[i] + t] : 1.f;
        }
    pl.at(p.positions ? p.positions[b * p.pos_batch + n] : n);

#pragma unroll 1
    for (int h = h0; h < h1; h += U) {
        if (h > h0) load(h);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float xa[CP][VEC], xb[CP][VEC], ss = 0.f;
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                Ch::get(ra[u][i], xa[i]);
                Ch::get(rb[u][i], xb[i]);
#pragma unroll
                for (int t = 0; t < VEC; ++t) ss = fmaf(xa[i][t], xa[i][t], fmaf(xb[i][t], xb[i][t], ss));
            }
            float s = 1.f;
            if (p.c > 0.f) {
                ss = group_sum<LPR>(ss);
                float eps = p.eps;
                if (__any_sync(0xffffffffu, !(ss <= kRotBig))) {   // squares that pass float32's range
                    const float down = ss <= kRotBig ? 1.f : kRotDown;
                    ss = 0.f;
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int t = 0; t < VEC; ++t) {
                            xa[i][t] *= down;
                            xb[i][t] *= down;
                            ss = fmaf(xa[i][t], xa[i][t], fmaf(xb[i][t], xb[i][t], ss));
                        }
                    ss = group_sum<LPR>(ss);
                    eps *= down * down;
                }
                s = rsqrtf(fmaf(p.c, ss, eps));
            }
#pragma unroll
            for (int i = 0; i < CP; ++i) {
#pragma unroll
                for (int t = 0; t < VEC; ++t) {
                    xa[i][t] *= s * wa[i][t];
                    xb[i][t] *= s * wb[i][t];
                }
                pl.rotate(i, xa[i], xb[i], 1.f);
                if (live && pl.live[i] && h + u < h1) {
                    *reinterpret_cast<Raw *>(y + (h + u) * sd.y.h + pl.a[i]) = Ch::put(xa[i]);
                    *reinterpret_cast<Raw *>(y + (h + u) * sd.y.h + pl.b[i]) = Ch::put(xb[i]);
                }
            }
        }
    }
}

struct Forward {
    template <typename T, int VEC, int CLS, bool ADJ> static cudaError_t run(const NormRotateArgs &a) {
        using L = RotLanes<VEC, CLS>;
        constexpr int per = kRotThreads / L::LPR;
        RotParams p = rot_params(a);
        rot_ranges(p, (long long)rot_sms() * 2048 / L::LPR);
        const dim3 grid((unsigned)((p.tokens + per - 1) / per), p.side[0].parts + p.side[1].parts);
        norm_rotate_kernel<T, VEC, L::LPR, L::CP, ADJ><<<grid, kRotThreads, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
};

}  // namespace

cudaError_t launch_norm_rotate(const NormRotateArgs &a) { return rot_launch<Forward>(a); }

}  // namespace la
