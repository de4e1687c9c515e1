// norm_rotate.cu -- queries and keys normed by head, weighted and rotated by position, in one pass
// (norm_rotate.cuh says how a row lies in the lanes).
//
// Bound by HBM: each value is read once and written once, and stays in registers between; the next heads are on
// their way while these are worked on.  B8 N8192, 16 + 16 heads of 128, bf16: 180 to 184 us, 5.9 TB/s of the 6.7 that a copy reaches
// (CTAs of 256 threads 3% slower; one head in flight rather than two 11%, four 14%); fp32 318 us, the copy's rate.
#include "norm_rotate.cuh"

namespace la {
namespace {

constexpr int kRotThreads = 128;
constexpr int kRotInFlight = 8;   // pairs of values of a lane, on their way and again worked on

template <typename T, int VEC, int LPR, int CP, bool ADJ>
__global__ void __launch_bounds__(kRotThreads) norm_rotate_kernel(const RotParams p) {
    using Ch = Chunk<T, VEC>;
    using Raw = typename Ch::Raw;
    constexpr int U = kRotInFlight / (CP * VEC) > 0 ? kRotInFlight / (CP * VEC) : 1;   // heads in flight
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
    pl.at(p, p.positions ? p.positions[b * p.pos_batch + n] : n);

#pragma unroll 1
    for (int h = h0; h < h1; h += U) {
        float xa[U][CP][VEC], xb[U][CP][VEC], ss[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ss[u] = 0.f;
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                Ch::get(ra[u][i], xa[u][i]);
                Ch::get(rb[u][i], xb[u][i]);
            }
        }
        if (h + U < h1) load(h + U);   // the next ones, while these are worked on
        float eps[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < CP; ++i)
#pragma unroll
                for (int t = 0; t < VEC; ++t) ss[u] = fmaf(xa[u][i][t], xa[u][i][t], fmaf(xb[u][i][t], xb[u][i][t], ss[u]));
            eps[u] = p.eps;
        }
        if (p.c > 0.f) {
            bool again = false;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                ss[u] = group_sum<LPR>(ss[u]);
                again |= !sum_holds(ss[u], p.least);
            }
            if (__any_sync(0xffffffffu, again)) {   // squares that pass float32's range
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float by = rescale(ss[u], p.least);
                    ss[u] = 0.f;
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int t = 0; t < VEC; ++t) {
                            xa[u][i][t] *= by;
                            xb[u][i][t] *= by;
                            ss[u] = fmaf(xa[u][i][t], xa[u][i][t], fmaf(xb[u][i][t], xb[u][i][t], ss[u]));
                        }
                    ss[u] = group_sum<LPR>(ss[u]);
                    eps[u] = eps[u] * by * by;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float s = p.c > 0.f ? rsqrtf(fmaf(p.c, ss[u], eps[u])) : 1.f;
#pragma unroll
            for (int i = 0; i < CP; ++i) {
#pragma unroll
                for (int t = 0; t < VEC; ++t) {
                    xa[u][i][t] *= s * wa[i][t];
                    xb[u][i][t] *= s * wb[i][t];
                }
                pl.rotate(i, xa[u][i], xb[u][i], 1.f);
                if (live && pl.live[i] && h + u < h1) {
                    *reinterpret_cast<Raw *>(y + (h + u) * sd.y.h + pl.a[i]) = Ch::put(xa[u][i]);
                    *reinterpret_cast<Raw *>(y + (h + u) * sd.y.h + pl.b[i]) = Ch::put(xb[u][i]);
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
