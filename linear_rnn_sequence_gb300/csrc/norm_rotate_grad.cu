// norm_rotate_grad.cu -- gradients of the norm and rotation of queries and keys (norm_rotate.cuh).
//
//   u = the output's gradient turned back,  g = u * weight,
//   grad_x = s (g - c xh sum(g xh)),   grad_weight = sum over rows of u xh
//
// The norm's scale is computed again from x, which has to be read anyway: sum(x^2) and sum(g x) are
// joined over the lanes together.  Bound by HBM: two reads and one write a value.  A CTA goes through many
// tokens with the sums of its weights' gradients in registers (each token's heads are summed first, which
// keeps the long sums short), writes them once, and a second kernel adds the CTAs' rows in their order.  The next
// rows, the next token's among them, are on their way while these are worked on.  B8 N8192, 16 + 16 heads of 128, bf16: 293 us,
// 5.5 TB/s of the 6.7 that a copy reaches (one head in flight 376 us, four 402; three CTAs an SM, whose registers spill, 557);
// fp32 491 us, the copy's rate, although its kernels spill about 100 bytes a thread.
#include "norm_rotate.cuh"

namespace la {
namespace {

constexpr int kRotThreads = 256;

template <typename T, int VEC, int LPR, int CP, bool ADJ>
__global__ void __launch_bounds__(kRotThreads, 2) norm_rotate_grad_kernel(const RotParams p) {
    using Ch = Chunk<T, VEC>;
    using Raw = typename Ch::Raw;
    constexpr int U = CP * VEC <= 4 ? 2 : 1, PER = kRotThreads / LPR;   // heads in flight, tokens of a CTA at a time
    __shared__ float cols[PER * 2 * LPR * CP * VEC];
    const int gl = threadIdx.x % LPR, grp = threadIdx.x / LPR, part = blockIdx.y;
    const bool second = part >= p.side[0].parts;
    const RotSide sd = second ? p.side[1] : p.side[0];
    const int h0 = (second ? part - p.side[0].parts : part) * p.span, h1 = min(sd.heads, h0 + p.span);

    Place<VEC, CP, ADJ> pl;
    pl.template init<LPR>(p, gl);
    float wa[CP][VEC], wb[CP][VEC], da[CP][VEC], db[CP][VEC];
#pragma unroll
    for (int i = 0; i < CP; ++i)
#pragma unroll
        for (int t = 0; t < VEC; ++t) {
            wa[i][t] = sd.weight ? sd.weight[pl.a[i] + t] : 1.f;
            wb[i][t] = sd.weight ? sd.weight[pl.b[i] + t] : 1.f;
            da[i][t] = db[i][t] = 0.f;
        }

    struct At {   // a token's rows
        const T *x, *g;
        T *y;
        long long pos;
    };
    auto token = [&](long long t0) {
        const long long tok = t0 + grp < p.tokens ? t0 + grp : p.tokens - 1, b = tok / p.N;
        const int n = (int)(tok - b * p.N);
        return At{static_cast<const T *>(sd.x.p) + b * sd.x.b + n * sd.x.t, static_cast<const T *>(sd.g.p) + b * sd.g.b + n * sd.g.t,
                  static_cast<T *>(sd.y.p) + b * sd.y.b + n * sd.y.t, p.positions ? p.positions[b * p.pos_batch + n] : n};
    };
    Raw rx[U][2 * CP], rg[U][2 * CP];
    auto load = [&](const At &k, int h) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                rx[u][2 * i] = rx[u][2 * i + 1] = rg[u][2 * i] = rg[u][2 * i + 1] = Ch::zero();
                if (pl.live[i] && h + u < h1) {
                    rx[u][2 * i] = *reinterpret_cast<const Raw *>(k.x + (h + u) * sd.x.h + pl.a[i]);
                    rx[u][2 * i + 1] = *reinterpret_cast<const Raw *>(k.x + (h + u) * sd.x.h + pl.b[i]);
                    rg[u][2 * i] = *reinterpret_cast<const Raw *>(k.g + (h + u) * sd.g.h + pl.a[i]);
                    rg[u][2 * i + 1] = *reinterpret_cast<const Raw *>(k.g + (h + u) * sd.g.h + pl.b[i]);
                }
            }
    };
    const long long step = (long long)p.blocks * PER;
    long long t0 = (long long)blockIdx.x * PER;   // below the number of tokens: no more CTAs than that
    At here = token(t0);
    load(here, h0);
#pragma unroll 1
    while (true) {
        const bool live = t0 + grp < p.tokens, more = t0 + step < p.tokens;
        const At next = more ? token(t0 + step) : here;
        pl.at(p, here.pos);
        float ta[CP][VEC], tb[CP][VEC];   // this token's
#pragma unroll
        for (int i = 0; i < CP; ++i)
#pragma unroll
            for (int t = 0; t < VEC; ++t) ta[i][t] = tb[i][t] = 0.f;
#pragma unroll 1
        for (int h = h0; h < h1; h += U) {
            float xa[U][CP][VEC], xb[U][CP][VEC], ga[U][CP][VEC], gb[U][CP][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < CP; ++i) {
                    Ch::get(rx[u][2 * i], xa[u][i]);
                    Ch::get(rx[u][2 * i + 1], xb[u][i]);
                    Ch::get(rg[u][2 * i], ga[u][i]);
                    Ch::get(rg[u][2 * i + 1], gb[u][i]);
                }
            if (h + U < h1) load(here, h + U);   // the next ones, while these are worked on
            else if (more) load(next, h0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < CP; ++i) pl.rotate(i, ga[u][i], gb[u][i], -1.f);
                float ss, gx;
                auto sums = [&] {
                    ss = gx = 0.f;
#pragma unroll
                    for (int i = 0; i < CP; ++i)
#pragma unroll
                        for (int t = 0; t < VEC; ++t) {
                            ss = fmaf(xa[u][i][t], xa[u][i][t], fmaf(xb[u][i][t], xb[u][i][t], ss));
                            gx = fmaf(ga[u][i][t] * wa[i][t], xa[u][i][t], fmaf(gb[u][i][t] * wb[i][t], xb[u][i][t], gx));
                        }
                    ss = group_sum<LPR>(ss);
                    gx = group_sum<LPR>(gx);
                };
                float s = 1.f, along = 0.f, by = 1.f;
                if (p.c > 0.f) {
                    sums();
                    if (__any_sync(0xffffffffu, !sum_holds(ss, p.least))) {   // squares that pass float32's range
                        by = rescale(ss, p.least);
#pragma unroll
                        for (int i = 0; i < CP; ++i)
#pragma unroll
                            for (int t = 0; t < VEC; ++t) {
                                xa[u][i][t] *= by;
                                xb[u][i][t] *= by;
                            }
                        sums();
                    }
                    s = rsqrtf(fmaf(p.c, ss, p.eps * by * by));
                    along = p.c * s * s * gx;
                }
                const bool keep = live && h + u < h1;
                const float so = s * by;
#pragma unroll
                for (int i = 0; i < CP; ++i) {
#pragma unroll
                    for (int t = 0; t < VEC; ++t) {
                        if (keep) {
                            ta[i][t] = fmaf(ga[u][i][t], xa[u][i][t] * s, ta[i][t]);
                            tb[i][t] = fmaf(gb[u][i][t], xb[u][i][t] * s, tb[i][t]);
                        }
                        const float fa = ga[u][i][t] * wa[i][t], fb = gb[u][i][t] * wb[i][t];   // without a norm x has no say
                        xa[u][i][t] = p.c > 0.f ? so * fmaf(-along, xa[u][i][t], fa) : fa;
                        xb[u][i][t] = p.c > 0.f ? so * fmaf(-along, xb[u][i][t], fb) : fb;
                    }
                    if (keep && pl.live[i]) {
                        *reinterpret_cast<Raw *>(here.y + (h + u) * sd.y.h + pl.a[i]) = Ch::put(xa[u][i]);
                        *reinterpret_cast<Raw *>(here.y + (h + u) * sd.y.h + pl.b[i]) = Ch::put(xb[u][i]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < CP; ++i)
#pragma unroll
            for (int t = 0; t < VEC; ++t) {
                da[i][t] += ta[i][t];
                db[i][t] += tb[i][t];
            }
        if (!more) break;
        t0 += step;
        here = next;
    }
    if (!p.partials) return;
#pragma unroll
    for (int i = 0; i < CP; ++i)
#pragma unroll
        for (int t = 0; t < VEC; ++t)
            if (pl.live[i]) {
                cols[grp * p.d + pl.a[i] + t] = da[i][t];
                cols[grp * p.d + pl.b[i] + t] = db[i][t];
            }
    __syncthreads();
    float *out = p.partials + ((size_t)part * p.blocks + blockIdx.x) * p.d;
    for (int c = threadIdx.x; c < p.d; c += kRotThreads) {
        float x = 0.f;
        for (int i = 0; i < PER; ++i) x += cols[i * p.d + c];
        out[c] = x;
    }
}

// Sums over the CTAs' rows, q's (parts0 * blocks of them) before k's: 32 columns x 16 slices of the rows.
__global__ void __launch_bounds__(512)
norm_rotate_columns_kernel(const float *__restrict__ part, int rows_q, int rows_k, int d, float *dwq, float *dwk) {
    __shared__ float s[16][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), sl = threadIdx.x >> 5;
    float *out = blockIdx.y ? dwk : dwq;
    if (!out) return;
    const float *src = part + (blockIdx.y ? (size_t)rows_q * d : 0);
    const int n = blockIdx.y ? rows_k : rows_q;
    float x = 0.f;
    if (c < d)
#pragma unroll 4
        for (int i = sl; i < n; i += 16) x += src[(size_t)i * d + c];
    s[sl][threadIdx.x & 31] = x;
    __syncthreads();
    if (sl == 0 && c < d) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x];
        out[c] = t;
    }
}

// CTAs: two an SM, no more than there are tokens for.
template <int VEC, int CLS> RotParams planned(const NormRotateArgs &a) {
    constexpr int per = kRotThreads / RotLanes<VEC, CLS>::LPR;
    RotParams p = rot_params(a);
    const long long ctas = 2LL * rot_sms();
    rot_ranges(p, ctas * per);
    const long long need = (p.tokens + per - 1) / per, most = ctas / (p.side[0].parts + p.side[1].parts);
    p.blocks = (int)(need < most ? need : most > 1 ? most : 1);
    return p;
}

struct Grad {
    template <typename T, int VEC, int CLS, bool ADJ> static cudaError_t run(const NormRotateArgs &a) {
        using L = RotLanes<VEC, CLS>;
        const RotParams p = planned<VEC, CLS>(a);
        const dim3 grid(p.blocks, p.side[0].parts + p.side[1].parts);
        norm_rotate_grad_kernel<T, VEC, L::LPR, L::CP, ADJ><<<grid, kRotThreads, 0, a.stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || !p.partials) return e;
        norm_rotate_columns_kernel<<<dim3((p.d + 31) / 32, 2), 512, 0, a.stream>>>(
            p.partials, p.side[0].parts * p.blocks, p.side[1].parts * p.blocks, p.d, a.dwq, a.dwk);
        return cudaGetLastError();
    }
};

}  // namespace

// Any VEC's CTAs: at most 2 an SM, or one for each range of heads.
size_t norm_rotate_partials(const NormRotateArgs &a) {
    const size_t ctas = 2 * (size_t)rot_sms(), ranges = (size_t)a.Hq + a.Hk;
    return (ctas > ranges ? ctas : ranges) * a.d;
}

cudaError_t launch_norm_rotate_grad(const NormRotateArgs &a) { return rot_launch<Grad>(a); }

}  // namespace la
