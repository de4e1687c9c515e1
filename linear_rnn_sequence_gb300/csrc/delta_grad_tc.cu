// delta_grad_tc.cu -- delta_grad.cu's products on the tensor cores (bf16 inputs,
// d and dv in {64, 128}): an item is a block of 64 tokens and a key head, whose
// value heads (units) are summed in registers.
//
// The gradients of q and k are accumulated transposed, a TMEM lane for each of
// the d features (S, G the state before the block and its gradient after it):
//     dq^T = c . (S dy^T) + K^T P^T,
//     dk^T = w . (G e^T) - b c . (S du^T) + Q^T P + K^T F,
//     P_ij = D_ij b_j (dy_i . e_j)  (j <= i),   w_j = D_Cj b_j,
//     F_ij = F_ji = -b_i D_ij b_j (du_i . e_j)  (j < i),
// the scores dy_i . e_j and du_i . e_j as one product of the stacked rows
// [dy; du].  dq and its scores are computed to float32 (three pieces of each
// float32 operand, see delta_tc.cu), and so is G e^T: the gates' gradient is a difference of
// q . dq and v . dv, and <G, S'>.  What only dk depends on, which is rounded to bf16, takes
// two pieces: du and F rounded to nearest (at most 2^-17 is left), S and P^T the top two of their
// three (less than 2^-15, always of their sign); du's middle by e's middle and low pieces are dropped (2^-15).
//
// <G, S'> of the gates' gradient, S' the state behind the block, takes no other
// read: S' = c_C S + K^T W, so it is c_C <G, S> + sum_j w_j (G e)_j . k_j.
//
// S, G, e and du are read once, 192 KB a block at d = dv = 128 beside the 112 KB
// of inputs and outputs: 0.75 ms of HBM for B8 H16 N8192, where the kernel takes
// 1.2 ms (22,000 cycles a unit and SM).  Persistent CTAs, one an SM: 16 warps turn float32
// values into operands and accumulators into gradients, warp 0 also issues the
// MMAs.  Every operand is copied to shared memory while the unit before, or the
// MMAs, still run: S and then G as swizzled slabs, whose rows a lane reads without
// bank conflicts, in the place that P and F take later; e and du where their
// pieces go.  (Through registers, with S' read too, a unit took 27,500 cycles,
// 14,000 of them in loads that nothing else covered.)  What is left alternates
// between the MMAs (5,900 cycles at the pipe's rate) and the conversions, TMEM and shared
// memory having no room for a second unit; a warp of its own to issue MMAs would leave
// 96 registers a thread, and spills.
#include "delta_tc.cuh"

namespace la {
namespace {

constexpr int kGThr = 512, kBarG = 1;
// TMEM columns: pieces of S (3 DV/2); the scores' two accumulators, then two pieces of G (2 DV/2);
// S dy^T; the third piece of G; S du^T.  K^T P^T, Q^T P + K^T F and G e^T take the place of S.
constexpr uint32_t gS = 0, gPF = 192, gG = 192, gQ = 320, gGl = 384, gSu = 448, gQ2 = 0, gK2 = 64, gGe = 128;

struct GradTc {
    const float *beta, *lg, *S_ck, *G_ck, *e, *du;
    const __nv_bfloat16 *v;
    __nv_bfloat16 *dv;
    float *dbeta, *dlg;
    int H, Hk, N, layout, nblk, items;
    unsigned int *err, *err_where;
    unsigned long long limit_ns;
};
struct GradUnit {   // what a unit leaves for the sums over its tokens
    Gates gates;
    float db[kDC], vdv[kDC], qdq[4][kDC], gs[kGThr / 32];
};
struct GradSmall {
    GradUnit unit[2];
    uint64_t kq_full, y_full, sg_full, eu_full, pf_done, s_done, all_done, drained;
    uint32_t tmem_base;
    int loads[4];   // issued to the first four
    volatile int abort_flag;
};
template <int D, int DV> struct GradLay {
    static constexpr int kT = (D / 64) * 8192;            // K or Q, slabs of 64 features
    static constexpr int kX = (DV / 64) * 16384;          // per 64 columns: 64 rows, 64 rows
    static constexpr int kE = (DV / 64) * 8192;
    static constexpr int kSG = D * DV * 4;                // S or G; P, P^T and F take its place
    static constexpr bool kOwnQ = D + DV < 256;           // dq's tile has a place of its own, or du's
    static constexpr int oKQ = 0, oX1 = 2 * kT, oX2 = oX1 + kX, oEm = oX2 + kX, oEl = oEm + kE,
                         oSG = oEl + kE, oPT = oSG + 3 * 8192, oF = oPT + 2 * 8192,
                         oDK = oSG + (kSG > 7 * 8192 ? kSG : 7 * 8192), oDQ = kOwnQ ? oDK + kT : oX1 + 8192,
                         kDQ = kOwnQ ? 8192 : 16384, oSmall = oDK + (kOwnQ ? 2 : 1) * kT;
    static constexpr int total = oSmall + (int)sizeof(GradSmall);
    static constexpr int request = total + 1024;
};

// 16 columns of a thread's row as three pieces into TMEM: `stride` columns apart, and at `low`.
__device__ __forceinline__ void put_pieces(uint32_t at, uint32_t stride, uint32_t low, const float (&x)[16]) {
    uint32_t hi[8], mi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split3(x[2 * j], x[2 * j + 1], hi[j], mi[j], lo[j]);
    tmem_st8(at, hi);
    tmem_st8(at + stride, mi);
    tmem_st8(low, lo);
}

// Sum of x[t] over the warp's 32 lanes for t = 0 .. 15; lanes 0 .. 15 get that of t = lane.
__device__ __forceinline__ float reduce16(float (&x)[16], int lane) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {   // halves of the values move to the lane that keeps them
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? x[i + o] : x[i], give = up ? x[i] : x[i + o];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

// ONE: a single value head to a key head, whose gradients then need no sums.
template <int D, int DV, bool ONE>
__global__ void __launch_bounds__(kGThr, 1)
delta_grad_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap dqmap,
                     const __grid_constant__ CUtensorMap dkmap, const __grid_constant__ CUtensorMap smap,
                     const __grid_constant__ CUtensorMap gmap, const GradTc p) {
    using Lay = GradLay<D, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    GradSmall &S = *reinterpret_cast<GradSmall *>(sm + Lay::oSmall);
    uint8_t *sKQ = sm + Lay::oKQ, *sX1 = sm + Lay::oX1, *sX2 = sm + Lay::oX2, *sEm = sm + Lay::oEm,
            *sEl = sm + Lay::oEl, *sSG = sm + Lay::oSG, *sP = sSG, *sPT = sm + Lay::oPT, *sF = sm + Lay::oF,
            *sDK = sm + Lay::oDK, *sDQ = sm + Lay::oDQ;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int nblk = p.nblk, group = ONE ? 1 : p.H / p.Hk;
    const Guard g{&S.abort_flag, p.err, p.err_where, p.limit_ns};

    if (tid == 0) {
        S.abort_flag = 0;
        mbar_init(&S.kq_full, 1);
        mbar_init(&S.y_full, 1);
        mbar_init(&S.sg_full, 1);
        mbar_init(&S.eu_full, 1);
        mbar_init(&S.drained, 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) S.loads[i] = 0;
        mbar_init(&S.pf_done, 1);
        mbar_init(&S.s_done, 1);
        mbar_init(&S.all_done, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&S.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, S.tmem_base, 0);

    constexpr uint32_t i64 = idesc_bf16(128, kDC, 0, 0), iT = idesc_bf16(128, kDC, 1, 0);
    auto load_kq = [&](int it) {
        const int t0 = it % nblk * kDC, b = it / nblk / p.Hk, hk = it / nblk % p.Hk;
        mbar_arrive_expect_tx(&S.kq_full, 2 * kDC * D * 2);
        ++S.loads[0];
#pragma unroll
        for (int f = 0; f < D / 64; ++f) {
            tma_load_4d(sKQ + f * 8192, &kmap, &S.kq_full, f * 64, t0, hk, b);
            tma_load_4d(sKQ + Lay::kT + f * 8192, &qmap, &S.kq_full, f * 64, t0, hk, b);
        }
    };
    auto load_y = [&](int it, int gi) {
        const int t0 = it % nblk * kDC, b = it / nblk / p.Hk, h = it / nblk % p.Hk * group + gi;
        mbar_arrive_expect_tx(&S.y_full, kDC * DV * 2);
        ++S.loads[1];
#pragma unroll
        for (int f = 0; f < DV / 64; ++f) tma_load_4d(sX1 + f * 16384, &ymap, &S.y_full, f * 64, t0, h, b);
    };
    // index of value head gi of item it's key head
    auto head_of = [&](int it, int gi) { return (size_t)(it / nblk / p.Hk) * p.H + it / nblk % p.Hk * group + gi; };
    // S before a unit's block, or G after it: slabs of 32 columns
    auto load_sg = [&](bool G, int it, int gi) {
        const int at = (int)(head_of(it, gi) * (nblk + !G)) + it % nblk;
        mbar_arrive_expect_tx(&S.sg_full, Lay::kSG);
        ++S.loads[2];
#pragma unroll
        for (int f = 0; f < DV / 32; ++f)
            tma_load_3d(sSG + f * D * 128, G ? &gmap : &smap, &S.sg_full, f * 32, 0, at);
    };
    // e and du of a unit, float32, where their pieces go
    auto load_eu = [&](int it, int gi) {
        const int t0 = it % nblk * kDC;
        const size_t o = (head_of(it, gi) * p.N + t0) * DV;
        const uint32_t bytes = min(kDC, p.N - t0) * DV * 4;
        mbar_arrive_expect_tx(&S.eu_full, 2 * bytes);
        ++S.loads[3];
        bulk_load(sEm, p.e + o, bytes, &S.eu_full);
        bulk_load(sX2, p.du + o, bytes, &S.eu_full);
    };
    // scores, and what S gives
    auto issue_first = [&]() {
        tc_fence_after();
        const uint64_t x1 = desc_k(smem_u32(sX1)), x2 = desc_k(smem_u32(sX2));
        // [dy; du_h] (e_l, e_m, e_h), small ones first, and du_m e_h (the upper rows unused)
        uint32_t leader = elect_leader();
#pragma unroll 1
        for (int o = 0; o < 4; ++o) {
            const bool eh = o >= 2;
            const uint64_t a = o == 3 ? x2 : x1, bd = eh ? x2 : desc_k(smem_u32(o ? sEm : sEl));
            const uint32_t d = tb + gPF + (o == 3 ? 64 : 0), slab = eh ? 16384 / 16 : 8192 / 16;
#pragma unroll
            for (int ks = 0; ks < DV / 16; ++ks)
                mma_ss_if(leader, d, a + (ks >> 2) * 1024 + (ks & 3) * 2, bd + (ks >> 2) * slab + (ks & 3) * 2,
                          i64, (o != 0 && o != 3) || ks > 0);
        }
        mma_commit_if(leader, &S.pf_done);
        // S dy^T from three pieces, S du^T from (m, m) (m, h) (h, m) (h, h)
        leader = elect_leader();
#pragma unroll 1
        for (int pc = 2; pc >= 0; --pc)
            mma_rows<DV / 16, 16384>(leader, tb + gQ, tb + gS + pc * (DV / 2), smem_u32(sX1), i64, pc < 2);
        leader = elect_leader();
#pragma unroll 1
        for (int o = 0; o < 4; ++o)
            mma_rows<DV / 16, 16384>(leader, tb + gSu, tb + gS + (o < 2) * (DV / 2),
                                     smem_u32(o & 1 ? sX1 : sX2) + 8192, i64, o > 0);
        mma_commit_if(leader, &S.s_done);
    };
    // what G gives, where the lowest pieces of S were
    auto issue_g = [&]() {
        const uint32_t leader = elect_leader();
        tc_fence_after();
#pragma unroll 1
        for (int o = 0; o < 6; ++o) {   // pieces (G, e): (l, h) (h, l) (m, m) (m, h) (h, m) (h, h)
            const uint32_t a = tb + (o == 0 ? gGl : gG + (o == 2 || o == 3 ? DV / 2 : 0));
            if (o == 0 || o == 3 || o == 5)
                mma_rows<DV / 16, 16384>(leader, tb + gGe, a, smem_u32(sX2), i64, o > 0);
            else
                mma_rows<DV / 16, 8192>(leader, tb + gGe, a, smem_u32(o == 1 ? sEl : sEm), i64, true);
        }
    };
    // K^T P^T, Q^T P + K^T F in S's place
    auto issue_second = [&]() {
        tc_fence_after();
        // features 64 .. 127 repeat the others where there are none
        const uint32_t sk = smem_u32(sKQ);
        const uint64_t kd = smem_desc(sk, D > 64 ? 8192 : 0, 1024, kSwizzle128B);
        const uint64_t qd = smem_desc(sk + Lay::kT, D > 64 ? 8192 : 0, 1024, kSwizzle128B);
        const uint64_t pd = desc_k(smem_u32(sP)), ptd = desc_k(smem_u32(sPT)), fd = desc_k(smem_u32(sF));
        uint32_t leader = elect_leader();
#pragma unroll 1
        for (int pc = 2; pc >= 0; --pc)
#pragma unroll
            for (int ks = 0; ks < kDC / 16; ++ks)
                mma_ss_if(leader, tb + gQ2, kd + ks * 128, pd + pc * 512 + ks * 2, iT, pc < 2 || ks > 0);
        leader = elect_leader();
#pragma unroll 1
        for (int o = 0; o < 4; ++o) {   // (Q, P_m) (K, F_m) (Q, P_h) (K, F_h)
            const uint64_t a = o & 1 ? kd : qd, bd = (o & 1 ? fd : ptd) + (o < 2 ? 512 : 0);
#pragma unroll
            for (int ks = 0; ks < kDC / 16; ++ks)
                mma_ss_if(leader, tb + gK2, a + ks * 128, bd + ks * 2, iT, o > 0 || ks > 0);
        }
        mma_commit_if(leader, &S.all_done);
    };

    if (warp == 0 && elect_leader()) {
        load_kq(blockIdx.x);
        load_y(blockIdx.x, 0);
        load_sg(false, blockIdx.x, 0);
        load_eu(blockIdx.x, 0);
    }
    __syncwarp();
    {
        const int wq = warp & 3, row = wq * 32 + lane, cg = warp >> 2;   // TMEM lane; quarter of the columns
        const uint32_t lb = (uint32_t)(wq * 32) << 16;
        constexpr int SC = DV / 4;   // state columns of a thread
        const bool live = row < D;   // warp-uniform: lanes with a feature
        const size_t st = (size_t)D * DV;
        constexpr int kCopier = kGThr / 2;   // the thread of most copies
        // A thread's columns of its row of S or G: chunks of 16 bytes at c ^ (row & 7) of their slab, so
        // that eight lanes' reads spread over all banks.
        auto row16 = [&](int i, float (&x)[16]) {   // columns cg SC + i ..
            const int c = cg * SC + i;
            const uint8_t *at = sSG + (c >> 5) * D * 128 + row * 128;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4 *>(x + 4 * j) =
                    *reinterpret_cast<const float4 *>(at + ((((c & 31) >> 2) + j) ^ (row & 7)) * 16);
        };
        auto any_failed = [](bool f) { return __any_sync(0xffffffffu, group_any<kBarG, kGThr>(f)) != 0; };
        // the sums over a unit's tokens, once every warp has left its epilogue
        auto finish = [&](int it, int gi, const GradUnit &U) {
            const int b = it / nblk / p.Hk, h = it / nblk % p.Hk * group + gi, t0 = it % nblk * kDC;
            const int n_in = min(kDC, p.N - t0);
            const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
            if (tid < n_in) p.dbeta[rs.at(t0 + tid)] = U.db[tid];
            if (warp == 15 && p.lg) {   // running sums from the block's end, two tokens a lane
                F2 x2[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = 2 * lane + i;
                    float q = U.qdq[0][t] + U.qdq[1][t];
                    if (D > 64) q += U.qdq[2][t] + U.qdq[3][t];
                    const float d = q - U.vdv[t], z = d - q;
                    x2[i] = {d, (q - (d - z)) - (U.vdv[t] + z)};
                }
                const float e = warp_sum(lane < kGThr / 32 ? U.gs[lane] : 0.f);
                x2[0] = f2sum2(x2[0], x2[1]);
                F2 s = x2[0];
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const F2 y = {__shfl_down_sync(0xffffffffu, s.h, o), __shfl_down_sync(0xffffffffu, s.l, o)};
                    if (lane + o < 32) s = f2sum2(s, y);
                }
                F2 after = {__shfl_down_sync(0xffffffffu, s.h, 1), __shfl_down_sync(0xffffffffu, s.l, 1)};
                if (lane == 31) after = {0.f, 0.f};
                const F2 tail = {e, 0.f}, first = f2sum2(tail, s), second = f2sum2(tail, f2sum2(after, x2[1]));
                if (2 * lane < n_in) p.dlg[rs.at(t0 + 2 * lane)] = first.h + first.l;
                if (2 * lane + 1 < n_in) p.dlg[rs.at(t0 + 2 * lane + 1)] = second.h + second.l;
            }
        };

        float dq[16], dk[16];   // feature `row`, tokens 16 cg ..: sums over the value heads
        bool failed = false;
        int u = 0, k = 0, last_it = 0, last_gi = 0;
        for (int it = blockIdx.x; it < p.items && !failed; it += gridDim.x, ++k) {
            const int blk = it % nblk, b = it / nblk / p.Hk, hk = it / nblk % p.Hk;
            const int t0 = blk * kDC, n_in = min(kDC, p.N - t0);
#pragma unroll
            for (int i = 0; i < 16; ++i) dq[i] = dk[i] = 0.f;
            for (int gi = 0; gi < group; ++gi, ++u) {
                const int h = hk * group + gi;
                const size_t bh = head_of(it, gi);
                const TokenRows rv = token_rows(p.layout, b, h, p.H, p.N, DV),
                                rs = token_rows(p.layout, b, h, p.H, p.N, 1);
                GradUnit &U = S.unit[u & 1];
                // ---- e and du as pieces, tokens x dv; dv = b du and the tokens' sums
                constexpr int NT = DV / 64;
                float e[NT][8], du[NT][8], bt[NT];
                uint4 vw[NT];
                bool ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.eu_full, u & 1, g, 9));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int e0 = i * kGThr + tid, t = e0 / (DV / 8), c = e0 % (DV / 8) * 8;
                    bt[i] = 0.f;
                    vw[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (t < n_in) {
                        bt[i] = p.beta[rs.at(t0 + t)];
                        vw[i] = __ldg(reinterpret_cast<const uint4 *>(p.v + rv.at(t0 + t) + c));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[i][j] = du[i][j] = 0.f;
                    if (t < n_in) {
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            *reinterpret_cast<float4 *>(&e[i][j]) =
                                *reinterpret_cast<const float4 *>(sEm + (t * DV + c + j) * 4);
                            *reinterpret_cast<float4 *>(&du[i][j]) =
                                *reinterpret_cast<const float4 *>(sX2 + (t * DV + c + j) * 4);
                        }
                    }
                }
                // every value is in registers, an item's dq and dk have been stored, and the unit
                // before is done: its accumulators lie where S goes, its sums are complete
                if (tid == kCopier) bulk_wait_read<0>();
                if ((failed = any_failed(!ok))) break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int e0 = i * kGThr + tid, t = e0 / (DV / 8), c = e0 % (DV / 8) * 8;
                    const uint32_t v2[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
                    float db = 0.f, vd = 0.f, g2[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        g2[j] = bt[i] * du[i][j];
                        db = fmaf(du[i][j], e[i][j], db);
                        vd = fmaf(j & 1 ? bf16_hi_f(v2[j >> 1]) : bf16_lo_f(v2[j >> 1]), g2[j], vd);
                    }
                    if (t < n_in)
                        *reinterpret_cast<uint4 *>(p.dv + rv.at(t0 + t) + c) =
                            make_uint4(pack_bf16x2(g2[0], g2[1]), pack_bf16x2(g2[2], g2[3]),
                                       pack_bf16x2(g2[4], g2[5]), pack_bf16x2(g2[6], g2[7]));
#pragma unroll
                    for (int o = DV / 16; o > 0; o >>= 1) {
                        db += __shfl_xor_sync(0xffffffffu, db, o);
                        vd += __shfl_xor_sync(0xffffffffu, vd, o);
                    }
                    if (c == 0) { U.db[t] = db; U.vdv[t] = vd; }
                    uint32_t hi[4], mi[4], lo[4];
                    const uint32_t o16 = (c >> 6) * 16384 + sw128_off(t, c & 63),
                                   o8 = (c >> 6) * 8192 + sw128_off(t, c & 63);
#pragma unroll
                    for (int j = 0; j < 4; ++j) split3(e[i][2 * j], e[i][2 * j + 1], hi[j], mi[j], lo[j]);
                    *reinterpret_cast<uint4 *>(sX2 + o16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(sEm + o8) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                    *reinterpret_cast<uint4 *>(sEl + o8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) split2(du[i][2 * j], du[i][2 * j + 1], hi[j], mi[j]);
                    *reinterpret_cast<uint4 *>(sX1 + 8192 + o16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(sX2 + 8192 + o16) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                }
                fence_proxy_async();
                float x[SC];   // of S
                ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.sg_full, 0, g, 3));
                if (ok && live) {
#pragma unroll
                    for (int i = 0; i < SC; i += 16) {
                        float (&y)[16] = *reinterpret_cast<float (*)[16]>(x + i);
                        row16(i, y);
                        const uint32_t col = tb + lb + gS + (cg * SC + i) / 2;
                        put_pieces(col, DV / 2, col + DV, y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < SC; ++i) x[i] = 0.f;
                }
                tmem_wait_st();
                tc_fence_before();
                if (warp == 0) ok = mbar_wait<1>(&S.y_full, u & 1, g, 2) && ok;
                if ((failed = any_failed(!ok))) break;   // every operand is there
                const int next = it + (int)gridDim.x;
                if (warp == 0) {
                    if (elect_leader()) load_sg(true, it, gi);
                    __syncwarp();
                    issue_first();
                }
                if (warp == 1) {
                    float bv[2], gv[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = t0 + 2 * lane + i;
                        bv[i] = t < p.N ? p.beta[rs.at(t)] : 0.f;
                        gv[i] = t < p.N && p.lg ? p.lg[rs.at(t)] : 0.f;
                    }
                    block_gates<false>(U.gates, bv, gv, lane);
                }
                if (u > 0) finish(last_it, last_gi, S.unit[~u & 1]);
                last_it = it;
                last_gi = gi;
                // ---- P, P^T and F from the scores; 16 columns of a row
                ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.pf_done, u & 1, g, 6));
                uint32_t sc[16];
                if (ok) {
                    tc_fence_after();
                    tmem_ld16(tb + lb + gPF + cg * 16, sc);
                    if (row >= 64) {
                        uint32_t sc2[16];
                        tmem_ld16(tb + lb + gPF + 64 + cg * 16, sc2);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) sc[j] = f2u(u2f(sc[j]) + u2f(sc2[j]));
                    }
                    tmem_wait_ld();
                    tc_fence_before();
                }
                ok = mbar_wait<1>(&S.sg_full, 1, g, 5) && ok;
                if ((failed = any_failed(!ok))) break;   // the scores have been read
                tc_fence_after();
                float gs = 0.f;   // this thread's terms of <G, S>
                if (live) {
#pragma unroll
                    for (int i = 0; i < SC; i += 16) {
                        float y[16];
                        row16(i, y);
                        const uint32_t col = tb + lb + gG + (cg * SC + i) / 2;
                        put_pieces(col, DV / 2, col + (gGl - gG), y);
#pragma unroll
                        for (int j = 0; j < 16; ++j) gs = fmaf(x[i + j], y[j], gs);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                if ((failed = any_failed(false))) break;   // G has been read
                // the next unit's values on their way
                const int nit = gi + 1 < group ? it : next, ngi = gi + 1 < group ? gi + 1 : 0;
                if (warp == 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.s_done, u & 1, g, 4));
                    if (ok) issue_g();
                }
                if (warp == 0 && ok && nit < p.items && elect_leader()) load_y(nit, ngi);   // dy has been used
                if (tid == kCopier && nit < p.items) {
                    const size_t nbh = head_of(nit, ngi), nt = nbh * p.N + nit % nblk * kDC;
                    const uint32_t bytes = min(kDC, p.N - nit % nblk * kDC) * DV * 4;
                    prefetch_l2(p.e + nt * DV, bytes);
                    prefetch_l2(p.du + nt * DV, bytes);
                    prefetch_l2(p.S_ck + (nbh * (nblk + 1) + nit % nblk) * st, D * DV * 4);
                    prefetch_l2(p.G_ck + (nbh * nblk + nit % nblk) * st, D * DV * 4);
                }
                __syncwarp();
                {
                    const int i = row & 63, j0 = cg * 16;
                    float w[16];
                    decayed16<false, false>(U.gates, i, j0, sc, w);
                    if (row < 64) {
                        uint32_t hi[8], mi[8], lo[8];
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = j0 + j <= i ? w[j] : 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) split3(w[2 * j], w[2 * j + 1], hi[j], mi[j], lo[j]);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint32_t o = sw128_off(i, j0 + 8 * q);
                            *reinterpret_cast<uint4 *>(sP + o) =
                                make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                            *reinterpret_cast<uint4 *>(sP + 8192 + o) =
                                make_uint4(mi[4 * q], mi[4 * q + 1], mi[4 * q + 2], mi[4 * q + 3]);
                            *reinterpret_cast<uint4 *>(sP + 16384 + o) =
                                make_uint4(lo[4 * q], lo[4 * q + 1], lo[4 * q + 2], lo[4 * q + 3]);
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t o = sw128_off(j0 + j, i), sh = (j & 1) * 16;
                            *reinterpret_cast<uint16_t *>(sPT + o) = (uint16_t)(hi[j >> 1] >> sh);
                            *reinterpret_cast<uint16_t *>(sPT + 8192 + o) = (uint16_t)(mi[j >> 1] >> sh);
                        }
                    } else {
                        const float nb = -U.gates.b[i];
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            uint32_t hi, mi;
                            split2(j0 + j < i ? nb * w[j] : 0.f, j0 + j + 1 < i ? nb * w[j + 1] : 0.f, hi, mi);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (j0 + j + e <= i) {   // both of F_ij and F_ji (zero on the diagonal)
                                    const uint32_t o = sw128_off(i, j0 + j + e), ot = sw128_off(j0 + j + e, i);
                                    const uint16_t a = (uint16_t)(hi >> (16 * e)), m = (uint16_t)(mi >> (16 * e));
                                    *reinterpret_cast<uint16_t *>(sF + o) = a;
                                    *reinterpret_cast<uint16_t *>(sF + 8192 + o) = m;
                                    *reinterpret_cast<uint16_t *>(sF + ot) = a;
                                    *reinterpret_cast<uint16_t *>(sF + 8192 + ot) = m;
                                }
                        }
                    }
                }
                fence_proxy_async();
                if (warp == 0) ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.kq_full, k & 1, g, 1));
                if ((failed = any_failed(!ok))) break;
                if (warp == 0) issue_second();
                // ---- gradients
                ok = mbar_wait<1>(&S.kq_full, k & 1, g, 7) && mbar_wait<1>(&S.all_done, u & 1, g, 8);
                if (!__all_sync(0xffffffffu, ok)) { failed = true; }
                if (!failed && tid == kCopier && nit < p.items) {   // e, du, P, P^T and F have been used
                    load_eu(nit, ngi);
                    load_sg(false, nit, ngi);
                }
                __syncwarp();
                float gw = 0.f;
                if (!failed && live) {
                    tc_fence_after();
                    const Gates &G = U.gates;
                    const int j0 = cg * 16;
                    uint32_t a[16], a2[16];
                    float c[16], w[16];
                    tmem_ld16(tb + lb + gQ + j0, a);
                    tmem_ld16(tb + lb + gQ2 + j0, a2);
                    load16(&G.c[j0], c);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float y = fmaf(c[j], u2f(a[j]), u2f(a2[j]));
                        dq[j] += y;
                        const uint16_t qv =
                            *reinterpret_cast<const uint16_t *>(sKQ + Lay::kT + (row >> 6) * 8192 + sw128_off(j0 + j, row & 63));
                        w[j] = y * __uint_as_float((uint32_t)qv << 16);
                    }
                    if (p.lg) {
                        const float s = reduce16(w, lane);
                        if (lane < 16) U.qdq[wq][j0 + lane] = s;
                    }
                    tmem_ld16(tb + lb + gGe + j0, a);
                    tmem_ld16(tb + lb + gSu + j0, a2);
                    load16(&G.w[j0], w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float y = w[j] * u2f(a[j]);
                        dk[j] += y;
                        const uint16_t kv =
                            *reinterpret_cast<const uint16_t *>(sKQ + (row >> 6) * 8192 + sw128_off(j0 + j, row & 63));
                        gw = fmaf(y, __uint_as_float((uint32_t)kv << 16), gw);
                    }
                    load16(&G.b[j0], w);
                    tmem_ld16(tb + lb + gK2 + j0, a);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) dk[j] += fmaf(-(w[j] * c[j]), u2f(a2[j]), u2f(a[j]));
                    tc_fence_before();
                }
                if (p.lg) {   // <G, S'> = c_C <G, S> + sum_j w_j (G e)_j . k_j
                    gs = warp_sum(fmaf(U.gates.cC, gs, gw));
                    if (lane == 0) U.gs[warp] = gs;
                }
                if (failed) {   // every warp meets at the next barrier, or at the end
                    any_failed(true);
                    break;
                }
            }
            if (failed) break;
            // ---- dq and dk: tokens x features
            if (live) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t o = sw128_off(cg * 16 + j, row & 63);
                    *reinterpret_cast<__nv_bfloat16 *>(sDQ + (row >> 6) * Lay::kDQ + o) = __float2bfloat16_rn(dq[j]);
                    *reinterpret_cast<__nv_bfloat16 *>(sDK + (row >> 6) * 8192 + o) = __float2bfloat16_rn(dk[j]);
                }
            }
            fence_proxy_async();
            if ((failed = any_failed(false))) break;
            if (tid == kCopier) {
#pragma unroll
                for (int f = 0; f < D / 64; ++f) {
                    tma_store_4d(&dqmap, sDQ + f * Lay::kDQ, f * 64, t0, hk, b);
                    tma_store_4d(&dkmap, sDK + f * 8192, f * 64, t0, hk, b);
                }
                bulk_commit();
                if (it + (int)gridDim.x < p.items) load_kq(it + (int)gridDim.x);   // K and Q have been used
            }
        }
        if (!failed && u > 0) finish(last_it, last_gi, S.unit[~u & 1]);   // behind the last item's barrier
        if (tid == kCopier) bulk_wait<0>();
        if (failed && warp == 0) {   // let MMAs and copies in flight finish
            __syncwarp();
            if (elect_leader()) mma_commit(&S.drained);
            const uint64_t until = globaltimer_ns() + 1000000000ull;
            auto done = [](uint64_t *bar, int n) { return n == 0 || mbar_try_wait(bar, (n - 1) & 1); };
            while (globaltimer_ns() < until &&
                   !(done(&S.kq_full, S.loads[0]) && done(&S.y_full, S.loads[1]) &&
                     done(&S.sg_full, S.loads[2]) && done(&S.eu_full, S.loads[3]) && mbar_try_wait(&S.drained, 0))) {}
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

template <int D, int DV, bool ONE> cudaError_t launch_grad_tc(const DeltaArgs &a) {
    CUtensorMap qm, km, ym, dqm, dkm, sm, gm;
    const DeltaBwdWs w = delta_bwd_ws(a);
    const int nblk = delta_blocks(a.N), BH = a.B * a.H;
    if (!encode_tokens(&qm, a.q, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&km, a.k, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&ym, a.dy, a.layout, a.B, a.H, a.N, DV) ||
        !encode_tokens(&dqm, a.dq, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&dkm, a.dk, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_3d(&sm, w.S, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, DV, D, BH * (nblk + 1), 32, D,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_3d(&gm, w.G, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, DV, D, BH * nblk, 32, D,
                   CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    GradTc p{};
    p.beta = a.beta; p.lg = a.log_gate;
    p.S_ck = w.S; p.G_ck = w.G; p.e = w.e; p.du = w.du;
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.dv = static_cast<__nv_bfloat16 *>(a.dv_grad);
    p.dbeta = a.dbeta; p.dlg = a.dlog_gate;
    p.H = a.H; p.Hk = a.Hk; p.N = a.N; p.layout = a.layout; p.nblk = nblk;
    p.items = p.nblk * a.B * a.Hk;
    WsHeader *hdr = static_cast<WsHeader *>(a.ws);
    p.err = &hdr->error;
    p.err_where = &hdr->error_where;
    const long long lim = debug_fault().wait_limit_ns;
    p.limit_ns = lim > 0 ? (unsigned long long)lim : 1000000000ull;
    auto kern = delta_grad_tc_kernel<D, DV, ONE>;
    constexpr int smem = GradLay<D, DV>::request;
    static_assert(smem <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int sms = num_sms();
    kern<<<p.items < sms ? p.items : sms, kGThr, smem, a.stream>>>(qm, km, ym, dqm, dkm, sm, gm, p);
    return cudaGetLastError();
}

template <bool ONE> cudaError_t launch_grad_dims(const DeltaArgs &a) {
    if (a.d == 64) return a.dv == 64 ? launch_grad_tc<64, 64, ONE>(a) : launch_grad_tc<64, 128, ONE>(a);
    return a.dv == 64 ? launch_grad_tc<128, 64, ONE>(a) : launch_grad_tc<128, 128, ONE>(a);
}

}  // namespace

cudaError_t launch_delta_grad_tc(const DeltaArgs &a) {
    return a.H == a.Hk ? launch_grad_dims<true>(a) : launch_grad_dims<false>(a);
}

}  // namespace la
