// delta_rev_tc.cu -- the reverse pass of the gated delta rule's gradients on the
// tensor cores (bf16 inputs, d and dv in {64, 128}): blocks of 64 tokens from
// the last to the first, one CTA per head.
//
// With G the gradient of the state after a block (notation of delta_tc.cu):
//     (I + b D' K K^T)^T du = D_C . (K G) + P0^T dy,   P0_ij = D_ij (q_i . k_j)  (j <= i),
//     G_before = c_C G + Q^T (c . dy) - K^T (b c . du),
// that is du = T^T (...) with T = (I + A)^-1, A_ij = b_i D_ij (k_i . k_j) below
// the diagonal.  The kernel writes du (float32) of every token and G after
// every block; the gradients themselves follow in delta_grad*.cu.
//
// It is the forward kernel run backwards, with its layout (a TMEM lane for
// each of the dv columns of G), its pieces and its roles.  Two operands come
// on top: dy^T P0 straight from the dy tile (exact bf16, dv-major), and c . dy
// as pieces, made beside the right-hand side by the warps of P0.  In TMEM the
// right-hand side takes the upper part of the place of G's pieces, c . dy the
// lower one, and -b c . du that of the right-hand side.  G is
// written while the next block's K G runs.
// B8 H16 N8192 d128: 0.69 ms (5.4 us a block; with c . dy made by the chain and G written
// in it, 0.13 ms more).
#include "delta_tc.cuh"

namespace la {
namespace {

constexpr uint32_t kColSP = 0, kColCY = 0, kColR = 96, kColW = 96;
constexpr uint32_t kColSD = 192;                // the change of G: D columns
constexpr uint32_t kColGK = 320;                // K G, then du
constexpr uint32_t kColPY = 384;                // P0^T dy
constexpr uint32_t kColKK = 448;

struct RevTc {
    const float *beta, *lg;
    int H, group, N, layout, nblk;
    int nseg, seg_blocks;          // segments of a head, blocks of one
    const float *G_end;            // by (head, segment); null: zero
    float *dS_in;
    float *G_ck, *du;
    float *G_local;                // LOCAL, by (head, segment)
    unsigned int *err, *err_where;
    unsigned long long limit_ns;
    int drop_item;
};
struct RevSmall {
    Gates gates[4];
    uint64_t kq_full[kStages], v_full[2], kk_full, kk_read, g_ready[2], t_ready[2], t_free[2], p_ready, ks_done,
        py_done, cy_ready, e_done, s_done, o_read, drain[3];
    uint32_t tmem_base;
    volatile int abort_flag;
};
template <int D, int DV> struct RevLay {
    static constexpr int kKQ = (D / 64) * 16384, kV = (DV / 64) * 8192, kT = 3 * 8192, kP = 3 * 8192;
    static constexpr int oKQ = 0, oV = oKQ + kStages * kKQ, oT = oV + 2 * kV, oP = oT + 2 * kT, oSmall = oP + kP;
    static constexpr int total = oSmall + (int)sizeof(RevSmall);
    static constexpr int request = total + 1024;
};

// n counts steps: step n is block nblk - 1 - n of the item's segment.  LOCAL: segments but the first
// of each head, from a zero G at their ends, leaving G at their starts and nothing else.
template <int D, int DV, bool LOCAL>
__global__ void __launch_bounds__(kChain + 2 * kInner + kOut, 1)
delta_rev_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap ymap, const RevTc p) {
    using Lay = RevLay<D, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    RevSmall &S = *reinterpret_cast<RevSmall *>(sm + Lay::oSmall);
    uint8_t *sKQ = sm + Lay::oKQ, *sV = sm + Lay::oV, *sT = sm + Lay::oT, *sP = sm + Lay::oP;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int segs = LOCAL ? p.nseg - 1 : p.nseg, bh = blockIdx.x / segs, seg = blockIdx.x - bh * segs + (LOCAL ? 1 : 0);
    const int b = bh / p.H, h = bh - b * p.H, hk = h / p.group;
    const int blk0 = seg * p.seg_blocks, nblk = min(p.seg_blocks, p.nblk - blk0);   // blocks of this item
    const size_t item = (size_t)bh * p.nseg + seg;
    const Guard g{&S.abort_flag, p.err, p.err_where, p.limit_ns};

    if (tid == 0) {
        S.abort_flag = 0;
        for (int i = 0; i < kStages; ++i) mbar_init(&S.kq_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.v_full[i], 1);
            mbar_init(&S.t_ready[i], kInner);
            mbar_init(&S.g_ready[i], 32);
            mbar_init(&S.t_free[i], 1);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&S.drain[i], 1);
        mbar_init(&S.kk_full, 1);
        mbar_init(&S.kk_read, 2 * kInner);   // a thread for each row of K, and of Q
        mbar_init(&S.p_ready, 64);
        mbar_init(&S.ks_done, 1);
        mbar_init(&S.py_done, 1);
        mbar_init(&S.cy_ready, kOut);
        mbar_init(&S.e_done, 1);
        mbar_init(&S.s_done, 1);
        mbar_init(&S.o_read, kOut);
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&ymap);
        prefetch_tmap(&qmap);
    }
    if (warp == 0) {
        tmem_alloc(&S.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, S.tmem_base, 0);
    const int wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lb = (uint32_t)(wq * 32) << 16;
    constexpr uint32_t i64 = idesc_bf16(128, kDC, 0, 0);

    if (warp < 8) {
        // ------------------------------------------------------------ chain
        constexpr uint32_t iS = idesc_bf16(128, D, 0, 1);      // B = K or Q, feature-major
        constexpr uint32_t iPY = idesc_bf16(128, kDC, 1, 0);   // A = dy, dv-major
        const int half = warp >> 2;
        const bool live = row < DV;
        constexpr int SC = D / 2;
        int kq_issued = 0, v_issued = 0;
        auto load_kq = [&](int n) {
            uint64_t *bar = &S.kq_full[n % kStages];
            mbar_arrive_expect_tx(bar, 2 * kDC * D * 2);
            ++kq_issued;
            if (n == 0 && (int)blockIdx.x == p.drop_item) return;   // test hook: announced, never issued
            uint8_t *dst = sKQ + (n % kStages) * Lay::kKQ;
            const int tok = (blk0 + nblk - 1 - n) * kDC;
#pragma unroll
            for (int f = 0; f < D / 64; ++f) {
                tma_load_4d(dst + f * 16384 + (n & 1) * 8192, &kmap, bar, f * 64, tok, hk, b);
                tma_load_4d(dst + f * 16384 + (~n & 1) * 8192, &qmap, bar, f * 64, tok, hk, b);
            }
        };
        auto load_v = [&](int n) {
            uint64_t *bar = &S.v_full[n & 1];
            mbar_arrive_expect_tx(bar, kDC * DV * 2);
            ++v_issued;
            uint8_t *dst = sV + (n & 1) * Lay::kV;
#pragma unroll
            for (int f = 0; f < DV / 64; ++f)
                tma_load_4d(dst + f * 8192, &ymap, bar, f * 64, (blk0 + nblk - 1 - n) * kDC, h, b);
        };
        if (warp == 0 && elect_leader()) {   // always the same lane: it keeps the counts
            for (int n = 0; n < kStages && n < nblk; ++n) {
                load_kq(n);
                if (n < 2) load_v(n);
            }
        }
        __syncwarp();
        float st[SC];
        const size_t sbase = (size_t)half * SC * DV + row;
#pragma unroll
        for (int i = 0; i < SC; ++i)
            st[i] = !LOCAL && live && p.G_end ? p.G_end[item * D * DV + sbase + (size_t)i * DV] : 0.f;
        auto write_state = [&](float *dst) {
#pragma unroll
            for (int i = 0; i < SC; ++i) dst[(size_t)i * DV] = st[i];
        };
        auto put_state = [&](int i0) {   // pieces of 16 columns
            uint32_t hi[8], mi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                split3(st[i0 + 2 * i], st[i0 + 2 * i + 1], hi[i], mi[i], lo[i]);
            const uint32_t col = tb + lb + kColSP + (half * SC + i0) / 2;
            tmem_st8(col, hi);
            tmem_st8(col + D / 2, mi);
            tmem_st8(col + D, lo);
        };
        float *gck = LOCAL ? nullptr : p.G_ck + ((size_t)bh * p.nblk + blk0 + nblk - 1) * D * DV + sbase;
        if (live) {
#pragma unroll
            for (int i = 0; i < SC; i += 16) put_state(i);
        }
        tmem_wait_st();
        tc_fence_before();
        // the group's agreement, uniform to the compiler as well
        auto any_failed = [](bool f) { return __any_sync(0xffffffffu, group_any<kBarChain, kChain>(f)) != 0; };
        bool failed = any_failed(false);

        for (int n = 0; n < nblk && !failed; ++n) {
            const uint32_t kk = smem_u32(sKQ) + (n % kStages) * Lay::kKQ + (n & 1) * 8192;     // K
            const uint32_t qq = smem_u32(sKQ) + (n % kStages) * Lay::kKQ + (~n & 1) * 8192;    // Q
            const Gates &G = S.gates[n & 3];
            bool ok = true;
            if (warp == 0) {
                ok = mbar_wait<1>(&S.kq_full[n % kStages], (n / kStages) & 1, g, 1);
                if (n > 0) ok = ok && mbar_wait<1>(&S.o_read, (n - 1) & 1, g, 2);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
                    // small pieces first: the accumulator truncates, relative to what it holds
#pragma unroll 1
                    for (int pc = 2; pc >= 0; --pc)
                        mma_rows<D / 16, 16384>(leader, tb + kColGK, tb + kColSP + pc * (D / 2), kk, i64, pc < 2);
                    mma_commit_if(leader, &S.ks_done);
                }
                ok = ok && mbar_wait<1>(&S.v_full[n & 1], (n >> 1) & 1, g, 3);
                ok = ok && mbar_wait<1>(&S.p_ready, n & 1, g, 8);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
                    // dv rows 64 .. 127 repeat the others where there are none
                    const uint64_t yd = smem_desc(smem_u32(sV) + (n & 1) * Lay::kV, DV > 64 ? 8192 : 0, 1024,
                                                  kSwizzle128B);
                    const uint64_t pd = desc_k(smem_u32(sP));
#pragma unroll 1
                    for (int pc = 2; pc >= 0; --pc)
#pragma unroll
                        for (int ks = 0; ks < kDC / 16; ++ks)
                            mma_ss_if(leader, tb + kColPY, yd + ks * 128, pd + pc * 512 + ks * 2, iPY,
                                      pc < 2 || ks > 0);
                    mma_commit_if(leader, &S.py_done);
                }
            }
            if (!LOCAL && live) write_state(gck);   // beside K G
            // ---- the right-hand side D_C . (K G) + P0^T dy
            ok = ok && mbar_wait<1>(&S.t_ready[n & 1], (n >> 1) & 1, g, 4);
            ok = ok && mbar_wait<1>(&S.ks_done, n & 1, g, 5);
            ok = ok && mbar_wait<1>(&S.py_done, n & 1, g, 6);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && live) {
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int j0 = half * 32 + u * 16;
                    uint32_t gk[16], py[16], hi[8], mi[8], lo[8];
                    float w[16], z[16];
                    tmem_ld16(tb + lb + kColGK + j0, gk);
                    tmem_ld16(tb + lb + kColPY + j0, py);
                    load16(&G.w[j0], w);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) z[j] = u2f(py[j]);
                    fma16(w, gk, z);
#pragma unroll
                    for (int i = 0; i < 8; ++i) split3(w[2 * i], w[2 * i + 1], hi[i], mi[i], lo[i]);
                    const uint32_t col = tb + lb + kColR + j0 / 2;
                    tmem_st8(col, hi);
                    tmem_st8(col + 32, mi);
                    tmem_st8(col + 64, lo);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            if ((failed = any_failed(!ok))) break;
            // ---- du = T^T (...)
            if (warp == 0) {
                const uint32_t leader = elect_leader();
                tc_fence_after();
                const uint32_t t = smem_u32(sT) + (n & 1) * Lay::kT;
                // the pieces (of the right-hand side, of T^T) but those whose product is below 2^-22 of
                // the whole, small ones first: (2, 0) (0, 2) (1, 1) (1, 0) (0, 1) (0, 0)
#pragma unroll 1
                for (int o = 0; o < 6; ++o) {
                    const int pr = (0x201100u >> (20 - 4 * o)) & 3, pt = (0x021010u >> (20 - 4 * o)) & 3;
                    mma_rows<kDC / 16, 0>(leader, tb + kColGK, tb + kColR + pr * 32, t + pt * 8192, i64, o > 0);
                }
                mma_commit_if(leader, &S.e_done);
                mma_commit_if(leader, &S.t_free[n & 1]);
            }
            const uint64_t kd = smem_desc(kk, 16384, 1024, kSwizzle128B), qd = smem_desc(qq, 16384, 1024, kSwizzle128B);
            if (warp == 0) {   // the small pieces of Q^T (c . dy); its large ones come with the others'
                ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.cy_ready, n & 1, g, 11));
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
#pragma unroll 1
                    for (int pc = 2; pc >= 1; --pc)
#pragma unroll
                        for (int ks = 0; ks < kDC / 16; ++ks)
                            mma_ts_if(leader, tb + kColSD, tb + kColCY + pc * 32 + ks * 8, qd + ks * 128, iS,
                                      pc < 2 || ks > 0);
                    if (leader && n + 2 < nblk) load_v(n + 2);   // dy has been read, P0^T dy is done
                    __syncwarp();
                }
            }
            // ---- -b c . du
            ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.e_done, n & 1, g, 7));
            if (ok && live) {
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int j0 = half * 32 + u * 16;
                    uint32_t acc[16], hi[8], mi[8], lo[8];
                    float w[16], c[16];
                    tmem_ld16(tb + lb + kColGK + j0, acc);
                    load16(&G.b[j0], w);
                    load16(&G.c[j0], c);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        f2unpack(f2mul(f2pack(-w[j], -w[j + 1]), f2pack(c[j], c[j + 1])), w[j], w[j + 1]);
                    mul16(w, acc);
#pragma unroll
                    for (int i = 0; i < 8; ++i) split3(w[2 * i], w[2 * i + 1], hi[i], mi[i], lo[i]);
                    const uint32_t col = tb + lb + kColW + j0 / 2;
                    tmem_st8(col, hi);
                    tmem_st8(col + 32, mi);
                    tmem_st8(col + 64, lo);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            if ((failed = any_failed(!ok))) break;
            // ---- G = c_C G + Q^T (c . dy) - K^T (b c . du)
            if (warp == 0) {
                const uint32_t leader = elect_leader();
                tc_fence_after();
#pragma unroll 1
                for (int o = 0; o < 4; ++o) {   // small pieces of -b c . du, then the large ones of both
                    const uint32_t a = tb + (o == 2 ? kColCY : kColW + (o == 0 ? 64 : o == 1 ? 32 : 0));
                    const uint64_t d = o == 2 ? qd : kd;
#pragma unroll
                    for (int ks = 0; ks < kDC / 16; ++ks)
                        mma_ts_if(leader, tb + kColSD, a + ks * 8, d + ks * 128, iS, 1);
                }
                mma_commit_if(leader, &S.s_done);
            }
            ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.s_done, n & 1, g, 9));
            if (warp == 0 && ok && n + kStages < nblk) {
                if (elect_leader()) load_kq(n + kStages);
                __syncwarp();
            }
            if (ok && live) {
                tc_fence_after();
                const uint64_t cC2 = f2pack(G.cC, G.cC);
#pragma unroll
                for (int i = 0; i < SC; i += 16) {
                    uint32_t acc[16];
                    tmem_ld16(tb + lb + kColSD + half * SC + i, acc);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        f2unpack(f2fma(cC2, f2pack(st[i + j], st[i + j + 1]), f2pack(u2f(acc[j]), u2f(acc[j + 1]))),
                                 st[i + j], st[i + j + 1]);
                    if (n + 1 < nblk) put_state(i);
                }
                tmem_wait_st();
                tc_fence_before();
                if (!LOCAL) gck -= D * DV;
            }
            failed = any_failed(!ok);
        }
        if (LOCAL) {
            if (!failed && live) write_state(p.G_local + item * D * DV + sbase);
        } else if (!failed && live && p.dS_in && seg == 0) {
            write_state(p.dS_in + (size_t)bh * D * DV + sbase);
        }
        if (warp == 0 && elect_leader()) {
            mma_commit(&S.drain[0]);
            drain_wait(&S.drain[0], 0, g.limit_ns);
            if (S.abort_flag) {   // let the copies in flight land
                for (int n = max(0, kq_issued - kStages); n < kq_issued; ++n)
                    if (!(n == 0 && (int)blockIdx.x == p.drop_item))
                        drain_wait(&S.kq_full[n % kStages], (n / kStages) & 1, g.limit_ns);
                for (int n = max(0, v_issued - 2); n < v_issued; ++n)
                    drain_wait(&S.v_full[n & 1], (n >> 1) & 1, g.limit_ns);
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        // ------------------------------------------------------------ T, ahead of the chain
        const TokenRows rs = token_rows(p.layout, b, h, p.H, p.N, 1);
        const int grp = (warp - 8) >> 1, t = tid - kChain - grp * kInner, bar = kBarInner + grp;
        uint8_t *sTg = sT + grp * Lay::kT;
        float *A = reinterpret_cast<float *>(sTg);
        const bool gates_warp = (warp & 1) != 0;
        float bv[2], gv[2];   // gates warp: the next block's beta and log gates
        auto fetch = [&](int n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = (blk0 + nblk - 1 - n) * kDC + 2 * lane + i;
                bv[i] = tok < p.N ? p.beta[rs.at(tok)] : 0.f;
                gv[i] = tok < p.N && p.lg ? p.lg[rs.at(tok)] : 0.f;
            }
        };
        auto any_out = [&](bool f) {
            uint32_t r;
            asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                         "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                         : "=r"(r) : "r"((uint32_t)f), "r"(bar), "n"(kInner) : "memory");
            return __any_sync(0xffffffffu, r != 0) != 0;
        };
        if (gates_warp) fetch(grp);
        for (int n = grp; n < nblk; n += 2) {
            // T of step n - 2 has been used: its place is free, and so are gates[n & 3]
            Gates &G = S.gates[n & 3];
            bool ok = n < 2 || mbar_wait<1>(&S.t_free[grp], ((n >> 1) - 1) & 1, g, 23);
            // the block before's [K; Q] K^T and gates have been read
            if (n > 0) ok = ok && mbar_wait<1>(&S.kk_read, (n - 1) & 1, g, 24);
            if (!gates_warp) {
                ok = ok && mbar_wait<1>(&S.kq_full[n % kStages], (n / kStages) & 1, g, 20);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
                    const uint32_t base = smem_u32(sKQ) + (n % kStages) * Lay::kKQ;
                    const uint64_t ad = desc_k(base), kd = desc_k(base + grp * 8192);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                        mma_ss_if(leader, tb + kColKK, ad + o, kd + o, i64, ks > 0);
                    }
                    mma_commit_if(leader, &S.kk_full);
                }
            } else {
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    block_gates<true>(G, bv, gv, lane);
                    mbar_arrive(&S.g_ready[grp]);
                    if (n + 2 < nblk) fetch(n + 2);
                }
            }
            ok = ok && mbar_wait<1>(&S.g_ready[grp], (n >> 1) & 1, g, 25);
            ok = ok && mbar_wait<1>(&S.kk_full, n & 1, g, 21);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {   // A_ij = b_i D_ij (k_i . k_j), j < i
                tc_fence_after();
#pragma unroll 1
                for (int j0 = 0; j0 < kDC; j0 += 16) {
                    float x[16];
                    if (j0 >= (t | 31)) {   // warp-uniform: above the diagonal
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = 0.f;
                    } else {
                        uint32_t acc[16];
                        tmem_ld16(tb + lb + kColKK + j0, acc);
                        decayed16<true, true>(G, t, j0, acc, x);
                        const float bt = G.b[t];
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = j0 + j < t ? bt * x[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(A + t * kAP + j0 + j) =
                            make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
                tc_fence_before();
                mbar_arrive(&S.kk_read);
            }
            if (any_out(!ok)) break;   // A complete
            invert_unit_lower<false>(A, t, bar, nullptr);
            // T^T's pieces over A: a thread's row (T's column) is in registers before any is written
            float x[kDC];
#pragma unroll
            for (int j = 0; j < kDC; ++j) x[j] = A[j * kAP + t];
            named_bar(bar, kInner);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t hi[4], mi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split3(x[8 * q + 2 * e], x[8 * q + 2 * e + 1], hi[e], mi[e], lo[e]);
                const uint32_t o = sw128_off(t, 8 * q);
                *reinterpret_cast<uint4 *>(sTg + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(sTg + 8192 + o) = make_uint4(mi[0], mi[1], mi[2], mi[3]);
                *reinterpret_cast<uint4 *>(sTg + 16384 + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async();
            mbar_arrive(&S.t_ready[grp]);
        }
        if (!gates_warp && elect_leader()) {
            mma_commit(&S.drain[1 + grp]);
            drain_wait(&S.drain[1 + grp], 0, g.limit_ns);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ P0^T, and du to memory
        // P0_ij = D_ij (q_i . k_j), j <= i, by the warps whose lanes hold the rows of Q, stored by
        // columns; made for the next step once this one's has been used.
        uint32_t sc[4][16];
        auto rows_of_q = [&](int n) { return (row >> 6) != (n & 1); };
        auto read_scores = [&](int n) {
            // the gates' phase too before arriving at kk_read, which lets the next block's gates come
            const bool ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.g_ready[n & 1], (n >> 1) & 1, g, 26) &&
                                                        mbar_wait<1>(&S.kk_full, n & 1, g, 27));
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < 4; ++u) tmem_ld16(tb + lb + kColKK + 16 * u, sc[u]);
                tmem_wait_ld();
                tc_fence_before();
                mbar_arrive(&S.kk_read);
            }
            return ok;
        };
        auto make_p = [&](int n) {
            const Gates &G = S.gates[n & 3];
            const int i = row & 63;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x[16];
                decayed16<false, true>(G, i, 16 * u, sc[u], x);
                uint8_t *at = sP + 16 * u * 128 + (i & 7) * 2;   // row j, column i
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    uint32_t hi, mi, lo;
                    split3(16 * u + j <= i ? x[j] : 0.f, 16 * u + j + 1 <= i ? x[j + 1] : 0.f, hi, mi, lo);
                    uint8_t *a0 = at + j * 128 + (((i >> 3) ^ (j & 7)) << 4);
                    uint8_t *a1 = at + (j + 1) * 128 + (((i >> 3) ^ ((j + 1) & 7)) << 4);
                    *reinterpret_cast<uint16_t *>(a0) = (uint16_t)hi;
                    *reinterpret_cast<uint16_t *>(a0 + 8192) = (uint16_t)mi;
                    *reinterpret_cast<uint16_t *>(a0 + 16384) = (uint16_t)lo;
                    *reinterpret_cast<uint16_t *>(a1) = (uint16_t)(hi >> 16);
                    *reinterpret_cast<uint16_t *>(a1 + 8192) = (uint16_t)(mi >> 16);
                    *reinterpret_cast<uint16_t *>(a1 + 16384) = (uint16_t)(lo >> 16);
                }
            }
            fence_proxy_async();
            mbar_arrive(&S.p_ready);
        };
        bool ok = true;
        if (rows_of_q(0)) {
            ok = read_scores(0);
            if (ok) make_p(0);
        }
        for (int n = 0; n < nblk; ++n) {
            const bool q_next = rows_of_q(n + 1), p_next = q_next && n + 1 < nblk;
            // these gates, seen by the other half when it made P; the next ones' phase cannot end before
            if (q_next) ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.g_ready[n & 1], (n >> 1) & 1, g, 28));
            if (p_next) ok = ok && read_scores(n + 1);
            // ---- c . dy, where G's pieces were
            ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.ks_done, n & 1, g, 29) &&
                                                   mbar_wait<1>(&S.v_full[n & 1], (n >> 1) & 1, g, 10));
            if (ok) {
                if (row < DV) {
                    tc_fence_after();
                    const float *c_of = S.gates[n & 3].c;
                    const uint8_t *ty = sV + (n & 1) * Lay::kV + (row >> 6) * 8192 + (row & 7) * 2;
                    const uint32_t ch = (uint32_t)(row & 63) >> 3;
#pragma unroll 1
                    for (int j0 = 0; j0 < kDC; j0 += 16) {
                        uint32_t hi[8], mi[8], lo[8];
                        float r[16], c[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r[j] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(
                                       ty + (j0 + j) * 128 + ((ch ^ (j & 7)) << 4)) << 16);
                        load16(c_of + j0, c);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            split3(c[2 * i] * r[2 * i], c[2 * i + 1] * r[2 * i + 1], hi[i], mi[i], lo[i]);
                        const uint32_t col = tb + lb + kColCY + j0 / 2;
                        tmem_st8(col, hi);
                        tmem_st8(col + 32, mi);
                        tmem_st8(col + 64, lo);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
                mbar_arrive(&S.cy_ready);
            }
            if (p_next) {   // where this step's has been used
                ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.py_done, n & 1, g, 31));
                if (ok) make_p(n + 1);
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait<1>(&S.e_done, n & 1, g, 30));
            if (!ok) break;
            tc_fence_after();
            if (!LOCAL && row < DV) {
                const int t0 = (blk0 + nblk - 1 - n) * kDC, in = p.N - t0;
                float *dst = p.du + ((size_t)bh * p.N + t0) * DV + row;
#pragma unroll 1
                for (int j0 = 0; j0 < kDC; j0 += 16) {
                    uint32_t acc[16];
                    tmem_ld16(tb + lb + kColGK + j0, acc);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j0 + j < in) dst[(size_t)j * DV] = u2f(acc[j]);
                    dst += 16 * DV;
                }
                tc_fence_before();
            }
            mbar_arrive(&S.o_read);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
    // what follows in the stream waits for this kernel, and so for the states' pass beside it
    griddep_wait();
}

template <int D, int DV, bool LOCAL>
cudaError_t launch_rev(const DeltaArgs &a, int nseg, int seg_blocks, const float *G_end, float *G_local) {
    CUtensorMap qm, km, ym;
    if (!encode_tokens(&qm, a.q, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&km, a.k, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&ym, a.dy, a.layout, a.B, a.H, a.N, DV))
        return cudaErrorInvalidValue;
    const DeltaBwdWs w = delta_bwd_ws(a);
    RevTc p{};
    p.beta = a.beta; p.lg = a.log_gate;
    p.H = a.H; p.group = a.H / a.Hk; p.N = a.N; p.layout = a.layout; p.nblk = delta_blocks(a.N);
    p.nseg = nseg; p.seg_blocks = seg_blocks;
    p.G_end = G_end; p.dS_in = a.dS_in; p.G_local = G_local;
    p.G_ck = w.G; p.du = w.du;
    WsHeader *hdr = static_cast<WsHeader *>(a.ws);
    p.err = &hdr->error;
    p.err_where = &hdr->error_where;
    const long long lim = debug_fault().wait_limit_ns;
    p.limit_ns = lim > 0 ? (unsigned long long)lim : 1000000000ull;
    p.drop_item = debug_fault().drop_load_item;
    auto kern = delta_rev_kernel<D, DV, LOCAL>;
    constexpr int smem = RevLay<D, DV>::request;
    static_assert(smem <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // beside the pass launched before it, of which it needs nothing, where the heads leave SMs idle
    return launch_overlapped(kern, dim3(a.B * a.H * (LOCAL ? nseg - 1 : nseg)), dim3(kChain + 2 * kInner + kOut),
                             smem, a.stream, qm, km, ym, p);
}
template <int D, int DV>
cudaError_t launch_rev_any(const DeltaArgs &a, int nseg, int seg_blocks, const float *G_end, float *G_local) {
    return G_local ? launch_rev<D, DV, true>(a, nseg, seg_blocks, G_end, G_local)
                   : launch_rev<D, DV, false>(a, nseg, seg_blocks, G_end, G_local);
}

}  // namespace

cudaError_t launch_delta_reverse_tc(const DeltaArgs &a, int nseg, int seg_blocks, const float *G_end, float *G_local) {
    if (a.d == 64)
        return a.dv == 64 ? launch_rev_any<64, 64>(a, nseg, seg_blocks, G_end, G_local)
                          : launch_rev_any<64, 128>(a, nseg, seg_blocks, G_end, G_local);
    return a.dv == 64 ? launch_rev_any<128, 64>(a, nseg, seg_blocks, G_end, G_local)
                      : launch_rev_any<128, 128>(a, nseg, seg_blocks, G_end, G_local);
}

}  // namespace la
