// delta_tc.cu -- the gated delta rule on the tensor cores (bf16 inputs, d and
// dv in {64, 128}): blocks of C = 64 tokens, one CTA per head.
//
// With c_i the product of the block's gates up to token i, D_ij = c_i / c_j
// and S the state before the block, the errors e of a block's tokens solve
//     (I + M) e = v - c . (K S),     M_ij = D_ij (k_i . k_j) b_j  (j < i),
// and with T = (I + M)^-1 (unit lower triangular)
//     e  = T (v - c . (K S)),
//     y  = c . (Q S) + P e,          P_ij = D_ij (q_i . k_j) b_j  (j <= i),
//     S' = c_C S + K^T W,            W_j = D_Cj b_j e_j.
// Everything that meets the state is held transposed, a TMEM lane for each of
// the dv columns of S: S^T, e^T and y^T are accumulators whose rows one thread
// reads, scales and writes back as the next product's TMEM operand, so the
// chain S -> K S -> e -> S' never leaves TMEM and registers.
//
// Precision: states, e and T are float32 values.  A float32 operand enters
// the MMAs as three bf16 pieces that add up to it exactly (the top, middle and
// low 8 bits of its significand, by truncation: the middle one is below 2^-7
// of it, the low one below 2^-15), so K S and K^T W, whose other
// operand is the bf16 input itself, lose nothing but the accumulator's
// float32 rounding, and T r drops the middle by low products, each below 2^-22
// of its term and of its sign (2^-24.7 of it on average).
// What only y depends on, which is rounded to bf16 anyway, takes two pieces:
// of the state in Q S the top two (less than 2^-15 is left, always of its sign), of P and
// e in P e two rounded to nearest (2^-17 is left of each, at most).
//
// Roles (16 warps): warps 0-7 carry the chain (two threads a row, each half of
// the columns; the float32 state lives in their registers); warps 8 and 9 turn
// K K^T of the even blocks into T, warps 10 and 11 that of the odd ones, both
// ahead of the chain; warps 12-15 turn Q K^T into P (two of them), make P e and
// write y.
// Bound by the chain of a block, about 9 K cycles of which the tensor pipe is
// busy a third: B8 H16 N8192 d128 0.62 ms, 1.8 TB/s; B1 H32 N131072 d64, split
// in four, 3.5 ms.
// What is not finite must reach no token before its own, but the MMAs run over whole blocks, in which the
// zeros above the diagonals of T and P meet later tokens' r and e.  So the kernel notes a row of y that is not
// finite, and a CTA with one runs again, with CARE: there a thread leaves out what follows the first value of
// its row of r or e that is not finite, and y and the state become NaN from there on.  (Those checks in every
// run took 8 to 10% of its time, the loops' code being as large as the instruction cache; a second launch for
// the second run took 4 us of the host's time a call; this takes 1% of B8 H16 N8192 d128, 609 -> 617 us.)
// The rows of [K; Q] K^T are TMEM lanes, which a warp reaches by its number
// mod 4: so odd blocks hold Q before K.  The chain's first warp issues its
// MMAs and the TMA loads.
#include "delta_tc.cuh"

namespace la {
namespace {

// TMEM columns.  The state's pieces take SP .. SP + 3 D/2; once K S and Q S
// are done, their place serves W (SP) and the pieces of e for P e (SP + 96).
// The residual r takes the place of K^T W, which comes after it.
constexpr uint32_t kColSP = 0, kColW = 0, kColE = 96;
constexpr uint32_t kColSD = 192, kColR = 192;   // K^T W: D columns
constexpr uint32_t kColKS = 320;                // K S, then T r, then P e
constexpr uint32_t kColQS = 384;
constexpr uint32_t kColKK = 448;                // [K; Q] K^T or, for odd blocks, [Q; K] K^T

struct DeltaTc {
    const float *beta, *lg;
    int H, group, N, layout, nblk;
    int nseg, seg_blocks;          // segments of a head, blocks of one
    int seg_items, parts;          // kSegment: segments of a head it takes, CTAs of one
    const float *S_in;             // by (head, segment)
    float *S_out;                  // by head
    float *S_ck, *e;               // kSave
    float *S_local, *Phi;          // kSegment, by (head, its segment)
    unsigned int *err, *err_where;
    unsigned long long limit_ns, stall_ns;   // stall_ns, drop_item: test hooks
    int drop_item;
};

struct DeltaSmall {
    Gates gates[4];
    uint64_t kq_full[kStages], v_full[2], kk_full, kk_read[2], g_ready[2], t_ready[2], t_free[2], p_ready, ks_done, qs_done, e_done, s_done, e_read, r_ready, pu_done, o_read, drain[4];
    int first[2][128];   // CARE, by half of the tokens and row of r: its first value that is not finite, or kDC
    int cut[128];        // CARE, by row of y: the first that is not finite, where the warp has one
    int t_bad[2][2];     // CARE, by T group and turn: the first row of T that is not what it should be, or kDC
    int y_bad;           // y is not finite somewhere
    uint32_t tmem_base;
    volatile int abort_flag;
};

template <int D, int DV> struct DeltaLay {
    static constexpr int kKQ = (D / 64) * 16384;      // per 64 features: K and Q rows, odd blocks Q first
    static constexpr int kV = (DV / 64) * 8192;
    static constexpr int kT = 3 * 8192, kP = 2 * 8192;   // T's place first holds A, [64][kAP] floats
    static constexpr int oKQ = 0, oV = oKQ + kStages * kKQ, oT = oV + 2 * kV, oP = oT + 2 * kT,
                         oY = oP + kP, oSmall = oY + kV;
    static constexpr int total = oSmall + (int)sizeof(DeltaSmall);
    static constexpr int request = total + 1024;
};

// What a launch computes.
enum DeltaMode {
    kForward,   // y, from the initial state of each (head, segment)
    kSave,      // the backward's first pass: e, and the state before every block and after the last
    kSegment    // segments from an empty state (rows < dv), and the segments' maps of the state:
                // S_end = Phi S_start + S_local, row dv + a being column a of Phi (from a unit state,
                // without values); `parts` CTAs of 128 rows each
};

template <bool Y> __device__ __forceinline__ void init_barriers(DeltaSmall &S) {
    for (int i = 0; i < kStages; ++i) mbar_init(&S.kq_full[i], 1);
    for (int i = 0; i < 2; ++i) {
        mbar_init(&S.v_full[i], 1);
        mbar_init(&S.t_ready[i], kInner);
        mbar_init(&S.g_ready[i], 32);
        mbar_init(&S.t_free[i], 1);
        mbar_init(&S.kk_read[i], Y ? 2 * kInner : kInner);   // a thread for each row of K, and of Q
    }
    for (int i = 0; i < 4; ++i) mbar_init(&S.drain[i], 1);
    mbar_init(&S.kk_full, 1);
    mbar_init(&S.p_ready, 64);
    mbar_init(&S.ks_done, 1);
    mbar_init(&S.qs_done, 1);
    mbar_init(&S.e_done, 1);
    mbar_init(&S.s_done, 1);
    mbar_init(&S.e_read, 1);
    mbar_init(&S.r_ready, 1);
    mbar_init(&S.pu_done, 1);
    mbar_init(&S.o_read, kOut);
    fence_mbar_init();
}

// The launch's shared memory, aligned by an offset, so that the compiler still sees shared memory.
__device__ __forceinline__ uint8_t *aligned_smem() {
    extern __shared__ uint8_t smem_raw[];
    return smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
}

// One run over an item: what each warp does.
template <int D, int DV, int MODE, bool CARE>
__device__ __forceinline__ void delta_run(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                          const CUtensorMap &ymap, const DeltaTc &p) {
    using Lay = DeltaLay<D, DV>;
    uint8_t *sm = aligned_smem();
    DeltaSmall &S = *reinterpret_cast<DeltaSmall *>(sm + Lay::oSmall);
    const uint32_t tb = __shfl_sync(0xffffffffu, S.tmem_base, 0);
    uint8_t *sKQ = sm + Lay::oKQ, *sV = sm + Lay::oV, *sT = sm + Lay::oT, *sP = sm + Lay::oP,
            *sY = sm + Lay::oY;
    // warp-uniform to the compiler too
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    constexpr bool Y = MODE == kForward, SAVE = MODE == kSave, SEG = MODE == kSegment;
    const int part = SEG ? blockIdx.x % p.parts : 0, item = SEG ? blockIdx.x / p.parts : blockIdx.x;
    const int segs = SEG ? p.seg_items : p.nseg, bh = item / segs, seg = item - bh * segs;
    const int b = bh / p.H, h = bh - b * p.H, hk = h / p.group;
    const int blk0 = seg * p.seg_blocks, nblk = min(p.seg_blocks, p.nblk - blk0);   // blocks of this item
    const Guard g{&S.abort_flag, p.err, p.err_where, p.limit_ns};

    // the state over the one that a second run starts from: not before it is known that there is none
    const bool in_place = Y && !CARE && p.S_out && p.S_in == p.S_out;
    const int wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lb = (uint32_t)(wq * 32) << 16;
    constexpr uint32_t i64 = idesc_bf16(128, kDC, 0, 0);

    if (warp < 8) {
        // ------------------------------------------------------------ chain
        constexpr uint32_t iS = idesc_bf16(128, D, 0, 1);   // B = K, feature-major
        const int half = warp >> 2;
        // column of S, or (SEG) dv + column of Phi; warp-uniform what it is
        const int col_of = part * 128 + row;
        const bool live = col_of < (SEG ? DV + D : DV), values = col_of < DV;
        constexpr int SC = D / 2;     // state columns of a thread
        int kq_issued = 0, v_issued = 0;
        auto load_kq = [&](int n) {
            uint64_t *bar = &S.kq_full[n % kStages];
            mbar_arrive_expect_tx(bar, (Y ? 2 : 1) * kDC * D * 2);
            ++kq_issued;
            if (n == 0 && (int)blockIdx.x == p.drop_item) return;   // test hook: announced, never issued
            uint8_t *dst = sKQ + (n % kStages) * Lay::kKQ;
#pragma unroll
            for (int f = 0; f < D / 64; ++f) {
                tma_load_4d(dst + f * 16384 + (n & 1) * 8192, &kmap, bar, f * 64, (blk0 + n) * kDC, hk, b);
                if (Y)
                    tma_load_4d(dst + f * 16384 + (~n & 1) * 8192, &qmap, bar, f * 64, (blk0 + n) * kDC, hk, b);
            }
        };
        auto load_v = [&](int n) {
            uint64_t *bar = &S.v_full[n & 1];
            mbar_arrive_expect_tx(bar, kDC * DV * 2);
            ++v_issued;
            uint8_t *dst = sV + (n & 1) * Lay::kV;
#pragma unroll
            for (int f = 0; f < DV / 64; ++f)
                tma_load_4d(dst + f * 8192, &vmap, bar, f * 64, (blk0 + n) * kDC, h, b);
        };
        if (warp == 0 && elect_leader()) {   // always the same lane: it keeps the counts
            for (int n = 0; n < kStages && n < nblk; ++n) {
                load_kq(n);
                if (n < 2) load_v(n);
            }
        }
        __syncwarp();
        // the state, its column `row`, rows half * SC ..
        float st[SC];
        const size_t sbase = (size_t)item * D * DV + (size_t)half * SC * DV + row;
#pragma unroll
        for (int i = 0; i < SC; ++i)
            st[i] = SEG ? (half * SC + i == col_of - DV ? 1.f : 0.f)
                        : live && p.S_in ? p.S_in[sbase + (size_t)i * DV] : 0.f;
        auto write_state = [&](float *dst, int ld) {   // dst: a [D][ld] matrix, at row half * SC, a column
#pragma unroll
            for (int i = 0; i < SC; ++i) dst[(size_t)i * ld] = st[i];
        };
        // where the states before this item's blocks go; the next item writes the one behind its last
        float *sck = SAVE ? p.S_ck + ((size_t)bh * (p.nblk + 1) + blk0) * D * DV + (size_t)half * SC * DV + row
                          : nullptr;
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
            const uint32_t kk = smem_u32(sKQ) + (n % kStages) * Lay::kKQ + (n & 1) * 8192;   // K
            const Gates &G = S.gates[n & 3];
            bool ok = true;
            if (warp == 0) {
                ok = mbar_wait<1>(&S.kq_full[n % kStages], (n / kStages) & 1, g, 1);
                if (Y && n > 0) ok = ok && mbar_wait<1>(&S.o_read, (n - 1) & 1, g, 2);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
                    // small pieces first: the accumulator truncates, relative to what it holds
#pragma unroll 1
                    for (int pc = 2; pc >= 0; --pc)
                        mma_rows<D / 16, 16384>(leader, tb + kColKS, tb + kColSP + pc * (D / 2), kk, i64, pc < 2);
                    mma_commit_if(leader, &S.ks_done);
                }
            }
            if (SAVE && live) write_state(sck, DV);   // beside K S
            // ---- r = v - c . (K S)
            ok = ok && mbar_wait<1>(&S.v_full[n & 1], (n >> 1) & 1, g, 3);
            ok = ok && mbar_wait<1>(&S.t_ready[n & 1], (n >> 1) & 1, g, 4);
            ok = ok && mbar_wait<1>(&S.ks_done, n & 1, g, 5);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && live) {
                tc_fence_after();
                // v of token j: chunk (row / 8) ^ (j % 8) of the token's 128-byte row
                const uint8_t *tv = sV + (n & 1) * Lay::kV + (row >> 6) * 8192 + half * 32 * 128 + (row & 7) * 2;
                const uint32_t ch = (uint32_t)(row & 63) >> 3;
                int first = kDC;
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int j0 = half * 32 + u * 16;
                    uint32_t acc[16], hi[8], mi[8], lo[8];
                    tmem_ld16(tb + lb + kColKS + j0, acc);
                    float r[16], c[16];
                    if (!SEG || values) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            r[j] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(
                                       tv + (u * 16 + j) * 128 + ((ch ^ (j & 7)) << 4)) << 16);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = 0.f;
                    }
                    load16(&G.c[j0], c);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) c[j] = -c[j];
                    fma16(c, acc, r);
                    if (CARE) cut16(c, j0, first);
#pragma unroll
                    for (int i = 0; i < 8; ++i) split3(c[2 * i], c[2 * i + 1], hi[i], mi[i], lo[i]);
                    const uint32_t col = tb + lb + kColR + j0 / 2;
                    tmem_st8(col, hi);
                    tmem_st8(col + 32, mi);
                    tmem_st8(col + 64, lo);
                }
                if (CARE) S.first[half][row] = first;
                tmem_wait_st();
                tc_fence_before();
            }
            if ((failed = any_failed(!ok))) break;
            // ---- e = T r
            if (warp == 0) {
                const uint32_t leader = elect_leader();
                tc_fence_after();
                const uint32_t t = smem_u32(sT) + (n & 1) * Lay::kT;
                // the pieces (r, T) but those whose product is below 2^-22 of the whole, small ones first:
                // (2, 0) (0, 2) (1, 1) (1, 0) (0, 1) (0, 0)
#pragma unroll 1
                for (int o = 0; o < 6; ++o) {
                    const int pr = (0x201100u >> (20 - 4 * o)) & 3, pt = (0x021010u >> (20 - 4 * o)) & 3;
                    mma_rows<kDC / 16, 0>(leader, tb + kColKS, tb + kColR + pr * 32, t + pt * 8192, i64, o > 0);
                }
                mma_commit_if(leader, &S.e_done);
                mma_commit_if(leader, &S.t_free[n & 1]);
                if (Y) {
                    const uint32_t qq = smem_u32(sKQ) + (n % kStages) * Lay::kKQ + (~n & 1) * 8192;
#pragma unroll 1
                    for (int pc = 1; pc >= 0; --pc)
                        mma_rows<D / 16, 16384>(leader, tb + kColQS, tb + kColSP + pc * (D / 2), qq, i64, pc < 1);
                    mma_commit_if(leader, &S.qs_done);
                }
                if (CARE && leader) mbar_arrive(&S.r_ready);
                if (leader && n + 2 < nblk) load_v(n + 2);   // every thread has read this block's v
                __syncwarp();
            }
            ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.e_done, n & 1, g, 7));
            if (ok && live) {
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int j0 = half * 32 + u * 16;
                    uint32_t acc[16], hi[8], mi[8], lo[8];
                    float w[16];
                    tmem_ld16(tb + lb + kColKS + j0, acc);
                    load16(&G.w[j0], w);
                    tmem_wait_ld();
                    mul16(w, acc);
                    if (CARE && min(S.first[0][row], S.first[1][row]) < kDC) w[0] = nan_f();
#pragma unroll
                    for (int i = 0; i < 8; ++i) split3(w[2 * i], w[2 * i + 1], hi[i], mi[i], lo[i]);
                    if (Y && u == 0) {   // W takes the place of the state's pieces
                        ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.qs_done, n & 1, g, 6));
                        if (!ok) break;
                    }
                    const uint32_t col = tb + lb + kColW + j0 / 2;
                    tmem_st8(col, hi);
                    tmem_st8(col + 32, mi);
                    tmem_st8(col + 64, lo);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            if ((failed = any_failed(!ok))) break;
            // ---- S' = c_C S + K^T W
            if (warp == 0) {
                const uint32_t leader = elect_leader();
                tc_fence_after();
                const uint64_t kd = smem_desc(kk, 16384, 1024, kSwizzle128B);
#pragma unroll 1
                for (int pc = 2; pc >= 0; --pc)
#pragma unroll
                    for (int ks = 0; ks < kDC / 16; ++ks)
                        mma_ts_if(leader, tb + kColSD, tb + kColW + pc * 32 + ks * 8, kd + ks * 128, iS,
                                  pc < 2 || ks > 0);
                mma_commit_if(leader, &S.s_done);
                if (Y && leader) mbar_arrive(&S.e_read);
                __syncwarp();
            }
            if (SAVE && live) {   // ---- e to the workspace
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int j0 = half * 32 + u * 16;
                    uint32_t acc[16];
                    tmem_ld16(tb + lb + kColKS + j0, acc);
                    tmem_wait_ld();
                    const int tok = (blk0 + n) * kDC + j0, in = p.N - tok;
                    float *dst = p.e + ((size_t)bh * p.N + tok) * DV + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < in) dst[(size_t)i * DV] = u2f(acc[i]);
                }
                tc_fence_before();
            }
            ok = ok && mbar_wait<1>(&S.s_done, n & 1, g, 9);
            ok = __all_sync(0xffffffffu, ok);
            // this block's K and Q have been read: [K; Q] K^T before T was ready, Q S before r
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
                    // SP is free: W, the last operand there, has been read
                    if (n + 1 < nblk && !Y) put_state(i);
                }
                if (Y && n + 1 < nblk) {
                    // at D = 128 the pieces of e lie in SP too: wait for P e
                    if (D > 64) ok = __all_sync(0xffffffffu, mbar_wait<1>(&S.pu_done, n & 1, g, 10));
                    tc_fence_after();
                    if (ok) {
#pragma unroll
                        for (int i = 0; i < SC; i += 16) put_state(i);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                sck += D * DV;
            }
            failed = any_failed(!ok);
        }
        if (SAVE && !failed && live && seg == segs - 1) write_state(sck, DV);
        if (in_place) {
            named_bar(kBarEnd, kChain + kOut);
            failed = failed || S.y_bad;
        }
        if (SEG) {
            if (!failed && live && values)
                write_state(p.S_local + (size_t)item * D * DV + (size_t)half * SC * DV + col_of, DV);
            else if (!failed && live)
                write_state(p.Phi + (size_t)item * D * D + (size_t)half * SC * D + col_of - DV, D);
        } else if (!failed && live && p.S_out && seg == segs - 1) {
            write_state(p.S_out + (size_t)bh * D * DV + (size_t)half * SC * DV + row, DV);
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
                const int tok = (blk0 + n) * kDC + 2 * lane + i;
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
            // T n - 2 has been used: its place is free, and so are gates[n & 3], whose last reader
            // is y n - 4 (block n - 2's K S waited for y n - 3)
            Gates &G = S.gates[n & 3];
            bool ok = n < 2 || mbar_wait<1>(&S.t_free[grp], ((n >> 1) - 1) & 1, g, 23);
            // the block before's [K; Q] K^T and gates have been read, and so those of every block before
            // it: a barrier for the even and one for the odd blocks, since the phase after block n - 2's
            // has the parity of the one before it, and the scores of block 0 may be read late
            if (n > 0) ok = ok && mbar_wait<1>(&S.kk_read[~n & 1], ((n - 1) >> 1) & 1, g, 24);
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
                    block_gates<false>(G, bv, gv, lane);
                    mbar_arrive(&S.g_ready[grp]);
                    if (n + 2 < nblk) fetch(n + 2);
                }
            }
            ok = ok && mbar_wait<1>(&S.g_ready[grp], (n >> 1) & 1, g, 25);
            ok = ok && mbar_wait<1>(&S.kk_full, n & 1, g, 21);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {   // A_ij = D_ij (k_i . k_j) b_j, j < i
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
                        decayed16<true, false>(G, t, j0, acc, x);
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = j0 + j < t ? x[j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<float4 *>(A + t * kAP + j0 + j) =
                            make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
                tc_fence_before();
                mbar_arrive(&S.kk_read[grp]);
            }
            if (any_out(!ok)) break;   // A complete
            int *bad = &S.t_bad[grp][(n >> 1) & 1];
            // the other turn's has been read before that barrier, and is used again behind several more
            if (CARE && t == 0) S.t_bad[grp][~(n >> 1) & 1] = kDC;
            invert_unit_lower<CARE>(A, t, bar, bad);
            // T's pieces over A: a thread's row is in registers before any is written
            float x[kDC];
#pragma unroll
            for (int j = 0; j < kDC; j += 4)
                *reinterpret_cast<float4 *>(x + j) = *reinterpret_cast<const float4 *>(A + t * kAP + j);
            if (CARE && t >= *bad) x[0] = nan_f();   // and with it e_t
            named_bar(bar, kInner);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t hi[4] = {}, mi[4] = {}, lo[4] = {};
                if (8 * q <= (t | 31))   // warp-uniform: zeros otherwise
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
        // ------------------------------------------------------------ P and y
        constexpr int kBarOut = kBarInner + 2;
        // P_ij = D_ij (q_i . k_j) b_j, j <= i, by the warps whose lanes hold the rows of Q.  The scores
        // of the next block are read before the wait for this block's P e, so that [K; Q] K^T can
        // move on; P itself follows y, its place being free then.
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
                mbar_arrive(&S.kk_read[n & 1]);
            }
            return ok;
        };
        auto make_p = [&](int n) {
            const Gates &G = S.gates[n & 3];
            const int i = row & 63;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t hi[8] = {}, mi[8] = {};
                if (16 * u <= (i | 31)) {   // warp-uniform: zeros otherwise
                    float x[16];
                    decayed16<false, false>(G, i, 16 * u, sc[u], x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = 16 * u + j <= i ? x[j] : 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) split2(x[2 * j], x[2 * j + 1], hi[j], mi[j]);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t o = sw128_off(i, 16 * u + 8 * q);
                    *reinterpret_cast<uint4 *>(sP + o) =
                        make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
                    *reinterpret_cast<uint4 *>(sP + 8192 + o) =
                        make_uint4(mi[4 * q], mi[4 * q + 1], mi[4 * q + 2], mi[4 * q + 3]);
                }
            }
            fence_proxy_async();
            mbar_arrive(&S.p_ready);
        };
        if (p.stall_ns)
            for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < p.stall_ns;) __nanosleep(1000);
        bool good = true;
        uint32_t z = 0;   // 0 y: anything else where y is not finite
        if (rows_of_q(0)) {
            good = read_scores(0);
            if (good) make_p(0);
        }
        for (int n = 0; n < nblk; ++n) {
            const Gates &G = S.gates[n & 3];
            // the gates, for the warps that have not waited for them with the scores (waiting again
            // could miss the phase: the next block's scores let the one after them come)
            bool ok = good && (rows_of_q(n) || mbar_wait<1>(&S.g_ready[n & 1], (n >> 1) & 1, g, 31));
            const bool next = n + 1 < nblk && rows_of_q(n + 1);
            if (next) ok = ok && read_scores(n + 1);
            if (CARE) ok = ok && mbar_wait<1>(&S.r_ready, n & 1, g, 35);
            ok = ok && mbar_wait<1>(&S.e_done, n & 1, g, 32);
            ok = ok && mbar_wait<1>(&S.qs_done, n & 1, g, 33);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && row < DV) {   // e as two pieces, in the place of the state's
                tc_fence_after();
                int first = CARE ? min(S.first[0][row], S.first[1][row]) : kDC;
#pragma unroll 1
                for (int j0 = 0; j0 < kDC; j0 += 16) {
                    uint32_t acc[16], hi[8], mi[8];
                    tmem_ld16(tb + lb + kColKS + j0, acc);
                    tmem_wait_ld();
                    if (CARE) {
                        float x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = u2f(acc[i]);
                        cut16(x, j0, first);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[i] = f2u(x[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) split2(u2f(acc[2 * i]), u2f(acc[2 * i + 1]), hi[i], mi[i]);
                    tmem_st8(tb + lb + kColE + j0 / 2, hi);
                    tmem_st8(tb + lb + kColE + j0 / 2 + 32, mi);
                }
                if (CARE) S.cut[row] = first;   // read by the same warp, behind a barrier
                tmem_wait_st();
                tc_fence_before();
            }
            if (tid == kChain + 2 * kInner) bulk_wait_read<0>();   // the last y has left its tile
            if (__any_sync(0xffffffffu, group_any<kBarOut, kOut>(!ok))) break;
            if (warp == 12) {   // P e over e, which the chain has read
                ok = mbar_wait<1>(&S.p_ready, n & 1, g, 8) && mbar_wait<1>(&S.e_read, n & 1, g, 34);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    const uint32_t leader = elect_leader();
                    tc_fence_after();
                    const uint32_t sp = smem_u32(sP);
#pragma unroll 1
                    for (int o = 0; o < 3; ++o)   // pieces (e, P): (0, 1) (1, 0) (0, 0)
                        mma_rows<kDC / 16, 0>(leader, tb + kColKS, tb + kColE + (o == 1) * 32, sp + (o == 0) * 8192,
                                              i64, o > 0);
                    mma_commit_if(leader, &S.pu_done);
                }
            }
            ok = ok && mbar_wait<1>(&S.pu_done, n & 1, g, 30);
            if (__any_sync(0xffffffffu, group_any<kBarOut, kOut>(!ok))) break;
            tc_fence_after();
            if (row < DV) {   // y = c . (Q S) + P e, 16 rows x 32 tokens at a time, through shared memory
                const int tq = (lane & 3) * 2;
#pragma unroll 1
                for (int it = 0; it < 4; ++it) {
                    const int j0 = (it & 1) * 32, hl = it >> 1;
                    const uint32_t ta = tb + lb + ((uint32_t)hl << 20) + j0;
                    uint32_t qs[16], pe[16], o[8];
                    tmem_ld_16x256b_x4(ta + kColQS, qs);
                    tmem_ld_16x256b_x4(ta + kColKS, pe);
                    float2 c[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) c[k] = *reinterpret_cast<const float2 *>(&G.c[j0 + 8 * k + tq]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {   // rows lane / 4 and + 8, tokens tq and + 1 of group k / 2
                        const float2 ck = c[k >> 1];
                        o[k] = pack_bf16x2(fmaf(ck.x, u2f(qs[2 * k]), u2f(pe[2 * k])),
                                           fmaf(ck.y, u2f(qs[2 * k + 1]), u2f(pe[2 * k + 1])));
                    }
                    if (CARE) {
                        const int *at = &S.cut[wq * 32 + hl * 16 + lane / 4], f[2] = {at[0], at[8]};
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int tok = j0 + 8 * (k >> 1) + tq;
                            o[k] |= (tok >= f[k & 1] ? 0x7FFFu : 0u) | (tok + 1 >= f[k & 1] ? 0x7FFF0000u : 0u);
                        }
                    } else {   // what leaks makes a row's P e NaN for every token: two of each row will do
                        z = fma_bf16x2(o[1], 0u, fma_bf16x2(o[0], 0u, z));
                    }
                    // matrices (group, row half): lane 8 m + i addresses token i of group m / 2, chunk m % 2
                    const int dv0 = wq * 32 + hl * 16 + ((lane >> 3) & 1) * 8, tok = j0 + (lane >> 4) * 8 + (lane & 7);
                    const uint32_t at = smem_u32(sY) + (dv0 >> 6) * 8192 + sw128_off(tok, dv0 & 63);
                    stmatrix_x4_trans(at, o[0], o[1], o[2], o[3]);
                    stmatrix_x4_trans(at + 16 * 128, o[4], o[5], o[6], o[7]);
                }
                tc_fence_before();
            }
            mbar_arrive(&S.o_read);
            fence_proxy_async();
            named_bar(kBarOut, kOut);
            if (tid == kChain + 2 * kInner) {
#pragma unroll
                for (int f = 0; f < DV / 64; ++f) tma_store_4d(&ymap, sY + f * 8192, f * 64, (blk0 + n) * kDC, h, b);
                bulk_commit();
            }
            if (next) make_p(n + 1);
        }
        if (!CARE) {
            if (z & 0x7FFF7FFFu) S.y_bad = 1;
            if (in_place) named_bar(kBarEnd, kChain + kOut);
        }
        if (tid == kChain + 2 * kInner) bulk_wait<0>();
        if (warp == 12 && elect_leader()) {
            mma_commit(&S.drain[3]);
            drain_wait(&S.drain[3], 0, g.limit_ns);
        }
        __syncwarp();
    }
}

// Only kForward launches warps 12-15.
template <int D, int DV, int MODE>
__global__ void __launch_bounds__(kChain + 2 * kInner + (MODE == kForward ? kOut : 0), 1)
delta_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ymap,
                const DeltaTc p) {
    constexpr bool Y = MODE == kForward;
    DeltaSmall &S = *reinterpret_cast<DeltaSmall *>(aligned_smem() + DeltaLay<D, DV>::oSmall);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (!Y) griddep_launch_dependents();   // a reverse pass that needs nothing of this launch
    if (tid == 0) {
        S.abort_flag = 0;
        S.y_bad = 0;
        init_barriers<Y>(S);
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        if (Y) prefetch_tmap(&qmap);
    }
    if (warp == 0) {
        tmem_alloc(&S.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    delta_run<D, DV, MODE, false>(qmap, kmap, vmap, ymap, p);
    tc_fence_before();
    __syncthreads();
    if (Y && S.y_bad && !S.abort_flag) {   // nothing is in flight: every copy and MMA has been waited for
        if (tid == 0) {
            for (uint64_t *b = S.kq_full; b <= &S.drain[3]; ++b) mbar_inval(b);
            init_barriers<Y>(S);
            for (int i = 0; i < 4; ++i) S.t_bad[i >> 1][i & 1] = kDC;
        }
        __syncthreads();
        tc_fence_after();
        delta_run<D, DV, MODE, true>(qmap, kmap, vmap, ymap, p);   // in line: a call's registers cost 7%
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(S.tmem_base, 512);
    }
}

// States at the segments' starts: P_0 = S_in (or 0), P_{s+1} = Phi_s P_s + S_local_s; with
// blockIdx.z = 1 their gradients at the segments' ends, G_{s-1} = Phi_s^T G_s + G_local_s from
// G_{nseg-1} = dS_out (or 0).  16 columns a CTA, walking the segments; a float32 product of [D x D]
// by [D x 16] a step.  Phi and the local ends are `items` to a head, P and G nseg.
constexpr int kPrefixCols = 16, kPrefixThr = 256;
struct PrefixArgs {
    const float *Phi, *local[2], *first[2];
    float *P[2];
    int nseg, items, DV;
};
template <int D>
__global__ void __launch_bounds__(kPrefixThr) delta_prefix_kernel(const PrefixArgs p) {
    const int nseg = p.nseg, DV = p.DV, rev = blockIdx.z;
    const float *__restrict__ Phi = p.Phi, *__restrict__ S_in = p.first[rev], *__restrict__ S_local = p.local[rev];
    float *__restrict__ P = p.P[rev];
    constexpr int NC = kPrefixCols * D / kPrefixThr;   // columns of a thread (a row of Phi each)
    __shared__ float Ps[D][kPrefixCols], F[D][33];
    const int bh = blockIdx.x, c0 = blockIdx.y * kPrefixCols;
    const int i = threadIdx.x % D, c = threadIdx.x / D * NC;
    const size_t st = (size_t)D * DV, at = (size_t)i * DV + c0 + c;
    float x[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) x[j] = S_in ? S_in[bh * st + at + j] : 0.f;
    for (int k = 0;; ++k) {
        const int s = rev ? nseg - 1 - k : k;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            Ps[i][c + j] = x[j];
            P[((size_t)bh * nseg + s) * st + at + j] = x[j];
        }
        if (k == nseg - 1) break;
        const size_t item = (size_t)bh * p.items + s;
#pragma unroll
        for (int j = 0; j < NC; ++j) x[j] = S_local[item * st + at + j];
        for (int a0 = 0; a0 < D; a0 += 32) {
            __syncthreads();
            for (int e = threadIdx.x; e < D * 32; e += kPrefixThr) {
                if (rev)
                    F[e % D][e / D] = Phi[item * D * D + (size_t)(a0 + e / D) * D + e % D];
                else
                    F[e / 32][e % 32] = Phi[item * D * D + (size_t)(e / 32) * D + a0 + e % 32];
            }
            __syncthreads();
#pragma unroll 8
            for (int a = 0; a < 32; ++a) {
                const float f = F[i][a];
#pragma unroll
                for (int j = 0; j < NC; ++j) x[j] = fmaf(f, Ps[a0 + a][c + j], x[j]);
            }
        }
        __syncthreads();
    }
}

// Segments of a head.  Splitting pays where the heads leave SMs idle: the segments but the last of
// each head then run once more, ahead, from an empty state (ceil((dv + d) / 128) CTAs each), and
// their ends are joined.  In units of a block's time (about 5 us): a wave of CTAs takes its
// segments' length; a second start, the join and their launches take about 8 + nseg / 2 (24 heads of
// 17 blocks: 94 us whole, 103 us in four; 32 heads of 2048 blocks: 8.4 ms whole, 3.5 ms in four).
void delta_segments(const DeltaArgs &a, int &nseg, int &seg_blocks) {
    const int nblk = delta_blocks(a.N), sms = num_sms(), parts = (a.dv + a.d + 127) / 128;
    const long long BH = (long long)a.B * a.H;
    auto waves = [&](long long ctas) { return (double)((ctas + sms - 1) / sms); };
    nseg = 1;
    seg_blocks = nblk;
    if (BH >= sms) return;
    double best = waves(BH) * nblk;
    for (int s = 2; s <= 64 && 2 * s <= nblk; ++s) {
        const int len = (nblk + s - 1) / s, n = (nblk + len - 1) / len;
        if (n != s) continue;
        const double cost = (waves(BH * (s - 1) * parts) + waves(BH * s)) * len + 8 + 0.5 * s;
        if (cost < best) {
            best = cost;
            nseg = s;
            seg_blocks = len;
        }
    }
}

// The same for the gradients: the segments' ends and maps, then the states' pass and the local
// reverse pass, then the reverse pass, against the reverse pass alone with the states' beside it.
// Block times of the passes: 1, 1, 1.3, 1.4; every pass fills the SMs or takes its chain's length.
void delta_bwd_segments(const DeltaArgs &a, int &nseg, int &seg_blocks) {
    const int nblk = delta_blocks(a.N), sms = num_sms(), parts = (a.dv + a.d + 127) / 128;
    const double BH = (double)a.B * a.H;
    auto most = [](double x, double y) { return x > y ? x : y; };
    nseg = 1;
    seg_blocks = nblk;
    double best = most(1.4 * nblk, 2.4 * BH * nblk / sms);
    for (int s = 2; s <= 64 && 2 * s <= nblk; ++s) {
        const int len = (nblk + s - 1) / s, n = (nblk + len - 1) / len;
        if (n != s) continue;
        const double cost = most(3.7 * len, (parts + 3.7) * BH * s * len / sms) + 16 + 0.5 * s;
        if (cost < best) {
            best = cost;
            nseg = s;
            seg_blocks = len;
        }
    }
}
// Floats of the split's arrays: by (head, segment) a map, and four states.
size_t delta_bwd_split_floats(const DeltaArgs &a, int nseg) {
    return nseg > 1 ? (size_t)a.B * a.H * nseg * ((size_t)a.d * a.d + 4 * (size_t)a.d * a.dv) : 0;
}

template <int D, int DV, int MODE> cudaError_t launch_tc(const DeltaArgs &a, DeltaTc p) {
    CUtensorMap qm, km, vm, ym{};
    if (!encode_tokens(&qm, a.q, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&km, a.k, a.layout, a.B, a.Hk, a.N, D) ||
        !encode_tokens(&vm, a.v, a.layout, a.B, a.H, a.N, DV) ||
        (MODE == kForward && !encode_tokens(&ym, a.y, a.layout, a.B, a.H, a.N, DV)))
        return cudaErrorInvalidValue;
    auto kern = delta_tc_kernel<D, DV, MODE>;
    constexpr int smem = DeltaLay<D, DV>::request;
    static_assert(smem <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int ctas = a.B * a.H * (MODE == kSegment ? p.seg_items * p.parts : p.nseg);
    kern<<<ctas, kChain + 2 * kInner + (MODE == kForward ? kOut : 0), smem, a.stream>>>(qm, km, vm, ym, p);
    return cudaGetLastError();
}

template <int D> cudaError_t launch_prefix(const DeltaArgs &a, const PrefixArgs &x, int ways) {
    delta_prefix_kernel<D><<<dim3(a.B * a.H, a.dv / kPrefixCols, ways), kPrefixThr, 0, a.stream>>>(x);
    return cudaGetLastError();
}

template <int D, int DV> DeltaTc tc_params(const DeltaArgs &a) {
    DeltaTc p{};
    p.beta = a.beta; p.lg = a.log_gate;
    p.H = a.H; p.group = a.H / a.Hk; p.N = a.N; p.layout = a.layout; p.nblk = delta_blocks(a.N);
    p.nseg = 1; p.seg_blocks = p.nblk; p.parts = (DV + D + 127) / 128;
    p.S_in = a.S_in; p.S_out = a.S_out;
    WsHeader *hdr = static_cast<WsHeader *>(a.ws);
    p.err = &hdr->error;
    p.err_where = &hdr->error_where;
    const long long lim = debug_fault().wait_limit_ns;
    p.limit_ns = lim > 0 ? (unsigned long long)lim : 1000000000ull;
    p.drop_item = debug_fault().drop_load_item;
    p.stall_ns = (unsigned long long)debug_fault().stall_ns;
    return p;
}

template <int D, int DV> cudaError_t launch_forward(const DeltaArgs &a) {
    DeltaTc p = tc_params<D, DV>(a);
    delta_segments(a, p.nseg, p.seg_blocks);
    if (p.nseg > 1) {
        p.seg_items = p.nseg - 1;
        const size_t items = (size_t)a.B * a.H * p.seg_items;
        p.S_local = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
        p.Phi = p.S_local + items * D * DV;
        float *P = p.Phi + items * D * D;
        cudaError_t e = launch_tc<D, DV, kSegment>(a, p);
        if (e == cudaSuccess)
            e = launch_prefix<D>(a, {p.Phi, {p.S_local, nullptr}, {a.S_in, nullptr}, {P, nullptr}, p.nseg,
                                     p.seg_items, DV}, 1);
        if (e != cudaSuccess) return e;
        p.S_in = P;
    }
    return launch_tc<D, DV, kForward>(a, p);
}

// e, the states and their gradients at every block (and dS_in).
template <int D, int DV> cudaError_t launch_passes(const DeltaArgs &a) {
    const DeltaBwdWs w = delta_bwd_ws(a);
    DeltaTc p = tc_params<D, DV>(a);
    p.S_ck = w.S;
    p.e = w.e;
    delta_bwd_segments(a, p.nseg, p.seg_blocks);
    cudaError_t e = cudaSuccess;
    const float *G_end = a.dS_out;
    if (p.nseg > 1) {
        p.seg_items = p.nseg;
        const size_t items = (size_t)a.B * a.H * p.nseg, st = (size_t)D * DV;
        p.Phi = w.split;
        p.S_local = p.Phi + items * D * D;
        float *P = p.S_local + items * st, *G_local = P + items * st, *GP = G_local + items * st;
        e = launch_tc<D, DV, kSegment>(a, p);
        if (e == cudaSuccess) e = launch_delta_reverse_tc(a, p.nseg, p.seg_blocks, nullptr, G_local);
        if (e == cudaSuccess)
            e = launch_prefix<D>(a, {p.Phi, {p.S_local, G_local}, {a.S_in, a.dS_out}, {P, GP}, p.nseg,
                                     p.seg_items, DV}, 2);
        if (e != cudaSuccess) return e;
        p.S_in = P;
        G_end = GP;
    }
    e = launch_tc<D, DV, kSave>(a, p);
    return e == cudaSuccess ? launch_delta_reverse_tc(a, p.nseg, p.seg_blocks, G_end, nullptr) : e;
}

}  // namespace

bool delta_tc_supported(const DeltaArgs &a) {
    return a.dt == LA_DTYPE_BF16 && (a.d == 64 || a.d == 128) && (a.dv == 64 || a.dv == 128);
}
// header | (split sequences) the segments' ends and maps, the states at their starts
size_t delta_tc_workspace(const DeltaArgs &a) {
    int nseg, len;
    delta_segments(a, nseg, len);
    size_t floats = 0;
    if (nseg > 1) {
        const size_t BH = (size_t)a.B * a.H, st = (size_t)a.d * a.dv;
        floats = BH * (nseg - 1) * (st + (size_t)a.d * a.d) + BH * nseg * st;
    }
    return sizeof(WsHeader) + 4 * floats;
}
size_t delta_tc_split_floats(const DeltaArgs &a) {
    int nseg, len;
    delta_bwd_segments(a, nseg, len);
    return delta_bwd_split_floats(a, nseg);
}
cudaError_t launch_delta_forward_tc(const DeltaArgs &a) {
    if (a.d == 64) return a.dv == 64 ? launch_forward<64, 64>(a) : launch_forward<64, 128>(a);
    return a.dv == 64 ? launch_forward<128, 64>(a) : launch_forward<128, 128>(a);
}
cudaError_t launch_delta_passes_tc(const DeltaArgs &a) {
    if (a.d == 64) return a.dv == 64 ? launch_passes<64, 64>(a) : launch_passes<64, 128>(a);
    return a.dv == 64 ? launch_passes<128, 64>(a) : launch_passes<128, 128>(a);
}

}  // namespace la
