// retention_tc.cu -- retention on the tensor cores (bf16 inputs, d and dv in {64, 128}): blocks of C = 128
// tokens, one CTA a head (or a segment of one).
//
//   scores  P  = Q K^T                        (128 x 128, K = d)
//   masked  P~ = gamma^|i-j| P                (two bf16 pieces, over P in TMEM)
//   y          = gamma^(i+1) (Q S) + P~ V     (dv = 128: one accumulator, scaled between the two products)
//   state   S' = gamma^C S + K^T W,           W_j = gamma^(C-1-j) v_j
// and the same with the exponents of retention.cuh from behind (REV).
//
// The products that make the state do not wait for what is made of it, and a block's scores are ready before its turn, so
// the tensor pipe goes from one product to the next while warps work on what they need:
//   warps 0-3    a row (token) a thread: P~ from P; the scaling of Q S; then y, through shared memory (where the
//                block's V was) and a tensor copy;
//   warps 4-11   W into TMEM as (K^T W)^T's left operand; the state, its columns (of dv) as TMEM lanes, d/2 of each in a
//                thread's registers; S^T in two bf16 pieces to shared memory for Q S;
//   warp 12      issues the MMAs: of a block the first half of K^T W (64 of d), Q S, the second half over the first's
//                accumulator (d = 64: there is one), P~ V, then the next block's Q K^T;
//   warp 13      issues the copies;
//   two more     (d = 64) P~ of half the columns of the rows that see most.
// W is the one operand without a second place in TMEM: its three pieces, the halves of K^T W, the state's update between
// them and Q S, which stands between the halves, are the chain that bounds a block of d = 128: at dv = 128 about 5,300 cycles, of
// which the products take 4,100 (K^T W 1,540, Q S and P~ V 1,020 each, Q K^T 510).  For d = 64 it is the one over P~, P~ V and y
// to the next scores.  B8 H16 N8192 d128: 220 us, 4.9 TB/s of the 6.7 that a copy reaches (inputs that stay the same from call
// to call 202); B1 H32 N131072 d64, in 19 segments: 615 us.
//
// With dv = 64 the upper 64 TMEM lanes hold W of the block's second 64 tokens (and zeros for the first, as the lower ones do for
// the second), so that every warp makes half as much of it; the lanes' sums stay two states that add up to S, and Q S takes
// both (a seventh faster at B8 H16 N8192 d64 than W in the lower lanes alone with one accumulator for y, when it came in).
//
// Precision: the state is float32 in registers, and what is added to it is exact but for the accumulator's float32: W is
// rounded to float32 once and enters as three bf16 pieces that add up to it (the top, middle and low 8 bits), against
// bf16 K, small pieces first.  What only y depends on, each score and each value of the state that it meets, enters as two
// pieces: 2^-15 of each at most is lost, no more than the bound of the float32 sums.  With one piece, 2^-8 of each, y was
// off by sqrt(2) times its own rounding where the terms are of random signs, but by a tenth of itself where they cancel
// (states with a common part of 64 times the rest that the queries do not see); the second pieces took the calls above
// from 190 to 220 and from 560 to 615 us.  y is rounded to bf16.
//
// What is not finite reaches no token before its own: masked scores are zeros, and a value of v that is not finite would
// make 0 * inf of them.  It also makes its column of K^T W something not finite, which (d = 128) the warps of the state see
// before P~ V is issued; for d = 64, where P~ V would have to wait for that (a tenth slower), the warps that
// make W look at every v.  In a block with such values these become zero in shared memory, and y NaN from the first's
// token on, for its column.
#include "delta_tc.cuh"
#include "retention.cuh"

namespace la {
namespace {

constexpr int kTC = 128;                      // tokens of a block
constexpr int kState = 256;                   // threads of the state's warps

// TMEM columns: P (P~ over it), y, half of K^T W, three pieces of W.  For the segments' sums alone: K^T W, and W
// twice, so that the next one is made while the products of this one run.
constexpr uint32_t kColP = 0, kColY = 128, kColKV = 256, kColW3 = 320;
constexpr uint32_t kColSumW = 128;   // K^T W from column 0, W from 128 and 320 on

struct RetainTc {
    const float *gamma, *S_in;
    float *S_out;            // kWhole: the final state, from the last segment taken; kSums: by (head, segment)
    int H, N, nblk, nseg, seg_blocks;
    int seg0, segs;          // segments of a head that are launched: seg0 ..
    bool trans;              // S_in and S_out are [dv][d]
    unsigned int *err, *err_where;
    unsigned long long limit_ns;
    int drop_item;
};

constexpr int kMostStages = 4;
struct RetainSmall {
    uint64_t q_full[kMostStages], k_full[kMostStages], v_full[kMostStages], pv_done[kMostStages], y_written[kMostStages], kv_done[2], kv_read, qk_done, p_ready, s_ready,
        qs_done, y_scaled, y_free, w_ready[2], drain;   // w_ready[1], and kv_read by all: kSums
    float pg[2 * kTC + 4];        // pg[kTC - n] = gamma^n, zeros behind
    alignas(16) float near[16];   // gamma^(15 - j) (REV: gamma^j)
    int v_bad[4];                 // block index + 1 of a block with a value that is not finite; y of a block may still be to come
                                  // when W of the next but one is made
    uint8_t first[2][kTC];        // then, by column: how many tokens come before its first one (REV: up to its last one)
    uint32_t tmem_base;
    volatile int abort_flag;
};

// What a launch computes: y from each segment's state; each segment's own sum.
enum RetainMode { kWhole, kSums };

template <int D, int DV, int MODE> struct RetainLay {
    static constexpr bool OUT = MODE == kWhole;
    // d = 64, where the chain from a block's scores over P~, P~ V and y to the next block's is the longest: two warps more for P~
    // (B8 H16 N8192 d64 118 us, without them 129; dv = 128 169 and 185; at d = 128 they would cost 2%)
    static constexpr bool HELP = OUT && D == 64;
    static constexpr int threads = HELP ? 512 : 448;
    static constexpr int kQ = (D / 64) * 16384, kV = (DV / 64) * 16384;
    // S: one piece of one state (of two if dv = 64); two pieces.  kSums: float32
    static constexpr int kHalfS = DV * D * 2, kS = OUT ? (128 / DV) * 2 * kHalfS : DV * D * 4;
    // blocks in flight: as many as fit, four at most; of Q one where that makes room for a second block of K and V
    // (d = dv = 128)
    static constexpr int kBlock = (OUT ? 2 : 1) * kQ + kV, kFree = 232448 - kS - 1024 - (int)sizeof(RetainSmall);
    static constexpr int kFit = kFree / kBlock < kMostStages ? kFree / kBlock : kMostStages;
    static constexpr int kNst = kFit >= 2 ? kFit : 2, kNsq = OUT ? (kFit >= 2 ? kFit : 1) : 0;
    static constexpr int oQ = 0, oK = oQ + kNsq * kQ, oV = oK + kNst * kQ, oS = oV + kNst * kV, oSmall = oS + kS;
    static constexpr int request = oSmall + (int)sizeof(RetainSmall) + 1024;
};

// Three pieces of a pair by truncation, as split3, at two thirds of its time: the logical operations that take a piece
// off a value run at half the rate of a multiply-add.
__device__ __forceinline__ void pieces3(float x0, float x1, uint32_t &h, uint32_t &m, uint32_t &l) {
    h = __byte_perm(f2u(x0), f2u(x1), 0x7632);
    x0 = minus_bf16_lo(x0, h);
    x1 = minus_bf16_hi(x1, h);
    m = __byte_perm(f2u(x0), f2u(x1), 0x7632);
    l = __byte_perm(f2u(minus_bf16_lo(x0, m)), f2u(minus_bf16_hi(x1, m)), 0x7632);
}
// Two pieces: the first cut (what is finite stays so), what is left of it rounded to nearest, 2^-15 of the value at most off.
__device__ __forceinline__ void pieces2(float x0, float x1, uint32_t &h, uint32_t &l) {
    h = __byte_perm(f2u(x0), f2u(x1), 0x7632);
    l = pack_bf16x2(minus_bf16_lo(x0, h), minus_bf16_hi(x1, h));
}

__device__ __forceinline__ uint8_t *retain_smem() {
    extern __shared__ uint8_t smem_raw[];
    return smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
}

template <int D, int DV, bool REV, int MODE>
__global__ void __launch_bounds__(RetainLay<D, DV, MODE>::threads, 1)
retain_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ymap, const RetainTc p) {
    using Lay = RetainLay<D, DV, MODE>;
    constexpr bool OUT = MODE == kWhole;
    constexpr int NST = Lay::kNst, NSQ = Lay::kNsq > 0 ? Lay::kNsq : 1;
    constexpr int NH = D / 64;   // halves of K^T W
    constexpr bool TWIN = DV == 64;   // two states, of the tokens' halves; Q S and P~ V in accumulators of their own
    constexpr bool SPLIT = TWIN && NH == 2;   // Q S in two parts
    // the warps above 11; HELP: the two quarters of the rows that see most columns have a second one (TMEM lanes go by warp % 4)
    constexpr bool HELP = Lay::HELP;
    constexpr int kMma = HELP && REV ? 14 : 12, kCopy = kMma + 1;
    uint8_t *sm = retain_smem();
    RetainSmall &S = *reinterpret_cast<RetainSmall *>(sm + Lay::oSmall);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int bh = blockIdx.x / p.segs, seg = p.seg0 + blockIdx.x % p.segs, b = bh / p.H, h = bh - b * p.H;
    const int first_blk = seg * p.seg_blocks, nch = min(p.seg_blocks, p.nblk - first_blk);
    const float gamma = p.gamma[h];
    if (!OUT) griddep_launch_dependents();   // the scan, which waits for this grid's end
    // the n-th block taken, and its tokens
    auto token_of = [&](int n) { return (first_blk + (REV ? nch - 1 - n : n)) * kTC; };
    auto length_of = [&](int n) { return min(kTC, p.N - token_of(n)); };

    if (tid == 0) {
        S.abort_flag = 0;
        for (int i = 0; i < 4; ++i) S.v_bad[i] = 0;
        for (int i = 0; i < NST; ++i) {
            mbar_init(&S.q_full[i], 1);
            mbar_init(&S.k_full[i], 1);
            mbar_init(&S.v_full[i], 1);
            mbar_init(&S.pv_done[i], 1);
            mbar_init(&S.y_written[i], 128);
        }
        mbar_init(&S.kv_done[0], 1);
        mbar_init(&S.kv_done[1], 1);
        mbar_init(&S.kv_read, OUT ? kState / 2 : kState);
        mbar_init(&S.qk_done, 1);
        mbar_init(&S.p_ready, HELP ? 192 : 128);
        mbar_init(&S.s_ready, kState);
        mbar_init(&S.qs_done, 1);
        mbar_init(&S.y_scaled, 128);
        mbar_init(&S.y_free, 128);
        mbar_init(&S.w_ready[0], kState);
        mbar_init(&S.w_ready[1], kState);
        mbar_init(&S.drain, 1);
        fence_mbar_init();
        prefetch_tmap(&kmap);
        prefetch_tmap(&vmap);
        if (OUT) prefetch_tmap(&qmap);
    }
    if (tid >= 64 && tid <= 64 + 2 * kTC) S.pg[tid - 64] = tid <= 64 + kTC ? gamma_power(gamma, 64 + kTC - tid) : 0.f;
    if (tid >= 32 && tid < 48) S.near[tid - 32] = gamma_power(gamma, REV ? tid - 32 : 47 - tid);
    if (warp == kMma) {
        tmem_alloc(&S.tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, S.tmem_base, 0);
    const Guard g{&S.abort_flag, p.err, p.err_where, p.limit_ns};
    const int wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lb = (uint32_t)(wq * 32) << 16;
    const float *pw = S.pg + kTC;   // pw[-n] = gamma^n
    uint8_t *sQ = sm + Lay::oQ, *sK = sm + Lay::oK, *sV = sm + Lay::oV, *sS = sm + Lay::oS;
    auto y_tile = [&](int n) { return sV + (n % NST) * Lay::kV; };   // W and P~ V have read V
    auto turn = [](int n) { return (uint32_t)(n / NST) & 1u; };      // parity of block n's use of its place
    auto turn_q = [](int n) { return (uint32_t)(n / NSQ) & 1u; };

    // P~ of 32 columns off the diagonal, over P itself: of each 32 columns 16 for the first pieces, 16 for the second
    auto fill = [&](int jb, const float (&nr)[16]) {
        const uint32_t pcol = tb + lb + kColP + jb;
        uint32_t x[32], o[16], o2[16];
        tmem_ld16(pcol, *reinterpret_cast<uint32_t(*)[16]>(x));
        tmem_ld16(pcol + 16, *reinterpret_cast<uint32_t(*)[16]>(x + 16));
        const float f0 = pw[REV ? row - jb : jb + 15 - row], f1 = pw[REV ? row - jb - 16 : jb + 31 - row];
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float f = j < 8 ? f0 : f1;
            float a, bb;
            f2unpack(f2mul(f2mul(f2pack(f, f), f2pack(nr[2 * j & 15], nr[(2 * j + 1) & 15])), f2pack(u2f(x[2 * j]), u2f(x[2 * j + 1]))),
                     a, bb);
            pieces2(a, bb, o[j], o2[j]);
        }
        tmem_st16(pcol, o);
        tmem_st16(pcol + 16, o2);
    };

    if (warp == kCopy) {
        // ------------------------------------------------------------ copies
        if (elect_leader()) {
            auto load = [&](uint8_t *dst, const CUtensorMap &m, uint64_t *bar, int slabs, int n, bool drop) {
                mbar_arrive_expect_tx(bar, slabs * 16384);
                if (drop) return;   // test hook: announced, never issued
                for (int f = 0; f < slabs; ++f) tma_load_4d(dst + f * 16384, &m, bar, f * 64, token_of(n), h, b);
            };
            auto store = [&](int n) {   // y of a block, when it is written
                if (!mbar_wait<2>(&S.y_written[n % NST], turn(n), g, 1)) return false;
#pragma unroll
                for (int f = 0; f < DV / 64; ++f) tma_store_4d(&ymap, y_tile(n) + f * 16384, f * 64, token_of(n), h, b);
                bulk_commit();
                return true;
            };
            int nk = 0, nv = 0, nq = 0;   // copies issued
            auto load_q = [&](int n) {
                load(sQ + n % NSQ * Lay::kQ, qmap, &S.q_full[n % NSQ], D / 64, n, false);
                ++nq;
            };
            for (int n = 0; n < nch; ++n) {
                const int s = n % NST;
                // the block before it there has been used: its last product is P~ V
                if (n >= NST && !mbar_wait<2>(&S.pv_done[s], turn(n) ^ 1u, g, 2)) break;
                load(sK + s * Lay::kQ, kmap, &S.k_full[s], D / 64, n, n == 0 && (int)blockIdx.x == p.drop_item);
                ++nk;
                if (OUT && NSQ == NST) load_q(n);
                if (OUT && n >= NST) {   // y where V comes
                    if (!store(n - NST)) break;
                    bulk_wait_read<0>();
                }
                load(sV + s * Lay::kV, vmap, &S.v_full[s], DV / 64, n, false);
                ++nv;
                // the next one into L2, while its places are still taken (d = 128: a twelfth faster, when it came in; with d = 64
                // more blocks are in flight, and it cost a twentieth)
                if (OUT && D > 64 && n >= 1 && n + 1 < nch) {
                    for (int f = 0; f < D / 64; ++f) {
                        tma_prefetch_4d(&kmap, f * 64, token_of(n + 1), h, b);
                        tma_prefetch_4d(&qmap, f * 64, token_of(n + 1), h, b);
                    }
                    for (int f = 0; f < DV / 64; ++f) tma_prefetch_4d(&vmap, f * 64, token_of(n + 1), h, b);
                }
                if (OUT && NSQ != NST) {   // Q's one place: the block before's last product with it is Q S
                    if (n >= 1 && !mbar_wait<2>(&S.qs_done, (n - 1) & 1, g, 3)) break;
                    load_q(n);
                }
            }
            if (OUT) {
                if (nv == nch)
                    for (int m = max(0, nch - NST); m < nch; ++m)
                        if (!store(m)) break;
                bulk_wait<0>();
            }
            // what is in flight lands (after a wait that ran out; otherwise it has been used)
            for (int m = max(0, nk - NST); m < nk; ++m)
                if (!(m == 0 && (int)blockIdx.x == p.drop_item)) drain_wait(&S.k_full[m % NST], turn(m), g.limit_ns);
            for (int m = max(0, nv - NST); m < nv; ++m) drain_wait(&S.v_full[m % NST], turn(m), g.limit_ns);
            for (int m = max(0, nq - NSQ); m < nq; ++m) drain_wait(&S.q_full[m % NSQ], turn_q(m), g.limit_ns);
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t iP = idesc_bf16(128, kTC, 0, 0), iQS = idesc_bf16(128, DV, 0, 0),
                           iKV = idesc_bf16(128, 64, 0, 1), iPV = idesc_bf16(128, DV, 0, 1);
        bool ok = true;
        auto all = [&](bool x) { ok = ok && __all_sync(0xffffffffu, x); };
        auto kv_half = [&](int n, int half) {   // (K^T W)^T, 64 columns of d
            const uint32_t to = OUT ? tb + kColKV : tb + half * 64, w = tb + (OUT ? kColW3 : kColSumW + (n & 1) * 192);
            const uint32_t leader = elect_leader();
            tc_fence_after();
            const uint64_t kd = smem_desc(smem_u32(sK) + (n % NST) * Lay::kQ + half * 16384, 16384, 1024, kSwizzle128B);
#pragma unroll   // a twentieth faster than a loop over the pieces at B8 H16 N8192 d64
            for (int pc = 2; pc >= 0; --pc)
#pragma unroll
                for (int ks = 0; ks < kTC / 16; ++ks)
                    mma_ts_if(leader, to, w + pc * 64 + ks * 8, kd + ks * 128, iKV, pc < 2 || ks > 0);
            if (OUT || half == NH - 1) mma_commit_if(leader, &S.kv_done[OUT ? half : 0]);
        };
        auto scores = [&](int n) {
            const int s = n % NST;
            all(mbar_wait<2>(&S.k_full[s], turn(n), g, 3) && mbar_wait<2>(&S.q_full[n % NSQ], turn_q(n), g, 4));
            if (!ok) return;
            const uint32_t leader = elect_leader();
            tc_fence_after();
            const uint64_t qd = desc_k(smem_u32(sQ) + n % NSQ * Lay::kQ), kd = desc_k(smem_u32(sK) + s * Lay::kQ);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                mma_ss_if(leader, tb + kColP, qd + o, kd + o, iP, ks > 0);
            }
            mma_commit_if(leader, &S.qk_done);
        };
        // Q S, small pieces of S first.  d = 128, dv = 64: their product stands between the halves of K^T W, the others' behind
        // them, where nothing but P~ V waits for it (B8 H16 N8192 175 us, all of it between the halves 185; with dv = 128 it is scaled
        // before P~ V)
        constexpr int SETS = TWIN ? 4 : 2;
        auto queries = [&](int n, int from, int to) {
            const uint32_t leader = elect_leader();
            tc_fence_after();
            const uint64_t qd = desc_k(smem_u32(sQ) + n % NSQ * Lay::kQ), sd = desc_k(smem_u32(sS));
#pragma unroll
            for (int t = from; t >= to; --t)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss_if(leader, tb + kColY, qd + (uint32_t)(((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                              sd + (uint32_t)((t * Lay::kHalfS + (ks >> 2) * DV * 128 + (ks & 3) * 32) >> 4), iQS,
                              t < SETS - 1 || ks > 0);
            if (to == 0) mma_commit_if(leader, &S.qs_done);
        };
        // A block with a value of v that is not finite: zero in shared memory, and where the columns' first ones are.
        auto mend_v = [&](int n) {
            for (int c = lane; c < DV; c += 32) {
                uint8_t *col = sV + (n % NST) * Lay::kV + (c >> 6) * 16384 + (c & 7) * 2;
                int f = REV ? 0 : kTC;
                for (int t = 0; t < kTC; ++t) {
                    uint16_t *v = reinterpret_cast<uint16_t *>(col + t * 128 + ((((c & 63) >> 3) ^ (t & 7)) << 4));
                    if ((*v & 0x7F80) == 0x7F80) {
                        *v = 0;
                        f = REV ? t + 1 : min(f, t);
                    }
                }
                S.first[n & 1][c] = (uint8_t)f;
            }
            fence_proxy_async();
            __syncwarp();
        };
        if (OUT) scores(0);
        for (int n = 0; n < nch && ok; ++n) {
            const int s = n % NST;
            if (!OUT) {
                all(mbar_wait<2>(&S.k_full[s], turn(n), g, 3) && mbar_wait<2>(&S.w_ready[n & 1], (n >> 1) & 1, g, 5) &&
                    (n == 0 || mbar_wait<2>(&S.kv_read, (n - 1) & 1, g, 8)));
                if (!ok) break;
                for (int half = 0; half < NH; ++half) kv_half(n, half);
                const uint32_t leader = elect_leader();
                mma_commit_if(leader, &S.pv_done[s]);
                continue;
            }
            all(mbar_wait<2>(&S.w_ready[0], n & 1, g, 5));
            if (!ok) break;
            kv_half(n, 0);
            all(mbar_wait<2>(&S.s_ready, n & 1, g, 6) && (n == 0 || mbar_wait<2>(&S.y_free, (n - 1) & 1, g, 7)));
            if (!ok) break;
            queries(n, SETS - 1, SPLIT ? SETS / 2 : 0);
            if (NH == 2) {
                all(mbar_wait<2>(&S.kv_read, n & 1, g, 8));
                if (!ok) break;
                kv_half(n, 1);
                if (SPLIT) queries(n, SETS / 2 - 1, 0);
            }
            if (*(volatile int *)&S.v_bad[n & 3] == n + 1) mend_v(n);
            all(mbar_wait<2>(&S.p_ready, n & 1, g, 9) && (TWIN || mbar_wait<2>(&S.y_scaled, n & 1, g, 10)));
            if (!ok) break;
            {
                const uint32_t leader = elect_leader();
                tc_fence_after();
                const uint64_t vd = smem_desc(smem_u32(sV) + s * Lay::kV, 16384, 1024, kSwizzle128B);
#pragma unroll
                for (int pc = 1; pc >= 0; --pc)   // small pieces first: 16 columns behind the others' 16
#pragma unroll
                    for (int ks = 0; ks < kTC / 16; ++ks)
                        mma_ts_if(leader, tb + kColY + (TWIN ? 64 : 0), tb + kColP + (ks >> 1) * 32 + pc * 16 + (ks & 1) * 8, vd + ks * 128,
                                  iPV, !TWIN || pc < 1 || ks > 0);
                mma_commit_if(leader, &S.pv_done[s]);
            }
            if (n + 1 < nch) scores(n + 1);
        }
        if (elect_leader()) {
            mma_commit(&S.drain);
            drain_wait(&S.drain, 0, g.limit_ns);
        }
        __syncwarp();
    } else if (HELP && warp >= 12) {
        // ------------------------------------------------------------ P~ of the half of the columns away from the diagonal
        float nr[16];
        load16(S.near, nr);
        for (int n = 0; n < nch; ++n) {
            if (!__all_sync(0xffffffffu, mbar_wait<2>(&S.qk_done, n & 1, g, 33))) break;
            tc_fence_after();
#pragma unroll 1
            for (int jb = REV ? 64 : 0; jb < (REV ? kTC : 64); jb += 32) fill(jb, nr);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&S.p_ready);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ W and the state
        constexpr int SC = D / 2;   // state values of a thread: column `row` of dv, half * SC .. of d
        const int half = (warp - 4) >> 2;
        const int part = TWIN ? wq >> 1 : 0, col = TWIN ? row & 63 : row;   // part: warp-uniform
        float st[SC];
        if (OUT) griddep_wait();   // segments' states: this launch may have started before the scan's end
        if (part == 0 && p.S_in) {
            const float *src = p.S_in + (size_t)(p.nseg > 1 ? bh * p.nseg + seg : bh) * D * DV;
            if (p.trans) {
#pragma unroll
                for (int i = 0; i < SC; i += 4)
                    *reinterpret_cast<float4 *>(st + i) = *reinterpret_cast<const float4 *>(src + (size_t)col * D + half * SC + i);
            } else {
#pragma unroll
                for (int i = 0; i < SC; ++i) st[i] = src[(size_t)(half * SC + i) * DV + col];
            }
        } else {
#pragma unroll
            for (int i = 0; i < SC; ++i) st[i] = 0.f;
        }
        auto put_state = [&] {   // S^T in two bf16 pieces, rows of d
#pragma unroll
            for (int i = 0; i < SC; i += 8) {
                const int c = half * SC + i;
                uint8_t *at = sS + part * Lay::kHalfS + (c >> 6) * (DV * 128) + sw128_off(col, c & 63);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) pieces2(st[i + 2 * j], st[i + 2 * j + 1], hi[j], lo[j]);
                *reinterpret_cast<uint4 *>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(at + (TWIN ? 2 : 1) * Lay::kHalfS) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async();
            mbar_arrive(&S.s_ready);
        };
        if (TWIN) {   // W of the other half's tokens: zeros
            const uint32_t none[16] = {};
#pragma unroll
            for (int i = 0; i < (OUT ? 3 : 6); ++i)
                tmem_st16(tb + lb + (OUT ? kColW3 : kColSumW) + i * 64 + (1 - part) * 32 + half * 16, none);
        }
        bool ok = true;
        auto wait_v = [&](int n) { return mbar_wait<2>(&S.v_full[n % NST], turn(n), g, 20); };
        auto make_w = [&](int n, uint32_t at_w) {
            const int L = length_of(n);
            tc_fence_after();
            const uint8_t *tv = sV + (n % NST) * Lay::kV;
            uint32_t z0 = 0, z1 = 0;   // 0 v: anything else where v is not finite
            const int tq = (lane & 3) * 2;
#pragma unroll 1
            for (int u = 0; u < (TWIN ? 1 : 2); ++u) {   // 32 tokens
                const int t0 = TWIN ? part * 64 + half * 32 : half * 64 + u * 32;
                // weights of tokens t0 + 8 g + tq and + 1 (behind the last token zeros, or of zeros)
                const float *wp = pw + (REV ? -(t0 + tq + 1) : t0 + tq + 1 - L);
                float w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] = wp[(REV ? -1 : 1) * ((k >> 1) * 8 + (k & 1))];
#pragma unroll
                for (int hl = 0; hl < 2; ++hl) {   // 16 columns of dv
                    uint32_t x[8], hi[8], mi[8], lo[8];
                    const int c = (TWIN ? wq & 1 : wq) * 4 + hl * 2 + ((lane >> 3) & 1);   // 16-byte chunk of a token's row
                    const int t = t0 + (lane >> 4) * 8 + (lane & 7);
                    const uint32_t at = smem_u32(tv) + (c >> 3) * 16384 + t * 128 + (((c & 7) ^ (t & 7)) << 4);
                    ldmatrix_x4_trans(at, x[0], x[1], x[2], x[3]);
                    ldmatrix_x4_trans(at + 16 * 128, x[4], x[5], x[6], x[7]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {   // tokens 8 (k / 2) + tq and + 1, column lane / 4 + 8 (k % 2)
                        if (OUT && NH == 1) (k & 1 ? z1 : z0) = fma_bf16x2(x[k], 0u, k & 1 ? z1 : z0);
                        pieces3(w[k & 6] * bf16_lo_f(x[k]), w[(k & 6) + 1] * bf16_hi_f(x[k]), hi[k], mi[k], lo[k]);
                    }
                    const uint32_t to = tb + lb + ((uint32_t)hl << 20) + at_w + t0 / 2;
                    tmem_st_16x128b_x4(to, hi);
                    tmem_st_16x128b_x4(to + 64, mi);
                    tmem_st_16x128b_x4(to + 128, lo);
                }
            }
            if (OUT && NH == 1 && ((z0 | z1) & 0x7FFF7FFFu)) S.v_bad[n & 3] = n + 1;
            tmem_wait_st();
            tc_fence_before();
        };
        auto update = [&](int n, uint32_t at_kv) {   // S' = gamma^L S + K^T W
            tc_fence_after();
            const float gl = pw[-length_of(n)];
            const uint64_t g2 = f2pack(gl, gl);
#pragma unroll
            for (int i = 0; i < SC; i += 32) {
                uint32_t a0[16], a1[16];
                const uint32_t from = tb + lb + at_kv + i;
                tmem_ld16(from, a0);
                tmem_ld16(from + 16, a1);
                tmem_wait_ld();
                // a value of v that is not finite leaves nothing finite here (a value of k may, too)
                if (OUT && NH == 2 && i == 0 && half == 0 && !finite(u2f(a0[0]))) S.v_bad[n & 3] = n + 1;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    f2unpack(f2fma(g2, f2pack(st[i + j], st[i + j + 1]), f2pack(u2f(a0[j]), u2f(a0[j + 1]))), st[i + j],
                             st[i + j + 1]);
                    f2unpack(f2fma(g2, f2pack(st[i + 16 + j], st[i + 17 + j]), f2pack(u2f(a1[j]), u2f(a1[j + 1]))),
                             st[i + 16 + j], st[i + 17 + j]);
                }
            }
            tc_fence_before();
        };
        if (!OUT) {   // the next W before this block's sum is waited for
            for (int n = -1; n < nch; ++n) {
                if (n + 1 < nch) {   // its place: the sum before the last has been waited for
                    if (!(ok = __all_sync(0xffffffffu, wait_v(n + 1)))) break;
                    make_w(n + 1, kColSumW + ((n + 1) & 1) * 192);
                    mbar_arrive(&S.w_ready[(n + 1) & 1]);
                }
                if (n < 0) continue;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait<2>(&S.kv_done[0], n & 1, g, 23)))) break;
                update(n, half * SC);
                mbar_arrive(&S.kv_read);
            }
        }
        for (int n = 0; OUT && n < nch; ++n) {
            ok = wait_v(n);
            // W's place is free (where this has not been waited for below)
            if (n >= 1 && NH == 2 && half == 0) ok = ok && mbar_wait<2>(&S.kv_done[1], (n - 1) & 1, g, 21);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            make_w(n, kColW3);
            mbar_arrive(&S.w_ready[0]);
            if ((NH == 1 || SPLIT) && n >= 1) {   // Q S of the block before has read its operand (else K^T W's end says so)
                ok = __all_sync(0xffffffffu, mbar_wait<2>(&S.qs_done, (n - 1) & 1, g, 22));
                if (!ok) break;
            }
            put_state();
            ok = __all_sync(0xffffffffu, mbar_wait<2>(&S.kv_done[NH == 2 ? half : 0], n & 1, g, 23));
            if (!ok) break;
            update(n, kColKV + (NH == 2 ? 0 : half * SC));
            if (NH == 2 && half == 0) mbar_arrive(&S.kv_read);
        }
        const bool last = seg == (REV ? 0 : p.nseg - 1);
        float *dst = OUT ? (p.S_out && last ? p.S_out + (size_t)bh * D * DV : nullptr)
                         : p.S_out + ((size_t)bh * p.nseg + seg) * D * DV;
        if (TWIN && dst) {   // the second half's state through where S was, which the last Q S has read
            if (OUT) ok = __all_sync(0xffffffffu, ok && mbar_wait<2>(&S.qs_done, (nch - 1) & 1, g, 24));
            float *other = reinterpret_cast<float *>(sS) + half * SC * DV + col;
            if (ok && part == 1)
#pragma unroll
                for (int i = 0; i < SC; ++i) other[i * DV] = st[i];
            named_bar(1, kState);
            if (ok && part == 0)
#pragma unroll
                for (int i = 0; i < SC; ++i) st[i] += other[i * DV];
        }
        if (ok && part == 0 && dst) {
            if (OUT && p.trans) {
#pragma unroll
                for (int i = 0; i < SC; i += 4)
                    *reinterpret_cast<float4 *>(dst + (size_t)col * D + half * SC + i) = make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < SC; ++i) dst[(size_t)(half * SC + i) * DV + col] = st[i];
            }
        }
    } else if (OUT) {
        // ------------------------------------------------------------ P~ and y
        const uint32_t pcol = tb + lb + kColP, col = tb + lb + kColY;
        float nr[16], dg[32];   // gamma^(to a block's nearest column); on the diagonal gamma^|i - j|, and what is kept there
        uint32_t keep[16];
        load16(S.near, nr);
        // columns that are its own: half of them where another warp takes the other
        const bool helped = HELP && (REV ? wq < 2 : wq >= 2);
        const int first = !REV && helped ? 64 : 0, count = helped ? 64 : kTC;
#pragma unroll
        for (int j = 0; j < 32; ++j) dg[j] = (REV ? j >= lane : j <= lane) ? pw[-abs(lane - j)] : 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            keep[j] = ((REV ? 2 * j >= lane : 2 * j <= lane) ? 0xFFFFu : 0u) | ((REV ? 2 * j + 1 >= lane : 2 * j + 1 <= lane) ? 0xFFFF0000u : 0u);
        for (int n = 0; n < nch; ++n) {
            if (!__all_sync(0xffffffffu, mbar_wait<2>(&S.qk_done, n & 1, g, 30))) break;
            {
                tc_fence_after();
#pragma unroll 1
                for (int jb = first; jb < first + count; jb += 32) {
                    const int side = jb - 32 * wq;       // warp-uniform
                    if (REV ? side > 0 : side < 0) {
                        fill(jb, nr);
                        continue;
                    }
                    uint32_t o[16], o2[16];
                    if (side != 0) {   // beyond the diagonal
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = o2[j] = 0u;
                    } else {           // bits that are not kept: a score that is not finite leaves nothing of itself
                        uint32_t x[32];
                        tmem_ld16(pcol + jb, *reinterpret_cast<uint32_t(*)[16]>(x));
                        tmem_ld16(pcol + jb + 16, *reinterpret_cast<uint32_t(*)[16]>(x + 16));
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            pieces2(dg[2 * j] * u2f(x[2 * j]), dg[2 * j + 1] * u2f(x[2 * j + 1]), o[j], o2[j]);
                            o[j] &= keep[j];
                            o2[j] &= keep[j];
                        }
                    }
                    tmem_st16(pcol + jb, o);
                    tmem_st16(pcol + jb + 16, o2);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&S.p_ready);
            }
            const float f = pw[-max(0, inter_exp(REV, row, length_of(n)))];   // behind the last token: of zeros
            if (!TWIN) {
                if (!__all_sync(0xffffffffu, mbar_wait<2>(&S.qs_done, n & 1, g, 31))) break;
                tc_fence_after();
                const uint64_t f2 = f2pack(f, f);
#pragma unroll 1
                for (int c = 0; c < DV; c += 64) {
                    uint32_t a[4][16];
#pragma unroll
                    for (int u = 0; u < 4; ++u) tmem_ld16(col + c + 16 * u, a[u]);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            float x, y;
                            f2unpack(f2mul(f2, f2pack(u2f(a[u][j]), u2f(a[u][j + 1]))), x, y);
                            a[u][j] = f2u(x);
                            a[u][j + 1] = f2u(y);
                        }
                        tmem_st16(col + c + 16 * u, a[u]);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&S.y_scaled);
            }
            if (!__all_sync(0xffffffffu, mbar_wait<2>(&S.pv_done[n % NST], turn(n), g, 32))) break;
            {
                uint8_t *sY = y_tile(n);
                tc_fence_after();
                const bool bad = *(volatile int *)&S.v_bad[n & 3] == n + 1;
#pragma unroll 1
                for (int c = 0; c < DV; c += 32) {
                    uint32_t a[2][16], e[2][16];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        tmem_ld16(col + c + 16 * u, a[u]);
                        if (TWIN) tmem_ld16(col + 64 + c + 16 * u, e[u]);
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t o[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = TWIN ? pack_bf16x2(fmaf(f, u2f(a[u][2 * j]), u2f(e[u][2 * j])), fmaf(f, u2f(a[u][2 * j + 1]), u2f(e[u][2 * j + 1])))
                                        : pack_bf16x2(u2f(a[u][2 * j]), u2f(a[u][2 * j + 1]));
                        if (bad) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const int first = S.first[n & 1][c + 16 * u + j];
                                if (REV ? row < first : row >= first) o[j >> 1] |= j & 1 ? 0x7FFF0000u : 0x7FFFu;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 8; j += 4)
                            *reinterpret_cast<uint4 *>(sY + (c >> 6) * 16384 + sw128_off(row, (c & 32) + 16 * u + 2 * j)) =
                                make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                }
                tc_fence_before();
                mbar_arrive(&S.y_free);
                fence_proxy_async();
                mbar_arrive(&S.y_written[n % NST]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

// Segments of a head.  Splitting pays where the heads leave SMs idle: the segments' own sums come first, their ends are
// joined, and every segment runs from its state.  In units of a block's time, 1.8 us (d64) to 3.2 (d128): a wave of CTAs takes its
// segments' length, once for y and about 0.6 times for the sums (measured as 0.42 at d64: B1 H32 N131072, 216 blocks in a row,
// sums 165 us, y 394; the rule leaves that margin), the extra launches and starts about 3 (with one piece of scores and states and
// before the launches overlapped: gradients of 24 heads of 9 blocks 79 us split in three, 83 whole; 8 heads of 8 blocks forward
// 29 and 33).
void retain_segments(const RetainArgs &a, int &nseg, int &seg_blocks) {
    const int nblk = (a.N + kTC - 1) / kTC, sms = num_sms();
    const long long BH = (long long)a.B * a.H;
    auto waves = [&](long long ctas) { return (double)((ctas + sms - 1) / sms); };
    nseg = 1;
    seg_blocks = nblk;
    if (BH >= sms) return;
    double best = waves(BH) * nblk;
    for (int s = 2; s <= 64 && s <= nblk; ++s) {
        const int len = (nblk + s - 1) / s, n = (nblk + len - 1) / len;
        if (n != s) continue;
        const double cost = 1.6 * waves(BH * s) * len + 3;
        if (cost < best) {
            best = cost;
            nseg = s;
            seg_blocks = len;
        }
    }
}

// behind: right behind the scan, and so early.
template <int D, int DV, bool REV, int MODE> cudaError_t launch_mode(const RetainArgs &a, const RetainTc &p, bool behind = false) {
    CUtensorMap qm{}, km, vm, ym{};
    if (!encode_tokens(&km, a.k, a.layout, a.B, a.H, a.N, D, kTC) || !encode_tokens(&vm, a.v, a.layout, a.B, a.H, a.N, DV, kTC) ||
        (MODE == kWhole && (!encode_tokens(&qm, a.q, a.layout, a.B, a.H, a.N, D, kTC) ||
                          !encode_tokens(&ym, a.y, a.layout, a.B, a.H, a.N, DV, kTC))))
        return cudaErrorInvalidValue;
    auto kern = retain_tc_kernel<D, DV, REV, MODE>;
    constexpr int smem = RetainLay<D, DV, MODE>::request;
    static_assert(smem <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (behind) return launch_overlapped(kern, dim3(a.B * a.H * p.segs), dim3(RetainLay<D, DV, MODE>::threads), smem, a.stream, qm, km, vm, ym, p);
    kern<<<a.B * a.H * p.segs, RetainLay<D, DV, MODE>::threads, smem, a.stream>>>(qm, km, vm, ym, p);
    return cudaGetLastError();
}

template <int D, int DV, bool REV> cudaError_t launch_tc(const RetainArgs &a) {
    RetainTc p{};
    p.gamma = a.gamma; p.H = a.H; p.N = a.N; p.nblk = (a.N + kTC - 1) / kTC;
    retain_segments(a, p.nseg, p.seg_blocks);
    WsHeader *hdr = static_cast<WsHeader *>(a.ws);
    p.err = &hdr->error;
    p.err_where = &hdr->error_where;
    const long long lim = debug_fault().wait_limit_ns;
    p.limit_ns = lim > 0 ? (unsigned long long)lim : 1000000000ull;
    p.drop_item = debug_fault().drop_load_item;
    if (p.nseg > 1) {   // the segments' sums; the last one taken is needed for the final state only
        float *states = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
        RetainTc s = p;
        s.S_out = states;
        s.segs = p.nseg - (a.S_out ? 0 : 1);
        s.seg0 = REV ? p.nseg - s.segs : 0;
        cudaError_t e = a.have_states ? cudaSuccess : launch_mode<D, DV, REV, kSums>(a, s);
        if (e == cudaSuccess && !a.have_states) e = launch_retain_scan(a, states, p.nseg, p.seg_blocks * kTC);
        if (e != cudaSuccess) return e;
        p.S_in = states;
        p.trans = a.have_states;
    } else {
        p.S_in = a.S_in;
        p.S_out = a.S_out;
        p.trans = a.trans;
    }
    p.segs = p.nseg;
    return launch_mode<D, DV, REV, kWhole>(a, p, p.nseg > 1 && !a.have_states);
}
template <int D, int DV> cudaError_t launch_way(const RetainArgs &a) {
    return a.rev ? launch_tc<D, DV, true>(a) : launch_tc<D, DV, false>(a);
}

}  // namespace

bool retain_tc_supported(const RetainArgs &a) {
    return a.dt == LA_DTYPE_BF16 && (a.d == 64 || a.d == 128) && (a.dv == 64 || a.dv == 128);
}
// header | (split sequences) the segments' sums, then states
size_t retain_tc_workspace(const RetainArgs &a) {
    int nseg, len;
    retain_segments(a, nseg, len);
    return nseg > 1 ? (size_t)a.B * a.H * nseg * a.d * a.dv * 4 : 0;
}
cudaError_t launch_retain_tc(const RetainArgs &a) {
    if (a.d == 64) return a.dv == 64 ? launch_way<64, 64>(a) : launch_way<64, 128>(a);
    return a.dv == 64 ? launch_way<128, 64>(a) : launch_way<128, 128>(a);
}

}  // namespace la
