// Attention over the 8-bit latent cache on the 5th-generation tensor core; codes
// go to it as they are stored.
//
// A CTA holds 64 query rows (token, head) and walks chunks of 128 cached tokens
// (two pages). Both products are formed transposed, with tokens or value
// dimensions as the 128 rows of the accumulator and the query rows as its
// columns, so that 64 rows (one token of 64 heads) fill the tensor core:
//
//   S^T [128 tokens, 64 hi | 64 lo] = K [128, D] (Qhi | Qlo)^T      kind::mxf8f6f4
//     A query row times 2^a, its largest magnitude in [2^7, 2^8), is the sum of
//     two E4M3 numbers, hi and lo / 16: exact for bf16 down to 2^-13 of the
//     largest, below that to 2^-22 of it. The rows' E8M0 scales 2^-a and 2^-a-4
//     undo it: s = hi + lo.
//   O^T [tiles of 128 dims, 64] += V^T (Phi + Plo)^T                the same
//     V is K's first columns, read from the same bytes. For every row and 32
//     tokens, b = round(max t) (t = s + e in the log2 domain, e the page scale's
//     exponent), the weights 2^(t - b + 8) < 363 are the sum of two E4M3 numbers
//     hi and lo / 16 (8 significant bits, absolute error 2^-14), and the block's
//     E8M0 scale is 2^(b - 8 - M) with M the row's reference: E4M3 alone spans 17
//     binades, too few beside a token that outweighs thousands of others; the
//     scale of every 32 tokens follows their own size. Row sums add the unrounded
//     weights times 2^(b - 8 - M - e) in fp32, so M is the first chunk's maximum of
//     b and b - e (an all-zero page has e = -60: its tokens weigh 2^60 times as much
//     in the sum as in O). It moves only when a block exceeds it by 2^60 (O and the
//     sum are then rescaled): E8M0 holds that, and a token's share of an element of
//     O stays below 2^70, its share of the sum below 2^61. The usual rescaling of O
//     whenever a maximum grows does not exist here.
//
// The full width, 512 + 64. Tensor memory: O^T 5 x 64 columns, S^T 128, scale
// words. Shared memory: the query tile 72 KB, two chunk stages of 72 KB (four
// boxes of 128 dims in the 128-byte swizzle, K-major for S^T and MN-major for
// O^T; the rope box in the 64-byte swizzle), Plo 8 KB; Phi takes the place of the
// chunk's rope box, which only S^T reads. A box goes back to the producer as soon
// as the products of its dimensions are done.
//
// The smaller widths (256 + 32, 128 + 32, 64 + 16) take boxes of 128 dims
// throughout, with zeros past the entry's end, and have room for three or four
// stages, both terms of the weights in a buffer of their own and every output tile
// in both terms at once (N = 128: V's codes are read once).
//
// Bound, full width: the loop of a stage, ~6700 clocks for the two chunks that the
// stages hold, against 5300 of tensor work. From a part freed to a part full 1300;
// scores 2000 (1165 alone; the other chunk's outputs run among them); softmax 2700
// (its shared-memory accesses wait behind the products' operand reads, which take
// the port's 2560 of 2650 clocks); first part free 600 later. A third stage, which
// would hide it, does not fit beside the queries. No one part of it is enough by
// itself: with half of the bytes loaded 6 % less, with 192 tensor clocks a chunk left
// out 1 %. An item costs ~16000 clocks more (queries converted ~5000, output
// ~6000, the pipeline drained and refilled). Two prompt chunks of 700 to 1024 tokens
// x 64 heads over 4-8K tokens: 1308 us, 1.30 PFLOP/s of the formulas' products; a
// block of 7 x 64 rows over 95000 tokens 86 us; 32 requests of 1-16K tokens, 64
// rows each, 58 us, 3.2 TB/s.
// Pairs of output products that share V (Phi's and Plo's of a tile) could take it
// from the tensor core's collector, 39 clocks a product against 48; that needs
// nothing issued between them, hence one issuing thread, and with one thread for
// scores and outputs the prompt chunks take 1500 us. Bound, smaller widths: the
// latency of the softmax's chain on two warps a scheduler, ~2500 clocks a chunk
// whatever the width (32 requests of 1K to 16K tokens and 64 heads: 39, 36 and 35
// us; products by mma.sync in f16, codes widened on the way, took 130, 71 and 49; two
// prompt chunks of 600 tokens over 4-8K 505, 471 and 462).
//
// Roles (12 warps): warp 0 TMA producer; warp 1 issues the scores (and owns tensor
// memory), warp 2 the outputs, so that whichever of the two is ready keeps the
// tensor core busy; warps 4-11 queries, softmax and output (a thread holds one
// token of 32 rows) with the registers that the first four give up. All waits are
// bounded; a timeout raises DSPARK_ERR_TIMEOUT.
#include <math.h>

#include "e4m3.cuh"
#include "internal.h"
#include "per_device.h"
#include "qattn.cuh"

namespace ds {

constexpr int kQtKeys = kQaChunk;                  // tokens per chunk
constexpr int kQtThreads = kQaThreads;
constexpr int kQtSoft0 = 4;                        // first softmax warp; registers: 168 x 384 = 88 x 128 + 208 x 256
constexpr int kQtRegsIssue = 88, kQtRegsSoft = 208;
constexpr int kQtBox = kQtKeys * 128;              // bytes: 128 tokens x 128 dims
constexpr int kQtTerm = kQtKeys * 64;              // one E4M3 term of the weights: 128 tokens x 64 rows
constexpr int kQtMoveLog2 = 60;
constexpr int kQtLost = kQcEmax + 1;               // in the place of a page's exponent: rows that see the page are NaN

// kWide: the full width, 512 + 64. The others leave room: more stages, whole
// stages handed over at once, both terms of the weights in a buffer of their own
// and every output tile taken in both terms at once.
template <int KV, int ROPE>
struct QtCfg {
    static constexpr bool kWide = KV == 512;
    static constexpr int kD = KV + ROPE;
    static constexpr int kTiles = KV < 128 ? 1 : KV / 128;            // output tiles of 128 dims
    static constexpr int kBoxes = kWide ? 4 : (kD + 127) / 128;       // boxes of 128 dims (zeros past the entry's end)
    static constexpr int kRope = kWide ? kQtKeys * 64 : 0;            // the rope's box of 64 dims
    static constexpr int kStage = kBoxes * kQtBox + kRope;
    static constexpr int kStages = kWide ? 2 : KV == 256 ? 3 : 4;
    static constexpr int kBars = kWide ? 5 : 1;                       // parts of a stage that are filled and freed
    static constexpr int kQ = kStage;                                 // (64 hi + 64 lo) query rows, laid out like a stage
    static constexpr int kP = kWide ? kQtTerm : 2 * kQtTerm;          // wide: Plo alone
    static constexpr int kLastSteps = (kD - 128 * (kBoxes - 1) + 31) / 32;  // 32-dim steps of the last box (not wide)
    static constexpr int kPer = ((kWide ? kD : 128 * (kBoxes - 1) + 32 * kLastSteps) / 8 + 3) / 4;  // query pieces a lane converts
    static constexpr int kRound = kPer % 3 == 0 ? 3 : kPer;
    static constexpr int kPitch = KV * 2 + 16;                        // staged output row, bytes
    // tensor-memory columns: O^T (wide: its first tile twice, Phi's and Plo's share; else every tile twice), S^T, scale words
    static constexpr int kColO = 0, kColS = kWide ? 320 : 128 * kTiles, kColSfa = kColS + 128, kColSfb = kColSfa + 4, kColSfq = kColSfb + 8;
    static_assert(kColSfq + 4 <= 512, "tensor memory");
    static_assert(kQaTile * kPitch <= kQ, "the staged output takes the place of the queries");
    static_assert(QaWork::kScratch <= kStages * kStage, "scratch of the work division");
};

template <int STAGES, int BARS>
struct QtMisc {
    uint64_t full[STAGES][BARS], free_[STAGES][BARS];  // wide: boxes 0..3, rope
    // Arrivals of one chunk on a barrier must not mix with those of the next. Scores, second terms and outputs follow one
    // another through all warps; first terms do not (a group of warps may be one chunk ahead of the other, which
    // may be moving its references), so they take turns on two barriers: the one of chunk i is used again
    // for chunk i + 2, behind the outputs of chunk i.
    uint64_t s_full, s_free, hi_ready[2], lo_ready, pv_done, q_ready, item_done, mma_done, grp[2];
    uint32_t tmem;
    volatile int abort;
    uint8_t issued[STAGES][8];         // loads in flight: 1 | parity << 1, per part
    int8_t e[STAGES][2];               // page scale exponents of a stage's pages
    int qe[kQaTile];                   // biased exponent that undoes a query row's scaling; 0: a non-finite query
    alignas(16) int lim[kQaTile];      // tokens that a row sees
    // Per warp, one value per row. Chunk i has w[i & 1] for its maxima, then what it adds to the exponents (e + 8 - b,
    // which tells the group's other warps b), and w[~i & 1] for the sums' factors, once the group has met: the others
    // have then read the chunk before's. Row sums and output factors of an item's end take turns likewise.
    alignas(16) float w[2][8][32];
};
template <int KV, int ROPE>
constexpr int qt_smem_bytes() {
    using C = QtCfg<KV, ROPE>;
    using Misc = QtMisc<C::kStages, C::kBars>;
    constexpr int n = C::kQ + C::kStages * C::kStage + C::kP + (int)sizeof(Misc);
    static_assert(n <= 232448, "shared memory");
    return n;
}

// One lane of the warp. A branch on it is known to hold a single thread, so an
// MMA's operands are formed in uniform registers: 64 clocks a score step, against
// 95 in a branch on lane == 0.
DS_DEVINL bool qt_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
DS_DEVINL float redux_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
// An integer 0 <= x < 2^8 held as a float: its bits, below those of 2^23.
DS_DEVINL uint32_t qt_bits(float x) { return __float_as_uint(x + 0x1p23f); }
DS_DEVINL float qt_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
DS_DEVINL void tmem_st1(uint32_t addr, uint32_t v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(v) : "memory");
}
DS_DEVINL void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
DS_DEVINL bool qt_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort));
}

template <int KV, int ROPE>
__global__ void __launch_bounds__(kQtThreads, 1)
    qattn_tc_kernel(const __grid_constant__ CUtensorMap tm_dims, const __grid_constant__ CUtensorMap tm_rope,
                    const QaParams p) {
    using C = QtCfg<KV, ROPE>;
    using W = QaWork;
    using Misc = QtMisc<C::kStages, C::kBars>;
    extern __shared__ __align__(1024) uint8_t qt_smem[];
    uint8_t *sQ = qt_smem, *sK = sQ + C::kQ, *sP = sK + C::kStages * C::kStage;
    Misc &ms = *(Misc *)(sP + C::kP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, grid = gridDim.x;

    pdl_trigger();
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s)
            for (int d = 0; d < C::kBars; ++d) {
                mbar_init(&ms.full[s][d], 1);
                mbar_init(&ms.free_[s][d], 1);
                ms.issued[s][d] = 0;
            }
        mbar_init(&ms.s_full, 1);
        mbar_init(&ms.s_free, 8);
        mbar_init(&ms.hi_ready[0], 8);
        mbar_init(&ms.hi_ready[1], 8);
        mbar_init(&ms.lo_ready, 8);
        mbar_init(&ms.pv_done, 1);
        mbar_init(&ms.q_ready, 8);
        mbar_init(&ms.item_done, 8);
        mbar_init(&ms.mma_done, 2);
        mbar_init(&ms.grp[0], 4);
        mbar_init(&ms.grp[1], 4);
        ms.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_dims);
        if (C::kWide) tma_prefetch_desc(&tm_rope);
    }
    if (warp == 1) tmem_alloc(&ms.tmem, 512);
    pdl_wait();
    W wk;
    wk.find(p, cta, grid, sK);
    fence_async_smem();  // the scratch was written through the generic proxy
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem;
    long long left = wk.end - wk.begin;
    volatile int *abort = &ms.abort;
    uint32_t ci = 0;  // chunks of this CTA so far

    if (warp < kQtSoft0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQtRegsIssue));
    if (warp == 0) {
        // ---- producer: page numbers and scales 32 pages at a time, one block ahead
        bool ok = true;
        while (left > 0 && ok) {
            const QaItem it = wk.item;
            const int take = (int)min((long long)(it.chunks - wk.off), left);
            const int npages = (it.len + kQcPage - 1) / kQcPage, first = 2 * wk.off;
            const int32_t *row = p.page_table + (size_t)it.b * p.max_pages;
            // page number i of the request (0 past its end; one outside the pool becomes the first behind the pool, where
            // the copy reads nothing and fills in zeros)
            auto page = [&](int i) {
                int pg = i < npages && i < first + 2 * take ? row[i] : 0;
                if (pg < 0 || pg >= p.n_pages) {
                    set_error(p.err, DSPARK_ERR_OOB);
                    pg = p.n_pages;
                }
                return pg;
            };
            // its scale's exponent; kQtLost: a page without a number or a scale
            auto exponent = [&](int i, int pg) {
                int e = 0;
                if (pg == p.n_pages) return kQtLost;
                if (i < npages && i < first + 2 * take && !qc_scale_exponent(p.scales[pg], &e)) {
                    set_error(p.err, DSPARK_ERR_BAD_INPUT);
                    return kQtLost;
                }
                return e;
            };
            int pg = page(first + lane), ex = exponent(first + lane, pg), pg_n = 0, ex_n = 0;
            for (int i = 0; i < take && ok; ++i, ++ci) {
                const int j = i & 15;
                if (j == 0) {
                    if (i > 0) {
                        pg = pg_n;
                        ex = ex_n;
                    }
                    pg_n = page(first + 2 * (i + 16) + lane);
                }
                if (j == 8) ex_n = exponent(first + 2 * (i + 8) + lane, pg_n);
                const int pa = __shfl_sync(~0u, pg, 2 * j), pb = __shfl_sync(~0u, pg, 2 * j + 1);
                const int ea = __shfl_sync(~0u, ex, 2 * j), eb = __shfl_sync(~0u, ex, 2 * j + 1);
                if (qt_elect()) {
                    const int st = ci % C::kStages, n = max(0, min(2, npages - (first + 2 * i)));
                    const uint32_t par = (ci / C::kStages) & 1;
                    uint8_t *dst = sK + st * C::kStage;
                    const int ya = pa * kQcPage, yb = pb * kQcPage;
                    // wide: the parts in the order in which they come free
#pragma unroll
                    for (int x = 0; x < C::kBars; ++x) {
                        const int d = !C::kWide ? 0 : x < 2 ? x ^ 1 : x == 2 ? 2 : 7 - x;  // 1, 0, 2, rope, 3
                        if (ci >= C::kStages && !mbar_wait_bounded(&ms.free_[st][d], par ^ 1, abort)) {
                            ok = false;
                            break;
                        }
                        uint64_t *bar = &ms.full[st][d];
                        // 16-bit elements: 64 (the rope's box: 32) of them a box row
                        if constexpr (C::kWide) {
                            const int bytes = d < 4 ? kQtBox / 2 : C::kRope / 2;
                            uint8_t *to = dst + d * kQtBox;
                            if (n > 0) tma_load_2d(to, d < 4 ? &tm_dims : &tm_rope, d < 4 ? d * 64 : 256, ya, bar);
                            if (n > 1) tma_load_2d(to + bytes, d < 4 ? &tm_dims : &tm_rope, d < 4 ? d * 64 : 256, yb, bar);
                        } else {
#pragma unroll
                            for (int d2 = 0; d2 < C::kBoxes; ++d2) {
                                if (n > 0) tma_load_2d(dst + d2 * kQtBox, &tm_dims, d2 * 64, ya, bar);
                                if (n > 1) tma_load_2d(dst + d2 * kQtBox + kQtBox / 2, &tm_dims, d2 * 64, yb, bar);
                            }
                        }
                        if (x == 0) {
                            // Every part's barrier at once, behind the first loads: each has completed its last phase (the
                            // stage's scores are done when its first part is free), and none completes without this.
                            ms.e[st][0] = (int8_t)ea;
                            ms.e[st][1] = (int8_t)eb;
#pragma unroll
                            for (int y = 0; y < C::kBars; ++y) {
                                const int part = !C::kWide ? C::kStage : y < 4 ? kQtBox : C::kRope;
                                if (n > 0) mbar_arrive_expect_tx(&ms.full[st][y], (uint32_t)(n * (part / 2)));
                                else mbar_arrive(&ms.full[st][y]);
                            }
                        }
                        ms.issued[st][d] = (uint8_t)(1 | par << 1);
                    }
                }
                ok = __all_sync(~0u, ok);
            }
            left -= take;
            if (left > 0) wk.next(p);
        }
    } else if (warp == 1) {
        // ---- scores: chunk ci + 1 while the softmax works on chunk ci
        if (qt_elect()) {
            // everything about an operand but its stage is a constant added to one word: the
            // issuing thread shares its scheduler with softmax warps
            const uint32_t q_lo = sdesc_lo(smem_u32(sQ)), k_lo = sdesc_lo(smem_u32(sK));
            constexpr uint32_t kHi128 = sdesc_hi(1024, 2), kHi64 = sdesc_hi(512, 4), id = idesc_mx_e4m3(128, 128, 0);
            const uint32_t sfk = tmem + C::kColSfa, sfq = tmem + C::kColSfq;
            bool ok = true;
            for (uint32_t items = 0; left > 0 && ok; ++items) {
                const int take = (int)min((long long)(wk.item.chunks - wk.off), left);
                ok = mbar_wait_bounded(&ms.q_ready, items & 1, abort);
                for (int i = 0; i < take && ok; ++i, ++ci) {
                    ok = i == 0 || mbar_wait_bounded(&ms.s_free, (ci - 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t st = ci % C::kStages, par = (ci / C::kStages) & 1;
                    const uint32_t a0 = k_lo + st * (C::kStage >> 4);
                    if constexpr (C::kWide) {
                        // boxes in the order in which they come free
#pragma unroll 1
                        for (int x = 0; x < 3; ++x) {
                            const int d = x < 2 ? x ^ 1 : 2;
                            ok = mbar_wait_bounded(&ms.full[st][d], par, abort);
                            if (!ok) break;
                            const uint32_t a = a0 + d * (kQtBox >> 4), b = q_lo + d * (kQtBox >> 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_mx_e4m3_w(tmem + C::kColS, a + 2 * k, kHi128, b + 2 * k, kHi128, id, sfk, sfq, k > 0 ? 1u : (uint32_t)(x > 0));
                        }
                        ok = ok && mbar_wait_bounded(&ms.full[st][4], par, abort);
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma_mx_e4m3_w(tmem + C::kColS, a0 + (4 * kQtBox >> 4) + 2 * k, kHi64, q_lo + (4 * kQtBox >> 4) + 2 * k, kHi64, id, sfk, sfq, 1);
                        ok = mbar_wait_bounded(&ms.full[st][3], par, abort);
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_mx_e4m3_w(tmem + C::kColS, a0 + (3 * kQtBox >> 4) + 2 * k, kHi128, q_lo + (3 * kQtBox >> 4) + 2 * k, kHi128, id, sfk, sfq, 1);
                    } else {
                        ok = mbar_wait_bounded(&ms.full[st][0], par, abort);
                        if (!ok) break;
#pragma unroll
                        for (int d = 0; d < C::kBoxes; ++d)
#pragma unroll
                            for (int k = 0; k < (d + 1 < C::kBoxes ? 4 : C::kLastSteps); ++k)
                                mma_mx_e4m3_w(tmem + C::kColS, a0 + d * (kQtBox >> 4) + 2 * k, kHi128, q_lo + d * (kQtBox >> 4) + 2 * k,
                                              kHi128, id, sfk, sfq, d > 0 || k > 0);
                    }
                    mma_commit(&ms.s_full);
                }
                left -= take;
                if (left > 0) wk.next(p);
            }
            mma_commit(&ms.mma_done);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- outputs
        if (qt_elect()) {
            const uint32_t k_lo = sdesc_lo(smem_u32(sK)), p_lo = sdesc_lo(smem_u32(sP));
            constexpr uint32_t kHi128 = sdesc_hi(1024, 2), kHi64 = sdesc_hi(512, 4);
            bool ok = true;
            while (left > 0 && ok) {
                const int take = (int)min((long long)(wk.item.chunks - wk.off), left);
                for (int i = 0; i < take; ++i, ++ci) {
                    const uint32_t st = ci % C::kStages, a0 = k_lo + st * (C::kStage >> 4);
                    const uint32_t sfa = tmem + C::kColSfa, sfb = tmem + C::kColSfb + 4 * (ci & 1), first = i > 0;
                    if constexpr (C::kWide) {
                        // Two tiles' Phi products start while the split's second terms are made. The first
                        // tile takes both terms at once (N = 128, its codes are read once); tensor memory
                        // has no room for a second such tile.
                        const uint32_t phi = a0 + (4 * kQtBox >> 4);
                        auto tile = [&](int d, uint32_t b, uint32_t sf, uint32_t acc) {
                            const uint32_t a = a0 + d * (kQtBox >> 4), col = tmem + C::kColO + 64 + 64 * d;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_mx_e4m3_w(col, a + 256 * k, kHi128, b + 128 * k, kHi64, idesc_mx_e4m3(128, 64, k) | kIdescBothMN, sfa, sf,
                                              k > 0 ? 1u : acc);
                        };
                        ok = mbar_wait_bounded(&ms.hi_ready[ci & 1], (ci >> 1) & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        tile(1, phi, sfb, first);
                        tile(2, phi, sfb, first);
                        ok = mbar_wait_bounded(&ms.lo_ready, ci & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        tile(1, p_lo, sfb + 2, 1);
                        mma_commit(&ms.free_[st][1]);
                        {
                            // Plo's 64 columns lie p_lo - phi behind Phi's: the distance of the operand's two halves
                            const uint32_t b = (phi & 0xffffu) | (p_lo - phi) << 16;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_mx_e4m3_w(tmem + C::kColO, a0 + 256 * k, kHi128, b + 128 * k, kHi64, idesc_mx_e4m3(128, 128, k) | kIdescBothMN,
                                              sfa, sfb, k > 0 ? 1u : first);
                        }
                        mma_commit(&ms.free_[st][0]);
                        tile(3, phi, sfb, first);
                        mma_commit(&ms.free_[st][4]);
                        tile(2, p_lo, sfb + 2, 1);
                        mma_commit(&ms.free_[st][2]);
                        tile(3, p_lo, sfb + 2, 1);
                        mma_commit(&ms.free_[st][3]);
                    } else {
                        ok = mbar_wait_bounded(&ms.lo_ready, ci & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        // both terms at once: Plo's 64 columns lie kQtTerm behind Phi's
                        const uint32_t b = (p_lo & 0xffffu) | (uint32_t)(kQtTerm >> 4) << 16;
#pragma unroll 1
                        for (int d = 0; d < C::kTiles; ++d)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_mx_e4m3_w(tmem + C::kColO + 128 * d, a0 + d * (kQtBox >> 4) + 256 * k, kHi128, b + 128 * k, kHi64,
                                              idesc_mx_e4m3(128, 128, k) | kIdescBothMN, sfa, sfb, k > 0 ? 1u : first);
                        mma_commit(&ms.free_[st][0]);
                    }
                    mma_commit(&ms.pv_done);
                }
                left -= take;
                if (left > 0) wk.next(p);
            }
            mma_commit(&ms.mma_done);
            mbar_drain(&ms.mma_done, 0);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQtRegsSoft));
        // ---- queries, softmax, output: thread = token 32 q4 + lane of the chunk, rows 32 g ..
        const int g = (warp - kQtSoft0) >> 2, q4 = warp & 3, tok = 32 * q4 + lane;
        const uint32_t tl = tmem + ((uint32_t)(32 * q4) << 16);
        uint32_t gph = 0;
        auto group_arrive = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.grp[g]);
        };
        auto group_wait = [&]() { return qt_warp_wait(&ms.grp[g], gph++ & 1, abort); };
        auto group_sync = [&]() {
            group_arrive();
            return group_wait();
        };
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_st1(tl + C::kColSfa + k, 0x7f7f7f7fu);  // V is not scaled
        long long unit = wk.begin;
        QaSplit sp;
        sp.q0 = sp.r0 = sp.rows = sp.lo_slot = 0;
        sp.c_hi = -1;
        int slot = 2 * cta;
        bool ok = true;
        for (uint32_t items = 0; left > 0 && ok; ++items, slot = 2 * cta + 1) {
            const QaItem it = wk.item;
            const int take = (int)min((long long)(it.chunks - wk.off), left);
            const bool first = wk.off == 0, whole = first && take == it.chunks;
            if (first && !whole) {
                sp.q0 = it.q0;
                sp.r0 = it.t * kQaTile;
                sp.rows = it.nq * p.H - sp.r0;
                sp.lo_slot = slot;
                sp.c_hi = wk.last_cta(unit);
            }
            const int r0 = it.t * kQaTile, R = it.nq * p.H;
            // query rows as E4M3 pairs: 8 rows a warp, four lanes a row
            {
                constexpr int kPer = C::kPer;  // 16-byte pieces of a row per lane
                const int r = 8 * (warp - kQtSoft0) + (lane >> 2);
                const bool in = r0 + r < R;
                const int tq = in ? (int)W::token(p, r0 + r) : 0, hd = in ? (r0 + r) - tq * p.H : 0;
                const uint4 *src = (const uint4 *)(p.q + (size_t)(it.q0 + tq) * p.q_stride + (size_t)hd * C::kD) + (lane & 3);
                uint4 v[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    v[j] = in && (4 * kPer * 8 == C::kD || (lane & 3) + 4 * j < C::kD / 8) ? __ldg(src + 4 * j) : make_uint4(0, 0, 0, 0);
                uint32_t mx = 0;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const uint32_t *u = (const uint32_t *)&v[j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = max(mx, max((u[i] << 16) & 0x7fffffffu, u[i] & 0x7fff0000u));
                }
                mx = max(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = max(mx, __shfl_xor_sync(~0u, mx, 2));
                const bool bad = mx >= 0x7f800000u;
                const int a = min(mx < 0x00800000u ? 0 : 7 - ((int)(mx >> 23) - 127), 100);
                const float f = qc_pow2(a);
                if (bad) {  // the row's outputs are NaN whatever it is here; scores stay finite
#pragma unroll
                    for (int j = 0; j < kPer; ++j) v[j] = make_uint4(0, 0, 0, 0);
                }
                // the item before: its staged output has been read
                if (items > 0 && !qt_warp_wait(&ms.item_done, (items - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                // a few pieces a round: the loop stays small (instruction fetch, not arithmetic, is what
                // straight-line code that runs once costs), the registers move up instead
#pragma unroll 1
                for (int j0 = 0; j0 < kPer; j0 += C::kRound) {
#pragma unroll
                    for (int j = 0; j < C::kRound; ++j) {
                        const int pc = (lane & 3) + 4 * (j0 + j);  // 8 elements each
                        const uint32_t *u = (const uint32_t *)&v[j];
                        uint32_t hi[2], lo[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[2], x[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t two = u[2 * i + k];
                                const uint32_t h16 = f32x2_to_f16x2(__uint_as_float(two << 16) * f, __uint_as_float(two & 0xffff0000u) * f);
                                w[k] = f16x2_to_e4m3x2(h16);
                                x[k] = f16x2_to_e4m3x2(f16x2_sub_x16(h16, e4m3x2_to_f16x2_(w[k])));
                            }
                            hi[i] = w[0] | w[1] << 16;
                            lo[i] = x[0] | x[1] << 16;
                        }
                        // 16-byte pieces: c ^ (row & 7) in 128-byte rows, c ^ (row / 2 & 3) in the rope's 64-byte
                        // rows; the same for row r + 64
                        const int d = pc >> 4, c = (pc & 15) >> 1;
                        const bool rope = C::kWide && d == 4;
                        const int rs = rope ? 64 : 128, ch = rope ? (c ^ ((r >> 1) & 3)) : (c ^ (r & 7));
                        uint8_t *at = sQ + d * kQtBox + r * rs + ch * 16 + (pc & 1) * 8;
                        *(uint2 *)at = make_uint2(hi[0], hi[1]);
                        *(uint2 *)(at + 64 * rs) = make_uint2(lo[0], lo[1]);
                    }
#pragma unroll
                    for (int j = 0; j + C::kRound < kPer; ++j) v[j] = v[j + C::kRound];
                }
                if ((lane & 3) == 0) {
                    ms.qe[r] = bad ? 0 : 127 - a;  // a <= 100 and >= 7 - 127
                    ms.lim[r] = in ? W::sees(p, it.nq, it.len, tq) : 0;
                    if (bad && first) set_error(p.err, DSPARK_ERR_BAD_INPUT);
                }
            }
            fence_async_smem();
            ok = group_sync();  // qe and lim of the rows of this group come from its own four warps
            if (!ok) break;
            const int qe = ms.qe[32 * g + lane];
            tmem_st1(tl + C::kColSfq + g, (uint32_t)max(qe, 4) * 0x01010101u);            // hi rows
            tmem_st1(tl + C::kColSfq + 2 + g, (uint32_t)(max(qe, 4) - 4) * 0x01010101u);  // lo rows: 2^-4 of it
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_ready);

            float l[32], mref = 0.f;  // mref: the reference of row 32 g + lane
            bool lost = false;        // that row has no answer
#pragma unroll
            for (int j = 0; j < 32; ++j) l[j] = 0.f;
            // every row of the tile sees at least what its first row sees
            const int all_see = W::sees(p, it.nq, it.len, (int)W::token(p, r0));
            for (int i = 0; i < take; ++i, ++ci) {
                const int base = (wk.off + i) * kQtKeys, st = ci % C::kStages;
                ok = qt_warp_wait(&ms.full[st][C::kWide ? 1 : 0], (ci / C::kStages) & 1, abort);  // e; long done when the scores are
                if (!ok) break;
                const int e = ms.e[st][q4 >> 1];
                const float fe = (float)e, c = fmaxf(qc_pow2(e) * p.scale_log2, 1.2e-38f);  // > 0: masked stays -inf
                ok = qt_warp_wait(&ms.s_full, ci & 1, abort);
                if (!ok) break;
                tc_fence_after();
                float t[32];
                {
                    uint32_t a[2][16], b[2][16];
                    tmem_ld16_issue(tl + C::kColS + 32 * g, a[0]);
                    tmem_ld16_issue(tl + C::kColS + 64 + 32 * g, b[0]);
                    tmem_ld16_issue(tl + C::kColS + 32 * g + 16, a[1]);
                    tmem_ld16_issue(tl + C::kColS + 64 + 32 * g + 16, b[1]);
                    tmem_ld_wait_tied(a[0]);
                    tmem_ld_wait_tied(a[1]);
                    tmem_ld_wait_tied(b[0]);
                    tmem_ld_wait_tied(b[1]);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        t[j] = __uint_as_float(a[j >> 4][j & 15]) + __uint_as_float(b[j >> 4][j & 15]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.s_free);
                if (base + kQtKeys > all_see) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const int4 m = *(const int4 *)&ms.lim[32 * g + j];
                        if (base + tok >= m.x) t[j] = -INFINITY;
                        if (base + tok >= m.y) t[j + 1] = -INFINITY;
                        if (base + tok >= m.z) t[j + 2] = -INFINITY;
                        if (base + tok >= m.w) t[j + 3] = -INFINITY;
                    }
                    const int nvalid = max(0, it.len - base);
                    if (nvalid < kQtKeys) {
                        // no tokens here: zero value rows, so that weights of 0 meet finite codes
                        uint8_t *kb = sK + st * C::kStage + nvalid * 128;
                        const int pieces = (kQtKeys - nvalid) * 8;  // per box
                        for (int x = tid - 32 * kQtSoft0; x < pieces; x += 256)
#pragma unroll
                            for (int d = 0; d < C::kBoxes; ++d) *(uint4 *)(kb + d * kQtBox + x * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                // block maxima (the lanes' 32 tokens are one scale block of one page; the
                // factor is positive, so the maximum of the raw scores is the one), then
                // lane j prepares row j: b, and the exponent's addend e + 8 - b
                float *wrow = ms.w[ci & 1][warp - kQtSoft0], *wsum = ms.w[~ci & 1][warp - kQtSoft0];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 m = make_float4(redux_max(t[j]), redux_max(t[j + 1]), redux_max(t[j + 2]), redux_max(t[j + 3]));
                    if (lane == 0) *(float4 *)(wrow + j) = m;
                }
                __syncwarp();
                // (up to 2^23 differences from b are exact: as far as fp32 tells scores apart; a block that the row sees
                // and whose maximum lies beyond that, or is none, makes the row NaN; so does a lost page)
                const float bx = __fmaf_rn(wrow[lane], c, fe);
                if (!(fabsf(bx) <= 0x1p23f) || e == kQtLost) lost |= ms.lim[32 * g + lane] > base + 32 * q4;
                const float bf = rintf(fminf(fmaxf(bx, -0x1p23f), 0x1p23f));
                __syncwarp();
                wrow[lane] = (fe + 8.f) - bf;
                group_arrive();  // the wait comes after the weights
                // weights
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 x = *(const float4 *)(wrow + j);
                    t[j] = qt_ex2(__fmaf_rn(t[j], c, x.x));
                    t[j + 1] = qt_ex2(__fmaf_rn(t[j + 1], c, x.y));
                    t[j + 2] = qt_ex2(__fmaf_rn(t[j + 2], c, x.z));
                    t[j + 3] = qt_ex2(__fmaf_rn(t[j + 3], c, x.w));
                }
                // their first E4M3 terms
                uint32_t h16[16], hi[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h16[2 * j] = f32x2_to_f16x2(t[4 * j], t[4 * j + 1]);
                    h16[2 * j + 1] = f32x2_to_f16x2(t[4 * j + 2], t[4 * j + 3]);
                    hi[j] = f16x2_to_e4m3x2(h16[2 * j]) | f16x2_to_e4m3x2(h16[2 * j + 1]) << 16;
                }
                // wide: Phi over the chunk's rope box (its scores are done)
                const int sw = (tok >> 1) & 3;
                uint8_t *ph = (C::kWide ? sK + st * C::kStage + 4 * kQtBox : sP) + tok * 64;
                if constexpr (C::kWide) {
                    *(uint4 *)(ph + ((2 * g) ^ sw) * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *(uint4 *)(ph + ((2 * g + 1) ^ sw) * 16) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    fence_async_smem();
                }
                ok = group_wait();
                if (!ok) break;
                float bq[4], bm = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float ek = (float)ms.e[st][k >> 1], s = 8.f - ms.w[ci & 1][4 * g + k][lane];  // s = b - e
                    bq[k] = s + ek;
                    bm = fmaxf(bm, s + fmaxf(ek, 0.f));
                }
                const bool move = i == 0 || bm - mref > (float)kQtMoveLog2;
                if (__any_sync(~0u, move)) {  // the same in the group's four warps
                    const float mnew = move ? bm : mref;
                    const float f = i == 0 ? 0.f : qt_ex2(mref - mnew);
                    mref = mnew;
                    if (i > 0) {
                        ok = qt_warp_wait(&ms.pv_done, (ci - 1) & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int j = 0; j < 32; ++j) l[j] *= __shfl_sync(~0u, f, j);
#pragma unroll 1
                        for (int k = 0; k < (C::kColS - C::kColO) / 32; ++k) {
                            float v[16];
                            uint32_t u[16];
                            const uint32_t at = tl + C::kColO + 64 * (k >> 1) + 32 * g + 16 * (k & 1);
                            tmem_ld16(at, v);
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(v[j] * __shfl_sync(~0u, f, 16 * (k & 1) + j));
                            tmem_st16(at, u);
                        }
                    }
                }
                // scale words of row 32 g + lane: 2^(b - 8 - M) for hi, 2^-4 of it for lo, one byte per 32 tokens
                {
                    uint32_t wh = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) wh |= (qt_bits(fminf(fmaxf(bq[k] - mref + (127.f - 8.f), 4.f), 250.f)) & 0xffu) << (8 * k);
                    tmem_st1(tl + C::kColSfb + 4 * (ci & 1) + g, wh);
                    tmem_st1(tl + C::kColSfb + 4 * (ci & 1) + 2 + g, wh - 0x04040404u);
                }
                if constexpr (C::kWide) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.hi_ready[ci & 1]);
                }
                // the second terms, once the chunk before has read its own
                uint32_t lo[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    lo[j] = f16x2_to_e4m3x2(f16x2_sub_x16(h16[2 * j], e4m3x2_to_f16x2_(hi[j] & 0xffffu))) |
                            f16x2_to_e4m3x2(f16x2_sub_x16(h16[2 * j + 1], e4m3x2_to_f16x2_(hi[j] >> 16))) << 16;
                if (ci > 0 && !qt_warp_wait(&ms.pv_done, (ci - 1) & 1, abort)) {
                    ok = false;
                    break;
                }
                uint8_t *pl = sP + (C::kWide ? 0 : kQtTerm) + tok * 64;
                if constexpr (!C::kWide) {
                    *(uint4 *)(ph + ((2 * g) ^ sw) * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *(uint4 *)(ph + ((2 * g + 1) ^ sw) * 16) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    tmem_st_wait();
                    tc_fence_before();
                }
                *(uint4 *)(pl + ((2 * g) ^ sw) * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                *(uint4 *)(pl + ((2 * g + 1) ^ sw) * 16) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                fence_async_smem();
                // lane j: what a weight of row j adds to the sum, 2^(b - 8 - M - e)
                wsum[lane] = __uint_as_float(qt_bits(fmaxf(bf - mref - fe + (127.f - 8.f), 0.f)) << 23);
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.lo_ready);
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 x = *(const float4 *)(wsum + j);
                    l[j] = __fmaf_rn(t[j], x.x, l[j]);
                    l[j + 1] = __fmaf_rn(t[j + 1], x.y, l[j + 1]);
                    l[j + 2] = __fmaf_rn(t[j + 2], x.z, l[j + 2]);
                    l[j + 3] = __fmaf_rn(t[j + 3], x.w, l[j + 3]);
                }
                __syncwarp();
            }
            if (!ok) break;
            // row sums: lane j ends with the sum of row 32 g + j over the warp's tokens, then over the four warps
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) {
#pragma unroll
                for (int k = 0; k < w; ++k) {
                    const bool up = (lane & w) != 0;
                    const float send = up ? l[k] : l[k + w], keep = up ? l[k + w] : l[k];
                    l[k] = keep + __shfl_xor_sync(~0u, send, w);
                }
            }
            float (*const sums)[32] = ms.w[ci & 1];
            const float nan = __uint_as_float(0x7fffffffu);
            sums[warp - kQtSoft0][lane] = lost ? nan : l[0];
            if (lost) set_error(p.err, DSPARK_ERR_BAD_INPUT);
            ok = group_sync() && qt_warp_wait(&ms.pv_done, (ci - 1) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            // 16 rows of the output: tile d's, the two terms' shares added where they are apart
            auto load_o = [&](int d, int half, float (&v)[16]) {
                const uint32_t at = tl + C::kColO + 32 * g + 16 * half + (C::kWide ? (d ? 64 + 64 * d : 0) : 128 * d);
                tmem_ld16(at, v);
                if (!C::kWide || d == 0) {
                    float x[16];
                    tmem_ld16(at + 64, x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += x[j];
                }
            };
            const bool real = KV >= 128 || q4 < KV / 32;  // 64 dims: half of the tile
            const float lsum = (sums[4 * g][lane] + sums[4 * g + 1][lane]) + (sums[4 * g + 2][lane] + sums[4 * g + 3][lane]);
            const bool bad = qe == 0 || isnan(lsum);
            const int row = 32 * g + lane, r = r0 + row;
            if (q4 == 0) {
                if (!whole) {
                    p.part_ml[slot * kQaTile + row] = make_float2(mref, bad ? nan : lsum);
                } else if (r < R && p.lse) {
                    const int tk = (int)W::token(p, r), tq = it.q0 + tk, hd = r - tk * p.H;
                    p.lse[(size_t)tq * p.H + hd] = bad ? nan : lsum > 0.f ? (mref + log2f(lsum)) * 0.6931471805599453f : -INFINITY;
                }
            }
            if (!whole) {
                float *dst = p.part_o + ((size_t)slot * kQaTile + 32 * g) * KV + 32 * q4 + lane;
#pragma unroll 1
                for (int k = 0; k < 2 * C::kTiles && real; ++k) {
                    float v[16];
                    load_o(k >> 1, k & 1, v);
                    float *at = dst + 16 * (k & 1) * KV + 128 * (k >> 1);
#pragma unroll
                    for (int j = 0; j < 16; ++j) at[j * KV] = v[j];
                }
            } else {
                // staged over the queries (every score is done), then whole rows
                float *inv = ms.w[~ci & 1][warp - kQtSoft0];
                inv[lane] = bad ? nan : lsum > 0.f ? 1.f / lsum : 0.f;
                __syncwarp();
                uint8_t *out = sQ + 32 * g * C::kPitch + (32 * q4 + lane) * 2;
#pragma unroll 1
                for (int k = 0; k < 2 * C::kTiles && real; ++k) {
                    float v[16];
                    load_o(k >> 1, k & 1, v);
                    uint8_t *at = out + 16 * (k & 1) * C::kPitch + 256 * (k >> 1);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 x = *(const float4 *)(inv + 16 * (k & 1) + j);
                        const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            *(__nv_bfloat16 *)(at + (j + y) * C::kPitch) = __float2bfloat16_rn(v[j + y] * f[y]);
                    }
                }
                ok = group_sync();
                if (!ok) break;
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    const int rw = 32 * g + 8 * q4 + k;
                    if (r0 + rw >= R) break;
                    const int tq = (int)W::token(p, r0 + rw), hd = r0 + rw - tq * p.H;
                    uint4 *dst = (uint4 *)(p.o + (size_t)(it.q0 + tq) * p.o_stride + (size_t)hd * KV);
                    const uint4 *from = (const uint4 *)(sQ + rw * C::kPitch);
#pragma unroll
                    for (int x = 0; x < KV / 8; x += 32)
                        if (KV >= 256 || x + lane < KV / 8) dst[x + lane] = from[x + lane];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.item_done);
            left -= take;
            unit += it.chunks - wk.off;
            if (left > 0) wk.next(p);
        }
        if (tid == 32 * kQtSoft0) p.split[cta] = sp;
    }
    tc_fence_before();
    __syncthreads();
    if (ms.abort) {
        if (tid == 0) {
            set_error(p.err, DSPARK_ERR_TIMEOUT);
            for (int s = 0; s < C::kStages; ++s)
                for (int d = 0; d < C::kBars; ++d)
                    if (ms.issued[s][d]) mbar_drain(&ms.full[s][d], ms.issued[s][d] >> 1);
        }
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int KV, int ROPE>
static cudaError_t launch_width(const QaParams &p, int grid, cudaStream_t st) {
    using C = QtCfg<KV, ROPE>;
    constexpr int kSmem = qt_smem_bytes<KV, ROPE>();
    static OncePerDevice once;
    const cudaError_t e =
        once([] { return cudaFuncSetAttribute(qattn_tc_kernel<KV, ROPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return e;
    // the pool as 16-bit elements: boxes of 128 (the rope's: 64) bytes of 64 tokens
    CUtensorMap dims, rope;
    if (!encode_u16_map(&dims, p.codes, (uint64_t)p.n_pages * kQcPage, C::kD, 128, kQcPage)) return cudaErrorInvalidValue;
    if (!C::kWide) rope = dims;
    else if (!encode_u16_map(&rope, p.codes, (uint64_t)p.n_pages * kQcPage, C::kD, 64, kQcPage)) return cudaErrorInvalidValue;
    return launch_pdl(qattn_tc_kernel<KV, ROPE>, dim3(grid), dim3(kQtThreads), (size_t)kSmem, st, dims, rope, p);
}

cudaError_t launch_qattn_tc(const QaParams &p, int kv_lora, int grid, cudaStream_t st) {
    switch (kv_lora) {
        case 512: return launch_width<512, 64>(p, grid, st);
        case 256: return launch_width<256, 32>(p, grid, st);
        case 128: return launch_width<128, 32>(p, grid, st);
        case 64: return launch_width<64, 16>(p, grid, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ds
