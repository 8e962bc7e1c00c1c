// Products of quantised rows with block-scaled weights, many rows (include/dspark.h, calls 12 and 13).
//
//   y[m, n] = sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} cx[m, k] cw[n, k]
//
// A pair of CTAs (cta_group::2) holds a tile of 256 rows x 256 outputs of one matrix (128
// where wider tiles would leave SMs without one), or 128 of the gate's and the same 128 of up's, so that
// the epilogue holds both factors of silu(g) u. Rows are the accumulator's lanes, 128
// a CTA; each CTA loads its rows and half of the outputs' codes. E4M3 codes go to the
// tensor core as they are stored (kind::f8f6f4); a block of 128 k is four MMAs into one of two
// accumulators, from which eight warps add it, times sx sw, to fp32 registers: scales
// are any fp32 numbers, and no sum is longer than 128 terms before it is one of fp32
// FMAs. The accumulator's columns are the first CTA's 64 of the first half, its 64 of
// the second, then the other CTA's, so that a warp's 128 columns have two factors.
//
// Bound: a block's products, followed by its sums (63 % of the tensor pipe's time, 62 % of the issue slots, gated product of
// 2048 rows), and power under a lasting load. Measured: 4000 x 8192 x 7168, bf16 result 175 us (2.7 PFLOP/s), fp32 with a
// residual 223; gated 2900 x 7168 x 2 14336 426 us, for seconds on end 494 at 1.66 GHz. One CTA a tile of 128 x 256
// took 319 us for the product with a residual.
#include <math.h>

#include "per_device.h"
#include "qlinear.h"

namespace ds {

constexpr int kQgSum0 = 4;                         // warps: loads, products, scales, none; then those that sum
constexpr int kQgSums = 8, kQgWide = 512 / kQgSums;  // columns of either half that a warp sums
constexpr int kQgThreads = 32 * (kQgSum0 + kQgSums);  // registers: 168 x 384 = 56 x 128 + 224 x 256
constexpr int kQgRegsIssue = 56, kQgRegsSum = 224, kQgRegs = 168;
constexpr int kQgBox = 128 * 128;                  // bytes: 128 rows or outputs x 128 k
constexpr int kQgStages = 5;
constexpr int kQgSlots = 2;                        // accumulators of 256 columns
constexpr int kQgOut = kQgSums * 4096;             // staged output: 4 KB a summing warp
constexpr int kQgGroup = 8;                        // blocks of k whose scales arrive together

struct QgBars {
    uint64_t full[kQgStages], empty[kQgStages], afull[kQgSlots], aempty[kQgSlots], done;  // full, aempty: the pair's, in its first CTA
    uint64_t sfull[2], sempty[2];                  // scales
    uint64_t group[4];                             // gated: the four warps of 32 rows
    uint32_t tmem;
    volatile int abort;
    uint32_t issued;                               // stages that the producer has requested
    alignas(16) float x[2][kQgGroup][128];         // scales: rows'
    alignas(16) float2 w[2][kQgGroup];             // the two halves'
    int8_t e[2][kQgSums / 4][128];                 // gated, tiles in turn: a row's scale exponent by column group
};
constexpr int kQgSmem = kQgStages * 2 * kQgBox + kQgOut + (int)sizeof(QgBars);
static_assert(kQgSmem <= 232448, "shared memory");

// The pair's forms of what common.cuh and e4m3.cuh have for one CTA.
DS_DEVINL uint32_t first_of_pair(const void *local) {  // the same place in the first CTA's shared memory
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(local)));
    return a;
}
DS_DEVINL void tma_load_2d_pair(void *dst, const CUtensorMap *m, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
DS_DEVINL void tmem_alloc_pair(uint32_t *slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
DS_DEVINL void tmem_dealloc_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
DS_DEVINL void mma_e4m3_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on this barrier of both CTAs once the MMAs issued before are done.
DS_DEVINL void mma_commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
// Without memory ordering at the pair's scope (that is a memory barrier in every block): what the arrival
// publishes are reads of tensor memory, ordered by tcgen05.wait and the tcgen05 fences.
DS_DEVINL void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// HALVES: columns of the tile / 128; gated: 2, the gate's and up's
template <bool GATED, int HALVES, bool ADD>
__global__ void __launch_bounds__(kQgThreads, 1)
    qgemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                 const __grid_constant__ CUtensorMap tm_w1, const QlParams p, int tiles_m, int tiles) {
    constexpr int kBoxW = 64 * 128, kStage = kQgBox + HALVES * kBoxW;  // a CTA's rows, its 64 of each half's outputs
    constexpr int kStep = GATED ? 128 : 128 * HALVES;
    static_assert(!GATED || HALVES == 2, "gate and up");
    extern __shared__ __align__(1024) uint8_t qg_smem[];
    uint8_t *sOut = qg_smem + kQgStages * 2 * kQgBox;
    QgBars &ms = *(QgBars *)(sOut + kQgOut);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &ms.abort;
    const int KB = p.KB, rank = (int)cluster_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (tid == 0) {
        for (int s = 0; s < kQgStages; ++s) {
            mbar_init(&ms.full[s], 1);
            mbar_init(&ms.empty[s], 1);
        }
        for (int s = 0; s < kQgSlots; ++s) {
            mbar_init(&ms.afull[s], 1);
            mbar_init(&ms.aempty[s], 2 * kQgSums);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ms.sfull[s], 32);
            mbar_init(&ms.sempty[s], kQgSums);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&ms.group[i], kQgSums / 4);
        mbar_init(&ms.done, 1);
        ms.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w0);
        if (GATED) tma_prefetch_desc(&tm_w1);
    }
    __syncthreads();  // (the cluster's barrier wants whole warps)
    cluster_sync();
    // Tensor memory is taken once the kernels before have ended, and the kernel behind is let in once it is taken: of
    // two that share an SM, neither holds what the other waits for. The producer needs none and goes ahead.
    pdl_wait();
    if (warp == 1) {
        tmem_alloc_pair(&ms.tmem, 512);
        pdl_trigger();
    }
    uint32_t tmem = 0;
    if (warp != 0) {
        tc_fence_before();
        named_bar_sync(7, kQgThreads - 32);
        tc_fence_after();
        tmem = ms.tmem;
    }

    if (warp < kQgSum0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQgRegsIssue));
        if (warp == 0) {
            if (ql_elect()) {
                uint32_t u = 0;
                bool ok = true;
                for (int t = pair; t < tiles && ok; t += pairs) {
                    const int m0 = t % tiles_m * 256 + 128 * rank, n0 = t / tiles_m * kStep + 64 * rank;
                    for (int kb = 0; kb < KB; ++kb, ++u) {
                        const uint32_t s = u % kQgStages, par = (u / kQgStages) & 1;
                        if (u >= kQgStages && !mbar_wait_bounded(&ms.empty[s], par ^ 1, abort)) {
                            ok = false;
                            break;
                        }
                        uint8_t *to = qg_smem + s * kStage;
                        const uint32_t bar = first_of_pair(&ms.full[s]);
                        if (rank == 0) mbar_arrive_expect_tx(&ms.full[s], 2 * kStage);
                        // 16-bit elements: 64 a box row
                        tma_load_2d_pair(to, &tm_x, kb * 64, m0, bar);
                        tma_load_2d_pair(to + kQgBox, &tm_w0, kb * 64, n0, bar);
                        if (HALVES == 2) tma_load_2d_pair(to + kQgBox + kBoxW, GATED ? &tm_w1 : &tm_w0, kb * 64, n0 + (GATED ? 0 : 128), bar);
                    }
                }
                ms.issued = u;
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0 && ql_elect()) {
                const uint32_t lo = sdesc_lo(smem_u32(qg_smem));
                constexpr uint32_t hi = sdesc_hi(1024, 2), id = idesc_e4m3_f32(256, 128 * HALVES);
                uint32_t u = 0;
                bool ok = true;
                for (int t = pair; t < tiles && ok; t += pairs)
                    for (int kb = 0; kb < KB; ++kb, ++u) {
                        const uint32_t s = u % kQgStages;
                        ok = mbar_wait_bounded(&ms.full[s], (u / kQgStages) & 1, abort);
                        const uint32_t a = lo + s * (kStage >> 4), b = a + (kQgBox >> 4);
                        ok = ok && (u < kQgSlots || mbar_wait_bounded(&ms.aempty[u % kQgSlots], ((u / kQgSlots) & 1) ^ 1, abort));
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_e4m3_pair(tmem + 256 * (u % kQgSlots), (uint64_t)hi << 32 | (a + 2 * k), (uint64_t)hi << 32 | (b + 2 * k), id, k > 0);
                        mma_commit_pair(&ms.afull[u % kQgSlots]);
                        mma_commit_pair(&ms.empty[s]);
                    }
                mma_commit_pair(&ms.done);
                ql_drain(&ms.done, 0);
            }
            __syncwarp();
        } else if (warp == 2) {
            // scales, a group of blocks ahead: a load's latency would otherwise stand in every block of the summing warps
            const int nb = (p.N + kQlBlock - 1) / kQlBlock;
            uint32_t g = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const int m0 = t % tiles_m * 256 + 128 * rank, b0 = t / tiles_m * kStep / kQlBlock;
                const float *s0 = p.sw[0] + (size_t)b0 * KB;
                const float *s1 = GATED ? p.sw[1] + (size_t)b0 * KB : s0 + (b0 + 1 < nb ? KB : 0);
                const float *s = lane & 1 ? s1 : s0;
                for (int kb = 0; kb < KB; kb += kQgGroup, ++g) {
                    const uint32_t at = g & 1;
                    ok = g < 2 || ql_warp_wait(&ms.sempty[at], ((g >> 1) & 1) ^ 1, abort);
                    if (!ok) break;
                    const int n = min(kQgGroup, KB - kb);
                    for (int j = 0; j < n; ++j) {
                        const float *x = p.sx + (size_t)(kb + j) * p.sx_stride;
#pragma unroll
                        for (int i = 0; i < 4; ++i) cp_async4(&ms.x[at][j][lane + 32 * i], x + min(m0 + lane + 32 * i, p.M - 1));
                    }
                    if ((lane >> 1) < n) cp_async4((float *)&ms.w[at][lane >> 1] + (lane & 1), s + kb + (lane >> 1));
                    cp_async_arrive(&ms.sfull[at]);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        // Registers are taken back behind the barrier, before which the summing warps have given theirs up: a warp that is done
        // at once (one has nothing to do) could otherwise take again what they have not got yet, and nothing would end their wait.
        __syncwarp();
        tc_fence_before();
        named_bar_sync(6, kQgThreads);
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQgRegs));
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQgRegsSum));
        const int q = warp & 3, h = (warp - kQgSum0) >> 2;  // lanes 32 q .., columns kQgWide h .. of each half
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 64 * HALVES * h;
        uint8_t *out = sOut + (warp - kQgSum0) * 4096;
        uint32_t u = 0, g = 0, count = 0;
        bool ok = true;
        for (int t = pair; t < tiles && ok; t += pairs, ++count) {
            const int m0 = t % tiles_m * 256 + 128 * rank + 32 * q, n0 = t / tiles_m * kStep, row = m0 + lane;
            float acc[kQgWide * HALVES];  // columns kQgWide h .. of the first half, then of the second
#pragma unroll
            for (int i = 0; i < kQgWide * HALVES; ++i) acc[i] = 0.f;
            if (ADD && row < p.M) {
                // the tile's share of `add` on its way into L2 while the products are formed
#pragma unroll
                for (int c = 0; c < HALVES; ++c) {
                    const int n = n0 + 128 * c + kQgWide * h;
                    if (n < p.N) prefetch_l2_bulk(p.add + (size_t)row * p.add_stride + n, 4 * min(kQgWide, p.N - n));
                }
            }
            for (int kb = 0; kb < KB; ++kb, ++u) {
                const int j = kb % kQgGroup;
                if (j == 0) {
                    ok = ql_warp_wait(&ms.sfull[g & 1], (g >> 1) & 1, abort);
                    if (!ok) break;
                }
                const float x = ms.x[g & 1][j][32 * q + lane];
                const float2 w = ms.w[g & 1][j];
                const float f0 = x * w.x, f1 = x * w.y;
                if (j == kQgGroup - 1 || kb == KB - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.sempty[g & 1]);
                    __syncwarp();
                    ++g;
                }
                ok = ql_warp_wait(&ms.afull[u & 1], (u >> 1) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = tl + 256 * (u & 1);
#pragma unroll
                for (int c = 0; c < 2 * HALVES; ++c) {
                    float v[32];
                    tmem_ld32_now(at + 32 * c, v);
                    if (c + 1 == 2 * HALVES) {  // read: its products may be replaced
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(first_of_pair(&ms.aempty[u & 1]));
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) acc[32 * c + i] = __fmaf_rn(v[i], c < 2 ? f0 : f1, acc[32 * c + i]);
                }
            }
            if (!ok) break;
            if constexpr (GATED) {
                float v[kQgWide];
                uint32_t mx = 0;
                bool far = false;
#pragma unroll
                for (int i = 0; i < kQgWide; ++i) {
                    v[i] = ql_gate_near(acc[i], acc[kQgWide * (HALVES - 1) + i]);
                    far |= acc[i] < kQlFar;
                }
                // rare: one test for all of a warp's gates (a choice for each: 424 us for 417, 2900 x 7168 x 2 14336)
                if (__any_sync(~0u, far)) {
#pragma unroll
                    for (int i = 0; i < kQgWide; ++i)
                        if (acc[i] < kQlFar) v[i] = ql_gate_far(acc[i], acc[kQgWide * (HALVES - 1) + i]);
                }
#pragma unroll
                for (int i = 0; i < kQgWide; ++i) {
                    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
                    if (a < 0x7f800000u) mx = max(mx, a);
                    else v[i] = __uint_as_float(0x7fffffffu);
                }
                int e = ql_exponent(mx);  // (of the largest: the largest of the groups')
                ms.e[count & 1][h][32 * q + lane] = (int8_t)e;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.group[q]);
                ok = ql_warp_wait(&ms.group[q], count & 1, abort);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < kQgSums / 4; ++i) e = max(e, (int)ms.e[count & 1][i][32 * q + lane]);
                const float inv = qc_pow2(-e);
                if (h == 0 && row < p.M) p.sh[(size_t)(n0 / kQlBlock) * p.sh_stride + row] = qc_pow2(e);
                // 64 bytes a row, 16-byte pieces swizzled; then four lanes a row
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = ql_e4m3x2(v[16 * c + 4 * i] * inv, v[16 * c + 4 * i + 1] * inv) |
                               ql_e4m3x2(v[16 * c + 4 * i + 2] * inv, v[16 * c + 4 * i + 3] * inv) << 16;
                    *(uint4 *)(out + lane * 64 + ((c ^ (lane >> 1)) & 3) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
                const int n = n0 + 64 * h + 16 * (lane & 3);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + (lane >> 2);
                    const uint4 w = *(const uint4 *)(out + r * 64 + ((lane ^ (r >> 1)) & 3) * 16);
                    if (m0 + r < p.M && n < p.N) *(uint4 *)(p.h + (size_t)(m0 + r) * p.N + n) = w;
                }
                __syncwarp();
            } else {
                // 32 columns at a time through shared memory: 128 bytes a row, 16-byte pieces swizzled; then eight lanes a
                // row, whose share of `add` is requested two steps ahead
                constexpr int kPer = kQgWide / 32;
                const int r0 = lane >> 3, left = p.M - m0;
                auto column = [&](int c) { return n0 + 128 * (c / kPer) + kQgWide * h + 32 * (c % kPer) + 4 * (lane & 7); };
                float4 a[2][8];
                auto fetch = [&](int c) {
                    const int n = column(c);
                    const float *at = p.add + (size_t)(m0 + r0) * p.add_stride + n;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        a[c & 1][i] = 4 * i + r0 < left && n < p.N ? __ldcs((const float4 *)(at + (size_t)(4 * i) * p.add_stride)) : make_float4(0.f, 0.f, 0.f, 0.f);
                };
                if (ADD) {
                    fetch(0);
                    if (kPer * HALVES > 1) fetch(1);
                }
#pragma unroll
                for (int c = 0; c < kPer * HALVES; ++c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float *v = acc + 32 * c + 4 * i;
                        *(float4 *)(out + lane * 128 + ((i ^ lane) & 7) * 16) = make_float4(v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
                    const int n = column(c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4 v = *(const float4 *)(out + (4 * i + r0) * 128 + ((lane ^ (4 * i + r0)) & 7) * 16);
                        if (ADD) {
                            v.x += a[c & 1][i].x;
                            v.y += a[c & 1][i].y;
                            v.z += a[c & 1][i].z;
                            v.w += a[c & 1][i].w;
                        }
                        if (4 * i + r0 < left && n < p.N) {
                            const size_t to = (size_t)(m0 + 4 * i + r0) * p.y_stride + n;
                            if (p.y_fp32) {
                                __stcs((float4 *)((float *)p.y + to), v);
                            } else {
                                const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
                                *(uint2 *)((__nv_bfloat16 *)p.y + to) = make_uint2(*(const uint32_t *)&lo, *(const uint32_t *)&hi);
                            }
                        }
                    }
                    if (ADD && c + 2 < kPer * HALVES) fetch(c + 2);
                    __syncwarp();
                }
            }
        }
        // all warps leave with their share of the launch again
        __syncwarp();
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQgRegs));
        tc_fence_before();
        named_bar_sync(6, kQgThreads);
    }
    if (tid == 0) {
        // Every arrival that the products' commits, or the other CTA's warps, send to this CTA has come: one that is still on
        // its way when the CTA has left would land in memory that is no longer its own.
        ql_drain(&ms.done, 0);
        for (uint32_t u = ms.issued > kQgStages ? ms.issued - kQgStages : 0; !ms.abort && u < ms.issued; ++u)
            ql_drain(&ms.empty[u % kQgStages], (u / kQgStages) & 1);
        for (uint32_t u = ms.issued > kQgSlots ? ms.issued - kQgSlots : 0; rank == 0 && !ms.abort && u < ms.issued; ++u)
            ql_drain(&ms.aempty[u % kQgSlots], (u / kQgSlots) & 1);  // and every one of the other CTA's
        if (ms.abort) {  // no copy outlives the pair
            for (uint32_t u = ms.issued > kQgStages ? ms.issued - kQgStages : 0; rank == 0 && u < ms.issued; ++u)
                ql_drain(&ms.full[u % kQgStages], (u / kQgStages) & 1);
            set_error(p.err, DSPARK_ERR_TIMEOUT);
        }
    }
    __syncwarp();
    cluster_sync();  // the pair's products and barriers are in either CTA's memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

template <bool GATED, int HALVES, bool ADD>
static QlPlan plan(const QlParams &p) {
    static OncePerDevice once;
    static ClusterRoom<decltype(&qgemm_kernel<GATED, HALVES, ADD>)> room;
    constexpr int kStep = GATED ? 128 : 128 * HALVES;
    QlPlan r = {HALVES, (long long)((p.M + 255) / 256) * ((p.N + kStep - 1) / kStep), 1, 0.f, cudaSuccess};
    r.error = once([] {
        return cudaFuncSetAttribute(qgemm_kernel<GATED, HALVES, ADD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQgSmem);
    });
    if (r.error != cudaSuccess) return r;
    r.error = room(qgemm_kernel<GATED, HALVES, ADD>, 2, kQgThreads, kQgSmem, &r.room);
    if (r.error == cudaSuccess && r.room < 1) r.error = cudaErrorLaunchOutOfResources;  // no pair fits this device
    if (r.error != cudaSuccess) return r;
    // us a block of k, from whole calls. Tiles of 256 against 128 outputs: 2112 x 7168, 256 rows 28.8 and 20.2, 4000 rows 54.9
    // and 65.7; 7168 x 14336, 512 rows 51.6 and 66.4; 12288 x 1536, 512 rows 20.3 and 18.2
    r.time = 4.f + (float)((r.tiles + r.room - 1) / r.room) * (1.f + p.KB * (HALVES == 2 ? 0.47f : 0.26f));
    return r;
}

template <bool GATED, int HALVES, bool ADD>
static cudaError_t launch(const QlParams &p, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                          const QlPlan &plan, cudaStream_t st) {
    CUtensorMap mx, m0, m1;
    if (!encode_u16_map(&mx, x.codes, x.rows, x.k, 128, 128) || !encode_u16_map(&m0, w0.codes, w0.n, w0.k, 128, 64))
        return cudaErrorInvalidValue;
    m1 = m0;
    if (GATED && !encode_u16_map(&m1, w1.codes, w1.n, w1.k, 128, 64)) return cudaErrorInvalidValue;
    if (plan.tiles >= 1ll << 30) return cudaErrorInvalidValue;
    const int pairs = (int)(plan.tiles < plan.room ? plan.tiles : plan.room);
    return launch_pdl_cluster(qgemm_kernel<GATED, HALVES, ADD>, dim3(2 * pairs), dim3(kQgThreads), (size_t)kQgSmem, st, 2, mx, m0, m1, p,
                              (p.M + 255) / 256, (int)plan.tiles);
}

QlPlan plan_qgemm(const QlParams &p, bool gated) {
    if (gated) return plan<true, 2, false>(p);
    const QlPlan wide = p.add ? plan<false, 2, true>(p) : plan<false, 2, false>(p);
    if (wide.error != cudaSuccess) return wide;
    const QlPlan half = p.add ? plan<false, 1, true>(p) : plan<false, 1, false>(p);
    return half.error != cudaSuccess || half.time < wide.time ? half : wide;
}
cudaError_t launch_qgemm(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                         const QlPlan &plan, cudaStream_t st) {
    if (gated) return launch<true, 2, false>(p, x, w0, w1, plan, st);
    if (plan.split == 1) return p.add ? launch<false, 1, true>(p, x, w0, w1, plan, st) : launch<false, 1, false>(p, x, w0, w1, plan, st);
    return p.add ? launch<false, 2, true>(p, x, w0, w1, plan, st) : launch<false, 2, false>(p, x, w0, w1, plan, st);
}

}  // namespace ds
