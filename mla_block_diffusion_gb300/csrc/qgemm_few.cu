// Products of few quantised rows (up to 64) with block-scaled weights (include/dspark.h, calls 12 and 13).
//
// The same sums as in qgemm.cu with outputs on the accumulator's 128 lanes and the
// rows (padded to NT = 16, 32 or 64) as its columns: the weights stream past the rows
// once, one CTA an SM, through a ring of 170 to 200 KB (128 to 176 KB of it weights). A tile is 128 outputs (gated: 128 of gate and
// the same 128 of up, which have a scale in common). With fewer tiles than SMs, the up to eight
// CTAs of a cluster share a tile's blocks of k, add their sums in rank order through
// distributed shared memory, and each finishes some of the rows: nothing goes through
// global memory and a result does not depend on timing.
//
// Bound: HBM (one byte a weight), if a block of 128 k does not hold up the ring. Its sums
// are a dependent chain (commit, wake, read, multiply, release), so
// four groups of four warps take blocks in turn (gated: two groups for each matrix), each
// with accumulators of its own in tensor memory and sums of its own in registers, which are
// added in order at the end.
// Measured (graphs, weights in turn): one row, 35840 x 7168 43.8 us (5.9 TB/s), gated 7168 x 2 14336 35.5 (5.8 TB/s),
// 7168 x 2112 7.4; 64 rows 48.3, 39.9 and 10.0.
#include <math.h>

#include "per_device.h"
#include "qlinear.h"

namespace ds {

constexpr int kQfSum0 = 4, kQfGroups = 4;                   // warps: loads, products, scales, none; then four groups of four that sum
constexpr int kQfThreads = 32 * (kQfSum0 + 4 * kQfGroups);  // registers: 96 x 640 >= 56 x 128 + 104 x 512
constexpr int kQfRegsIssue = 56, kQfRegsSum = 104, kQfRegs = 96;
constexpr int kQfMaxStages = 12;
constexpr int kQfMaxSplit = 8;                              // CTAs of a cluster
constexpr int kQfWindow = 8, kQfWindows = 4;                // blocks of k whose scales arrive together, and such windows in shared memory
constexpr int kQfRing = 200 * 1024;                         // stages: at most

template <int NT, bool GATED>
struct QfCfg {
    static constexpr int kMats = GATED ? 2 : 1, kTurns = kQfGroups / kMats;  // groups that take a matrix's blocks in turn
    static constexpr int kSlots = 8 / kMats;                                  // blocks in tensor memory
    static constexpr int kCols = 8 * NT;
    static constexpr int kStage = NT * 128 + kMats * 128 * 128;               // rows, then weights
    static constexpr int kStages = kQfRing / kStage < kQfMaxStages ? kQfRing / kStage : kQfMaxStages;
    struct Bars {
        uint64_t full[kStages], empty[kStages], afull[kSlots], aempty[kSlots], sfull[kQfWindows], sempty[kQfWindows], done;
        uint32_t tmem, issued;
        volatile int abort;
        alignas(16) float x[kQfWindows][kQfWindow][NT];
        alignas(16) float w[kQfWindows][kQfWindow][2];
    };
    static constexpr int kSmem = kStages * kStage + (int)sizeof(Bars);
    static_assert(kSmem <= 232448, "shared memory");
    static_assert((kQfGroups + kMats) * NT * 128 * 4 <= kStages * kStage, "the groups' sums, and theirs, in the stages' place");
    static_assert(kCols >= 32 && kCols <= 512 && kSlots % kTurns == 0, "tensor memory");
};

// 16 bytes of the same place in the shared memory of CTA `rank` of the cluster.
DS_DEVINL float4 ld_peer_f4(const float *local, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
DS_DEVINL void add4(float4 &a, const float4 &b) {
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(kQfThreads, 1)
    qgemm_few_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                     const __grid_constant__ CUtensorMap tm_w1, const QlParams p, int split) {
    using C = QfCfg<NT, GATED>;
    using Bars = typename C::Bars;
    extern __shared__ __align__(1024) uint8_t qf_smem[];
    Bars &ms = *(Bars *)(qf_smem + C::kStages * C::kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &ms.abort;
    const int rank = blockIdx.x % split, tile = blockIdx.x / split;
    const int n0 = tile * 128, rows = p.M;
    const int k0 = (int)((long long)rank * p.KB / split), KB = (int)((long long)(rank + 1) * p.KB / split) - k0;  // this CTA's blocks
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&ms.full[s], 1);
            mbar_init(&ms.empty[s], 1);
        }
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&ms.afull[s], 1);
            mbar_init(&ms.aempty[s], 4 * C::kMats);
        }
        for (int s = 0; s < kQfWindows; ++s) {
            mbar_init(&ms.sfull[s], 32);
            mbar_init(&ms.sempty[s], 4 * kQfGroups);
        }
        mbar_init(&ms.done, 1);
        ms.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w0);
        if (GATED) tma_prefetch_desc(&tm_w1);
    }
    __syncthreads();
    // Tensor memory is taken once the kernels before have ended, and the kernel behind is let in once it is taken: of
    // two that share an SM, neither holds what the other waits for. The producer needs none and goes ahead.
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(&ms.tmem, C::kCols);
        pdl_trigger();
    }
    uint32_t tmem = 0;
    if (warp != 0) {
        tc_fence_before();
        named_bar_sync(7, kQfThreads - 32);
        tc_fence_after();
        tmem = ms.tmem;
    }

    if (warp < kQfSum0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQfRegsIssue));
        if (warp == 0) {
            if (ql_elect()) {
                int u = 0;
                for (; u < KB; ++u) {
                    const int s = u % C::kStages;
                    if (u >= C::kStages && !mbar_wait_bounded(&ms.empty[s], ((u / C::kStages) & 1) ^ 1, abort)) break;
                    uint8_t *to = qf_smem + s * C::kStage;
                    mbar_arrive_expect_tx(&ms.full[s], C::kStage);
                    // 16-bit elements: 64 a box row
                    tma_load_2d(to + NT * 128, &tm_w0, (k0 + u) * 64, n0, &ms.full[s]);
                    if (GATED) tma_load_2d(to + NT * 128 + 128 * 128, &tm_w1, (k0 + u) * 64, n0, &ms.full[s]);
                    tma_load_2d(to, &tm_x, (k0 + u) * 64, 0, &ms.full[s]);
                }
                ms.issued = u;
            }
            __syncwarp();
        } else if (warp == 1) {
            if (ql_elect()) {
                const uint32_t lo = sdesc_lo(smem_u32(qf_smem));
                constexpr uint32_t hi = sdesc_hi(1024, 2), id = idesc_e4m3_f32(128, NT);
                int u = 0;
                for (; u < KB; ++u) {
                    const uint32_t s = u % C::kStages, slot = u % C::kSlots;
                    if (!mbar_wait_bounded(&ms.full[s], (u / C::kStages) & 1, abort)) break;
                    if (u >= C::kSlots && !mbar_wait_bounded(&ms.aempty[slot], ((u / C::kSlots) & 1) ^ 1, abort)) break;
                    tc_fence_after();
                    const uint32_t x = lo + s * (C::kStage >> 4), w = x + (NT * 128 >> 4);
#pragma unroll
                    for (int i = 0; i < C::kMats; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_e4m3(tmem + (slot * C::kMats + i) * NT, (uint64_t)hi << 32 | (w + i * 1024 + 2 * k), (uint64_t)hi << 32 | (x + 2 * k), id,
                                     k > 0);
                    // Only of a stage that is filled again, for which the producer waits: an arrival that is still on its way
                    // when the CTA has left would land in memory that is no longer its own.
                    if (u + C::kStages < KB) mma_commit(&ms.empty[s]);
                    mma_commit(&ms.afull[slot]);
                }
                mma_commit(&ms.done);
                ql_drain(&ms.done, 0);
                if (u < KB) {  // given up: the others may no longer wait for what was sent
                    for (int v = max(0, u - C::kStages); v < min(u, KB - C::kStages); ++v) ql_drain(&ms.empty[v % C::kStages], (v / C::kStages) & 1);
                    for (int v = max(0, u - C::kSlots); v < u; ++v) ql_drain(&ms.afull[v % C::kSlots], (v / C::kSlots) & 1);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // scales, some windows ahead
            const size_t block = (size_t)(n0 / kQlBlock) * p.KB + k0;
            const float *sw = (lane & 1 ? p.sw[1] : p.sw[0]) + block;
            for (int kb = 0, g = 0; kb < KB; kb += kQfWindow, ++g) {
                const uint32_t at = g % kQfWindows;
                if (g >= kQfWindows && !ql_warp_wait(&ms.sempty[at], ((g / kQfWindows) & 1) ^ 1, abort)) break;
                const int n = min(kQfWindow, KB - kb);
                for (int j = 0; j < n; ++j)
#pragma unroll
                    for (int i = 0; i < NT; i += 32) {
                        const int m = i + lane;
                        if (m < NT) cp_async4(&ms.x[at][j][m], p.sx + (size_t)(k0 + kb + j) * p.sx_stride + min(m, rows - 1));
                    }
                if ((lane >> 1) < n) cp_async4(&ms.w[at][lane >> 1][lane & 1], sw + kb + (lane >> 1));
                cp_async_arrive(&ms.sfull[at]);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        // Registers are taken back behind the barrier, before which the summing warps have given theirs up: a warp that is done
        // at once (one has nothing to do) could otherwise take again what they have not got yet, and nothing would end their wait.
        __syncwarp();
        tc_fence_before();
        named_bar_sync(6, kQfThreads);
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQfRegs));
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQfRegsSum));
        const int q = warp & 3, group = (warp - kQfSum0) >> 2, mat = group / C::kTurns, turn = group % C::kTurns;
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + mat * NT;
        float acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = 0.f;
        bool ok = true;
        for (int kb = 0, g = 0; kb < KB && ok; kb += kQfWindow, ++g) {
            const uint32_t at = g % kQfWindows;
            ok = ql_warp_wait(&ms.sfull[at], (g / kQfWindows) & 1, abort);
            const int n = min(kQfWindow, KB - kb);
#pragma unroll 1
            for (int j = turn; j < n && ok; j += C::kTurns) {  // (a window is a multiple of the turns)
                const int u = kb + j;
                const uint32_t slot = u % C::kSlots;
                ok = ql_warp_wait(&ms.afull[slot], (u / C::kSlots) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const float w = ms.w[at][j][mat];
#pragma unroll
                for (int c = 0; c < NT; c += 16) {
                    float v[16];
                    tmem_ld16_now(tl + slot * (C::kMats * NT) + c, v);
                    if (c + 16 == NT) {  // read: its products may be replaced
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.aempty[slot]);
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 x = *(const float4 *)&ms.x[at][j][c + i];
                        acc[c + i] = __fmaf_rn(v[i], x.x * w, acc[c + i]);
                        acc[c + i + 1] = __fmaf_rn(v[i + 1], x.y * w, acc[c + i + 1]);
                        acc[c + i + 2] = __fmaf_rn(v[i + 2], x.z * w, acc[c + i + 2]);
                        acc[c + i + 3] = __fmaf_rn(v[i + 3], x.w * w, acc[c + i + 3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.sempty[at]);
        }
        // Sums [group, row, output] in the stages' place once every product is done: a group's last block need not be the
        // last of all.
        if (ok) ok = ql_warp_wait(&ms.done, 0, abort);
        float *part = (float *)qf_smem + group * (NT * 128) + 32 * q + lane;
        if (ok) {
#pragma unroll
            for (int i = 0; i < NT; ++i) part[i * 128] = acc[i];
        }
        // all warps finish the tile together, each with its share of the launch again
        __syncwarp();
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQfRegs));
        tc_fence_before();
        named_bar_sync(6, kQfThreads);
    }
    // four outputs of a row: of this CTA's groups, added in order
    auto own = [&](int mat, int row, int c) {
        const float *at = (const float *)qf_smem + (mat * C::kTurns * NT + row) * 128 + c;
        float4 v = *(const float4 *)at;
#pragma unroll
        for (int i = 1; i < C::kTurns; ++i) add4(v, *(const float4 *)(at + i * NT * 128));
        return v;
    };
    float *sums = (float *)qf_smem + kQfGroups * NT * 128;  // [matrix, row, output] of this CTA
    if (split > 1) {
        for (int i = tid; i < C::kMats * rows * 32; i += kQfThreads) {
            const int mat = i / (rows * 32), row = i / 32 % rows, c = 4 * (i & 31);
            *(float4 *)(sums + (mat * NT + row) * 128 + c) = own(mat, row, c);
        }
        __syncthreads();
        cluster_sync();
    }
    auto total = [&](int mat, int row, int c) {
        if (split == 1) return own(mat, row, c);
        const float *at = sums + (mat * NT + row) * 128 + c;
        float4 o[kQfMaxSplit];
#pragma unroll
        for (int i = 0; i < kQfMaxSplit; ++i)
            if (i < split) o[i] = ld_peer_f4(at, i);
#pragma unroll
        for (int i = 1; i < kQfMaxSplit; ++i)
            if (i < split) add4(o[0], o[i]);
        return o[0];
    };
    // row i is finished by CTA i % split
    {
        // a warp a row, four outputs a lane
        for (int m = rank + split * warp; m < rows; m += split * (kQfThreads / 32)) {
            const int n = n0 + 4 * lane;
            float4 v = total(0, m, 4 * lane);
            if constexpr (GATED) {
                const float4 u = total(1, m, 4 * lane);
                float h[4] = {ql_gate(v.x, u.x), ql_gate(v.y, u.y), ql_gate(v.z, u.z), ql_gate(v.w, u.w)};
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = __float_as_uint(h[i]) & 0x7fffffffu;
                    if (a < 0x7f800000u) mx = max(mx, a);
                    else h[i] = __uint_as_float(0x7fffffffu);
                }
                const int e = ql_exponent(__reduce_max_sync(~0u, mx));
                const float inv = qc_pow2(-e);
                if (n < p.N)
                    *(uint32_t *)(p.h + (size_t)m * p.N + n) = ql_e4m3x2(h[0] * inv, h[1] * inv) | ql_e4m3x2(h[2] * inv, h[3] * inv) << 16;
                if (lane == 0) p.sh[(size_t)(n0 / kQlBlock) * p.sh_stride + m] = qc_pow2(e);
            } else if (n < p.N) {
                if (p.add) add4(v, *(const float4 *)(p.add + (size_t)m * p.add_stride + n));
                if (p.y_fp32) {
                    *(float4 *)((float *)p.y + (size_t)m * p.y_stride + n) = v;
                } else {
                    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
                    *(uint2 *)((__nv_bfloat16 *)p.y + (size_t)m * p.y_stride + n) = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
                }
            }
        }
    }
    __syncthreads();
    if (split > 1) cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
    if (tid == 0 && ms.abort) {  // no copy outlives the CTA
        for (int u = max(0, (int)ms.issued - C::kStages); u < (int)ms.issued; ++u) mbar_drain(&ms.full[u % C::kStages], (u / C::kStages) & 1);
        set_error(p.err, DSPARK_ERR_TIMEOUT);
    }
}

template <int NT, bool GATED>
static QlPlan plan(const QlParams &p) {
    using C = QfCfg<NT, GATED>;
    static OncePerDevice once;
    static ClusterRoom<decltype(&qgemm_few_kernel<NT, GATED>)> room;
    QlPlan r = {1, (p.N + 127) / 128, 1, 0.f, cudaSuccess};
    r.error = once([] {
        return cudaFuncSetAttribute(qgemm_few_kernel<NT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    });
    if (r.error != cudaSuccess) return r;
    // The largest cluster that leaves all tiles on the device at once and every CTA three blocks; none below 12 blocks, where
    // the clusters' sum costs more than it saves. us, whole and in clusters, 1 and 64 rows: 1024 outputs x 512 inputs 3.2 and
    // 4.9 against 3.8 and 6.2; x 1024 3.9 and 5.8 against (of two) 4.2 and 6.8; x 1536 4.7 and 6.6 against (of four) 3.9
    // and 6.5; 576 x 14336 25.0 and 29.5 against (of eight) 6.6 and 9.2.
    for (int s = 2, fit; s <= kQfMaxSplit && p.KB >= 12 && s <= p.KB / 3; ++s) {
        r.error = room(qgemm_few_kernel<NT, GATED>, s, kQfThreads, C::kSmem, &fit);
        if (r.error != cudaSuccess) return r;
        if (r.tiles <= fit) r.split = s;
    }
    return r;
}

template <int NT, bool GATED>
static cudaError_t launch(const QlParams &p, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                          const QlPlan &plan, cudaStream_t st) {
    using C = QfCfg<NT, GATED>;
    CUtensorMap mx, m0, m1;
    if (!encode_u16_map(&mx, x.codes, x.rows, x.k, 128, NT) || !encode_u16_map(&m0, w0.codes, w0.n, w0.k, 128, 128))
        return cudaErrorInvalidValue;
    m1 = m0;
    if (GATED && !encode_u16_map(&m1, w1.codes, w1.n, w1.k, 128, 128)) return cudaErrorInvalidValue;
    return launch_pdl_cluster(qgemm_few_kernel<NT, GATED>, dim3((unsigned)(plan.tiles * plan.split)), dim3(kQfThreads), (size_t)C::kSmem, st,
                              plan.split, mx, m0, m1, p, plan.split);
}

QlPlan plan_qgemm_few(const QlParams &p, bool gated) {
    if (p.M <= 16) return gated ? plan<16, true>(p) : plan<16, false>(p);
    if (p.M <= 32) return gated ? plan<32, true>(p) : plan<32, false>(p);
    return gated ? plan<64, true>(p) : plan<64, false>(p);
}
cudaError_t launch_qgemm_few(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0,
                             const dspark_qweight_t &w1, const QlPlan &plan, cudaStream_t st) {
    if (p.M <= 16) return gated ? launch<16, true>(p, x, w0, w1, plan, st) : launch<16, false>(p, x, w0, w1, plan, st);
    if (p.M <= 32) return gated ? launch<32, true>(p, x, w0, w1, plan, st) : launch<32, false>(p, x, w0, w1, plan, st);
    return gated ? launch<64, true>(p, x, w0, w1, plan, st) : launch<64, false>(p, x, w0, w1, plan, st);
}

}  // namespace ds
