// Products of few quantised rows (up to 64) with block-scaled weights (include/dspark.h, calls 12 and 13).
//
// The same sums as in qgemm.cu with outputs on the accumulator's 128 lanes and the
// rows (padded to NT = 16, 32 or 64) as its columns: the weights stream past the rows
// once, one CTA an SM, through a ring of 200 KB. A CTA takes 128 outputs (gated: 64 of gate and
// the same 64 of up) and a share of the blocks of k; the CTAs of a cluster share a tile's
// blocks (gated: and the two halves of 128 outputs, which have a scale in common), add
// their partial sums in rank order through distributed shared memory, and each finishes
// some of the rows, so nothing goes through global memory and a result does not depend on
// timing. Bound: HBM (one byte a weight). The cluster is the largest of up to 8 CTAs that
// leaves all tiles on the device at once.
#include <math.h>

#include "per_device.h"
#include "qlinear.h"

namespace ds {

constexpr int kQfWindow = 16;     // blocks of k whose factors lie in shared memory at a time
constexpr int kQfMaxCluster = 8;

template <int NT>
struct QfCfg {
    static constexpr int kX = 128 * 128;                                // weights, then rows
    static constexpr int kStage = kX + NT * 128;
    static constexpr int kFactors = kQfWindow * NT * 4;
    static constexpr int kMats = 2;                                     // factors of gate and of up lie apart
    static constexpr int kStages = (208 * 1024 - kMats * kFactors) / kStage;
    static constexpr int kSlots = 8, kCols = kSlots * NT;
    static constexpr int kThreads = 64 + 128;
    static_assert(kStages >= 3 && NT * 128 * 4 <= kStages * kStage, "shared memory");
    static_assert(kCols >= 32 && kCols <= 512 && (kCols & (kCols - 1)) == 0, "tensor memory");
    struct Bars {
        uint64_t full[kStages], empty[kStages], afull[kSlots], aempty[kSlots], done;
        uint32_t tmem, issued;
        volatile int abort;
    };
    static constexpr int kSmem = kStages * kStage + kMats * kFactors + (int)sizeof(Bars);
    static_assert(kSmem <= 232448 && kSmem > 116 * 1024, "shared memory: one CTA an SM");
};

// 16 bytes of the same place in the shared memory of CTA `rank` of the cluster.
DS_DEVINL float4 ld_peer_f4(const float *local, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

template <int NT, bool GATED>
__global__ void __launch_bounds__(QfCfg<NT>::kThreads, 1)
    qgemm_few_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                     const __grid_constant__ CUtensorMap tm_w1, const QlParams p, int split) {
    using C = QfCfg<NT>;
    using Bars = typename C::Bars;
    extern __shared__ __align__(1024) uint8_t qf_smem[];
    float *sF = (float *)(qf_smem + C::kStages * C::kStage);  // [gate, up][block][row]
    Bars &ms = *(Bars *)((uint8_t *)sF + C::kMats * C::kFactors);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &ms.abort;
    // gated: ranks 0 .. split - 1 hold the first half of the 128 outputs, split .. 2 split - 1 the second
    const int cluster = GATED ? 2 * split : split, peer = blockIdx.x % cluster, tile = blockIdx.x / cluster;
    const int rank = GATED ? peer % split : peer, half = GATED ? peer / split : 0;
    const int n0 = tile * 128, rows = p.M;
    const int k0 = (int)((long long)rank * p.KB / split), k1 = (int)((long long)(rank + 1) * p.KB / split);
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&ms.full[s], 1);
            mbar_init(&ms.empty[s], 1);
        }
        for (int s = 0; s < C::kSlots; ++s) {
            mbar_init(&ms.afull[s], 1);
            mbar_init(&ms.aempty[s], 4);
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
        named_bar_sync(7, C::kThreads - 32);
        tc_fence_after();
        tmem = ms.tmem;
    }

    if (warp == 0) {
        if (ql_elect()) {
            uint32_t u = 0;
            for (int kb = k0; kb < k1; ++kb, ++u) {
                const uint32_t s = u % C::kStages;
                if (u >= C::kStages && !mbar_wait_bounded(&ms.empty[s], ((u / C::kStages) & 1) ^ 1, abort)) break;
                uint8_t *to = qf_smem + s * C::kStage;
                mbar_arrive_expect_tx(&ms.full[s], C::kStage);
                // 16-bit elements: 64 a box row
                tma_load_2d(to, &tm_w0, kb * 64, n0 + 64 * half, &ms.full[s]);
                if (GATED) tma_load_2d(to + 64 * 128, &tm_w1, kb * 64, n0 + 64 * half, &ms.full[s]);
                tma_load_2d(to + C::kX, &tm_x, kb * 64, 0, &ms.full[s]);
            }
            ms.issued = u;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (ql_elect()) {
            const uint32_t lo = sdesc_lo(smem_u32(qf_smem));
            constexpr uint32_t hi = sdesc_hi(1024, 2), id = idesc_e4m3_f32(128, NT);
            const uint32_t n = k1 - k0;
            for (uint32_t u = 0; u < n; ++u) {
                const uint32_t s = u % C::kStages, a = u % C::kSlots;
                if (!mbar_wait_bounded(&ms.full[s], (u / C::kStages) & 1, abort)) break;
                if (u >= C::kSlots && !mbar_wait_bounded(&ms.aempty[a], ((u / C::kSlots) & 1) ^ 1, abort)) break;
                tc_fence_after();
                const uint32_t w = lo + s * (C::kStage >> 4), x = w + (C::kX >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_e4m3(tmem + a * NT, (uint64_t)hi << 32 | (w + 2 * k), (uint64_t)hi << 32 | (x + 2 * k), id, k > 0);
                mma_commit(&ms.empty[s]);
                mma_commit(&ms.afull[a]);
            }
            mma_commit(&ms.done);
            ql_drain(&ms.done, 0);
            for (uint32_t u = n > C::kStages ? n - C::kStages : 0; !*abort && u < n; ++u)  // and what the last stages' commits send
                ql_drain(&ms.empty[u % C::kStages], (u / C::kStages) & 1);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, me = tid - 64, mat = GATED && q >= 2;  // lanes 64 ..: up's outputs
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16);
        const float *fac = sF + mat * (kQfWindow * NT);
        const size_t block = (size_t)(n0 / kQlBlock) * p.KB;
        float acc[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i] = 0.f;
        const uint32_t n = k1 - k0;
        for (uint32_t u = 0; u < n; ++u) {
            const uint32_t w = u % kQfWindow, a = u % C::kSlots;
            if (w == 0) {
                __syncwarp();
                named_bar_sync(1, 128);  // the window before has been used
                const int blocks = min(kQfWindow, (int)(n - u));
                for (int i = me; i < blocks * NT; i += 128) {
                    const int b = k0 + (int)u + i / NT, m = i % NT;
                    const float x = m < rows ? __ldg(p.sx + (size_t)b * p.sx_stride + m) : 0.f;
                    sF[i] = x * __ldg(p.sw[0] + block + b);
                    if (GATED) sF[kQfWindow * NT + i] = x * __ldg(p.sw[1] + block + b);
                }
                __syncwarp();
                named_bar_sync(1, 128);
            }
            // every warp keeps to the barriers above, whatever a wait says
            if (!ql_warp_wait(&ms.afull[a], (u / C::kSlots) & 1, abort)) continue;
            tc_fence_after();
            constexpr int kLoad = NT < 32 ? NT : 32;
#pragma unroll
            for (int c = 0; c < NT; c += kLoad) {
                float v[kLoad];
                if constexpr (NT < 32) tmem_ld16_now(tl + a * NT + c, v);
                else tmem_ld32_now(tl + a * NT + c, v);
                if (c + kLoad == NT) {  // read: its products may be replaced
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.aempty[a]);
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < kLoad; i += 4) {
                    const float4 f = *(const float4 *)(fac + w * NT + c + i);
                    acc[c + i] = __fmaf_rn(v[i], f.x, acc[c + i]);
                    acc[c + i + 1] = __fmaf_rn(v[i + 1], f.y, acc[c + i + 1]);
                    acc[c + i + 2] = __fmaf_rn(v[i + 2], f.z, acc[c + i + 2]);
                    acc[c + i + 3] = __fmaf_rn(v[i + 3], f.w, acc[c + i + 3]);
                }
            }
        }
        // partial sums [row, output] in the stages' place: every product is done
        float *part = (float *)qf_smem + 32 * q + lane;
        if (!*abort) {
#pragma unroll
            for (int i = 0; i < NT; ++i) part[i * 128] = acc[i];
        }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    // row i of the tile is finished by CTA i % cluster: a warp a row, four outputs a lane
    for (int row = peer + cluster * warp; row < rows; row += cluster * (C::kThreads / 32)) {
        const int m = row;
        // partial sums of four outputs, in the place `at` of CTAs first .. first + split - 1
        auto gather = [&](const float *at, int first) {
            float4 s[kQfMaxCluster];
#pragma unroll
            for (int r = 0; r < kQfMaxCluster; ++r)
                if (r < split) s[r] = ld_peer_f4(at, first + r);
            float4 v = s[0];
#pragma unroll
            for (int r = 1; r < kQfMaxCluster; ++r)
                if (r < split) {
                    v.x += s[r].x;
                    v.y += s[r].y;
                    v.z += s[r].z;
                    v.w += s[r].w;
                }
            return v;
        };
        float4 v[C::kMats];
        if (GATED) {  // outputs 4 lane ..: of half lane / 16, gate's at 4 (lane % 16), up's 64 behind
            const float *at = (const float *)qf_smem + row * 128 + 4 * (lane & 15);
            v[0] = gather(at, lane >> 4 ? split : 0);
            v[1] = gather(at + 64, lane >> 4 ? split : 0);
        } else {
            v[0] = gather((const float *)qf_smem + row * 128 + 4 * lane, 0);
        }
        const int n = n0 + 4 * lane;
        if constexpr (GATED) {
            float h[4] = {ql_gate(v[0].x, v[1].x), ql_gate(v[0].y, v[1].y), ql_gate(v[0].z, v[1].z), ql_gate(v[0].w, v[1].w)};
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
            if (p.add) {
                const float4 a = *(const float4 *)(p.add + (size_t)m * p.add_stride + n);
                v[0].x += a.x;
                v[0].y += a.y;
                v[0].z += a.z;
                v[0].w += a.w;
            }
            if (p.y_fp32) {
                *(float4 *)((float *)p.y + (size_t)m * p.y_stride + n) = v[0];
            } else {
                const __nv_bfloat162 a = __floats2bfloat162_rn(v[0].x, v[0].y), b = __floats2bfloat162_rn(v[0].z, v[0].w);
                *(uint2 *)((__nv_bfloat16 *)p.y + (size_t)m * p.y_stride + n) = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
            }
        }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its sums
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
    if (tid == 0 && ms.abort) {  // no copy outlives the CTA
        for (uint32_t u = ms.issued > C::kStages ? ms.issued - C::kStages : 0; u < ms.issued; ++u)
            ql_drain(&ms.full[u % C::kStages], (u / C::kStages) & 1);
        set_error(p.err, DSPARK_ERR_TIMEOUT);
    }
}

template <int NT, bool GATED>
static QlPlan plan(const QlParams &p) {
    using C = QfCfg<NT>;
    static OncePerDevice once;
    static ClusterRoom<decltype(&qgemm_few_kernel<NT, GATED>)> room;
    QlPlan r = {1, (p.N + 127) / 128, 1, 0.f, cudaSuccess};
    r.error = once(
        [] { return cudaFuncSetAttribute(qgemm_few_kernel<NT, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    if (r.error != cudaSuccess) return r;
    constexpr int kHalves = GATED ? 2 : 1;
    for (int s = 1; s * kHalves <= kQfMaxCluster && s <= p.KB; ++s) {
        const int n = room(qgemm_few_kernel<NT, GATED>, s * kHalves, C::kThreads, C::kSmem);
        if (s > 1 && r.tiles > n) continue;
        r.split = s;
        r.room = n;
    }
    return r;
}

template <int NT, bool GATED>
static cudaError_t launch(const QlParams &p, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                          const QlPlan &plan, cudaStream_t st) {
    using C = QfCfg<NT>;
    CUtensorMap mx, m0, m1;
    constexpr int kBox = GATED ? 64 : 128;
    if (!encode_u16_map(&mx, x.codes, x.rows, x.k, 128, NT) || !encode_u16_map(&m0, w0.codes, w0.n, w0.k, 128, kBox))
        return cudaErrorInvalidValue;
    m1 = m0;
    if (GATED && !encode_u16_map(&m1, w1.codes, w1.n, w1.k, 128, kBox)) return cudaErrorInvalidValue;
    const int cluster = plan.split * (GATED ? 2 : 1);
    if (plan.tiles * cluster >= 1ll << 30) return cudaErrorInvalidValue;
    return launch_pdl_cluster(qgemm_few_kernel<NT, GATED>, dim3((unsigned)(plan.tiles * cluster)), dim3(C::kThreads), (size_t)C::kSmem, st,
                              cluster, mx, m0, m1, p, plan.split);
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
