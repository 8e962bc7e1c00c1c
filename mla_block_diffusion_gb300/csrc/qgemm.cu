// Products of quantised rows with block-scaled weights, many rows (include/dspark.h, calls 12 and 13).
//
//   y[m, n] = sum_b sx[b, m] sw[n / 128, b] sum_{k in block b} cx[m, k] cw[n, k]
//
// A tile is 128 rows x 256 outputs: 256 columns of one matrix, or 128 of the
// gate's and the same 128 of up's, so that the epilogue holds both factors of
// silu(g) u. Rows are the accumulator's lanes. E4M3 codes go to the tensor core as
// they are stored (kind::f8f6f4); a block of 128 k is four MMAs into one of two
// accumulators of 256 columns, from which the epilogue warps add it, times
// sx sw, to fp32 registers: scales are any fp32 numbers, and no sum is longer than
// 128 terms before it is one of fp32 FMAs. A thread holds 64 + 64 columns of one row,
// so that a block costs it two factors.
#include <math.h>

#include "per_device.h"
#include "qlinear.h"

namespace ds {

constexpr int kQgThreads = 384;                    // 4 warps that issue, 8 that sum; registers: 168 x 384 = 88 x 128 + 208 x 256
constexpr int kQgRegsIssue = 88, kQgRegsSum = 208;
constexpr int kQgBox = 128 * 128;                  // bytes: 128 rows or outputs x 128 k
constexpr int kQgStage = 3 * kQgBox;               // rows, two boxes of outputs
constexpr int kQgStages = 4;
constexpr int kQgOut = 8 * 4096;                   // staged output: 4 KB a summing warp

struct QgBars {
    uint64_t full[kQgStages], empty[kQgStages], afull[2], aempty[2], done;
    uint32_t tmem;
    volatile int abort;
    uint32_t issued;                               // stages that the producer has requested
    uint32_t amax[2][2][128];                      // gated, tiles in turn: a row's largest magnitude by column half
};
constexpr int kQgSmem = kQgStages * kQgStage + kQgOut + (int)sizeof(QgBars);
static_assert(kQgSmem <= 232448, "shared memory");

template <bool GATED>
__global__ void __launch_bounds__(kQgThreads, 1)
    qgemm_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w0,
                 const __grid_constant__ CUtensorMap tm_w1, const QlParams p, int tiles_m, int tiles) {
    extern __shared__ __align__(1024) uint8_t qg_smem[];
    uint8_t *sOut = qg_smem + kQgStages * kQgStage;
    QgBars &ms = *(QgBars *)(sOut + kQgOut);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &ms.abort;
    const int KB = p.KB;
    if (tid == 0) {
        for (int s = 0; s < kQgStages; ++s) {
            mbar_init(&ms.full[s], 1);
            mbar_init(&ms.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&ms.afull[s], 1);
            mbar_init(&ms.aempty[s], 8);
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
        tmem_alloc(&ms.tmem, 512);
        pdl_trigger();
    }
    uint32_t tmem = 0;
    if (warp != 0) {
        tc_fence_before();
        named_bar_sync(7, kQgThreads - 32);
        tc_fence_after();
        tmem = ms.tmem;
    }

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQgRegsIssue));
        if (warp == 0) {
            if (ql_elect()) {
                uint32_t u = 0;
                bool ok = true;
                for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                    const int m0 = t % tiles_m * 128, n0 = t / tiles_m * (GATED ? 128 : 256);
                    for (int kb = 0; kb < KB; ++kb, ++u) {
                        const uint32_t s = u % kQgStages, par = (u / kQgStages) & 1;
                        if (u >= kQgStages && !mbar_wait_bounded(&ms.empty[s], par ^ 1, abort)) {
                            ok = false;
                            break;
                        }
                        uint8_t *to = qg_smem + s * kQgStage;
                        mbar_arrive_expect_tx(&ms.full[s], kQgStage);
                        // 16-bit elements: 64 a box row
                        tma_load_2d(to, &tm_x, kb * 64, m0, &ms.full[s]);
                        tma_load_2d(to + kQgBox, &tm_w0, kb * 64, n0, &ms.full[s]);
                        if (GATED) tma_load_2d(to + 2 * kQgBox, &tm_w1, kb * 64, n0, &ms.full[s]);
                        else tma_load_2d(to + 2 * kQgBox, &tm_w0, kb * 64, n0 + 128, &ms.full[s]);
                    }
                }
                ms.issued = u;
            }
            __syncwarp();
        } else if (warp == 1) {
            if (ql_elect()) {
                const uint32_t lo = sdesc_lo(smem_u32(qg_smem));
                constexpr uint32_t hi = sdesc_hi(1024, 2), id = idesc_e4m3_f32(128, 256);
                uint32_t u = 0;
                bool ok = true;
                for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x)
                    for (int kb = 0; kb < KB; ++kb, ++u) {
                        const uint32_t s = u % kQgStages;
                        ok = mbar_wait_bounded(&ms.full[s], (u / kQgStages) & 1, abort) &&
                             (u < 2 || mbar_wait_bounded(&ms.aempty[u & 1], ((u >> 1) & 1) ^ 1, abort));
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = lo + s * (kQgStage >> 4), b = a + (kQgBox >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_e4m3(tmem + 256 * (u & 1), (uint64_t)hi << 32 | (a + 2 * k), (uint64_t)hi << 32 | (b + 2 * k), id, k > 0);
                        mma_commit(&ms.empty[s]);
                        mma_commit(&ms.afull[u & 1]);
                    }
                mma_commit(&ms.done);
                mbar_drain(&ms.done, 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQgRegsSum));
        const int q = warp & 3, h = (warp - 4) >> 2;  // lanes 32 q .., columns 64 h .. of either half
        const uint32_t tl = tmem + ((uint32_t)(32 * q) << 16) + 64 * h;
        uint8_t *out = sOut + (warp - 4) * 4096;
        uint32_t u = 0, count = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++count) {
            const int m0 = t % tiles_m * 128 + 32 * q, n0 = t / tiles_m * (GATED ? 128 : 256), row = m0 + lane;
            const int nb = (p.N + kQlBlock - 1) / kQlBlock, b0 = n0 / kQlBlock;
            const float *sx = p.sx + (row < p.M ? row : p.M - 1);
            const float *s0 = p.sw[0] + (size_t)b0 * KB;
            const float *s1 = GATED ? p.sw[1] + (size_t)b0 * KB : s0 + (b0 + 1 < nb ? KB : 0);
            unsigned long long acc[64];  // columns 64 h .. of the first half, then of the second
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            // scales two blocks ahead
            float x0 = __ldg(sx), x1 = KB > 1 ? __ldg(sx + p.sx_stride) : 0.f;
            float a0 = __ldg(s0), a1 = KB > 1 ? __ldg(s0 + 1) : 0.f, c0 = __ldg(s1), c1 = KB > 1 ? __ldg(s1 + 1) : 0.f;
            for (int kb = 0; kb < KB; ++kb, ++u) {
                const unsigned long long f0 = pack2(x0 * a0), f1 = pack2(x0 * c0);
                x0 = x1;
                a0 = a1;
                c0 = c1;
                if (kb + 2 < KB) {
                    x1 = __ldg(sx + (size_t)(kb + 2) * p.sx_stride);
                    a1 = __ldg(s0 + kb + 2);
                    c1 = __ldg(s1 + kb + 2);
                }
                ok = ql_warp_wait(&ms.afull[u & 1], (u >> 1) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = tl + 256 * (u & 1);
                uint32_t v[2][16];
                tmem_ld16_issue(at, v[0]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    tmem_ld_wait_tied(v[c & 1]);
                    if (c < 7) tmem_ld16_issue(at + (c + 1 & 3) * 16 + (c + 1 >> 2) * 128, v[~c & 1]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) fma2(acc[8 * c + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], c < 4 ? f0 : f1);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.aempty[u & 1]);
            }
            if (!ok) break;
            if constexpr (GATED) {
                float v[64];
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 g = unpack2(acc[i]), w = unpack2(acc[32 + i]);
                    v[2 * i] = ql_gate(g.x, w.x);
                    v[2 * i + 1] = ql_gate(g.y, w.y);
                    const uint32_t a = __float_as_uint(v[2 * i]) & 0x7fffffffu, b = __float_as_uint(v[2 * i + 1]) & 0x7fffffffu;
                    if (a < 0x7f800000u) mx = max(mx, a);
                    else v[2 * i] = __uint_as_float(0x7fffffffu);
                    if (b < 0x7f800000u) mx = max(mx, b);
                    else v[2 * i + 1] = __uint_as_float(0x7fffffffu);
                }
                ms.amax[count & 1][h][32 * q + lane] = mx;
                named_bar_sync(1 + q, 64);  // the two warps of these rows
                mx = max(mx, ms.amax[count & 1][h ^ 1][32 * q + lane]);
                const int e = ql_exponent(mx);
                const float inv = qc_pow2(-e);
                if (h == 0 && row < p.M) p.sh[(size_t)b0 * p.sh_stride + row] = qc_pow2(e);
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
                // 32 columns at a time through shared memory: 128 bytes a row, 16-byte pieces swizzled
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 a = unpack2(acc[16 * c + 2 * i]), b = unpack2(acc[16 * c + 2 * i + 1]);
                        *(float4 *)(out + lane * 128 + ((i ^ lane) & 7) * 16) = make_float4(a.x, a.y, b.x, b.y);
                    }
                    __syncwarp();
                    const int n = n0 + 128 * (c >> 1) + 64 * h + 32 * (c & 1) + 4 * (lane & 7);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3), m = m0 + r;
                        float4 v = *(const float4 *)(out + r * 128 + ((lane ^ r) & 7) * 16);
                        if (m < p.M && n < p.N) {
                            if (p.add) {
                                const float4 a = *(const float4 *)(p.add + (size_t)m * p.add_stride + n);
                                v.x += a.x;
                                v.y += a.y;
                                v.z += a.z;
                                v.w += a.w;
                            }
                            if (p.y_fp32) {
                                *(float4 *)((float *)p.y + (size_t)m * p.y_stride + n) = v;
                            } else {
                                const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
                                *(uint2 *)((__nv_bfloat16 *)p.y + (size_t)m * p.y_stride + n) =
                                    make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && ms.abort) {  // no copy outlives the CTA
        for (uint32_t u = ms.issued > kQgStages ? ms.issued - kQgStages : 0; u < ms.issued; ++u)
            mbar_drain(&ms.full[u % kQgStages], (u / kQgStages) & 1);
        set_error(p.err, DSPARK_ERR_TIMEOUT);
    }
}

template <bool GATED>
static cudaError_t launch(const QlParams &p, const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1, int num_sms,
                          cudaStream_t st) {
    static OncePerDevice once;
    const cudaError_t e =
        once([] { return cudaFuncSetAttribute(qgemm_kernel<GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQgSmem); });
    if (e != cudaSuccess) return e;
    const int tiles_m = (p.M + 127) / 128, tiles_n = (p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    const long long tiles = (long long)tiles_m * tiles_n;
    if (tiles >= 1ll << 30) return cudaErrorInvalidValue;
    return launch_pdl(qgemm_kernel<GATED>, dim3((unsigned)(tiles < num_sms ? tiles : num_sms)), dim3(kQgThreads), (size_t)kQgSmem, st,
                      x, w0, w1, p, tiles_m, (int)tiles);
}

cudaError_t launch_qgemm(const QlParams &p, bool gated, const CUtensorMap &x, const CUtensorMap &w0, const CUtensorMap &w1,
                         int num_sms, cudaStream_t st) {
    return gated ? launch<true>(p, x, w0, w1, num_sms, st) : launch<false>(p, x, w0, w1, num_sms, st);
}

}  // namespace ds
