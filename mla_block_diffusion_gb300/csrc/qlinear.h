// Internal declarations of the 8-bit layers (qlinear.cu, qgemm.cu, qgemm_few.cu).
#pragma once

#include <atomic>

#include "e4m3.cuh"
#include "internal.h"
#include "qcache.h"

namespace ds {

constexpr int kQlBlock = 128;     // inputs (and, for weights, outputs) that share a scale
constexpr int kQlEmin = -100;     // the least exponent of a scale that the quantiser writes

// A product of quantised rows and one weight matrix, or (gated) two of the same shape.
struct QlParams {
    int M, N, KB;                 // rows, outputs (of one matrix), blocks of k
    const float *sx;              // [KB, M], sx_stride from one block to the next
    long long sx_stride;
    const float *sw[2];           // [ceil(N / 128), KB]; gated: gate, up; else both the same
    // matmul
    const float *add;             // or null
    long long add_stride;
    void *y;
    int y_fp32;
    long long y_stride;
    // gated
    uint8_t *h;                   // [M, N]
    float *sh;                    // [ceil(N / 128), M]
    long long sh_stride;
    int *err;
};

// Least e >= kQlEmin with the finite number `bits` (fp32, its magnitude) <= 448 * 2^e (448 = 1.75 * 2^8).
DS_DEVINL int ql_exponent(uint32_t bits) {
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(kQlEmin, e);
}
// Two floats to two E4M3 codes (round to nearest even, saturating, NaN stays NaN), even low.
DS_DEVINL uint32_t ql_e4m3x2(float even, float odd) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(odd), "f"(even));
    return d;
}
// silu(g) * u, off by less than 2^-15 of it beside what g is off by: the fast exponential is off by 2 + 1.173 |x| units of
// 2^-23, and gates below -176 make nothing that a code can hold (2^-110) of any u. Below -87 exp(-g) leaves what the fast
// division takes (up to 2^126), while 1 + exp(g) is 1; exp(g) would leave the normal numbers, so that its root enters twice.
constexpr float kQlFar = -87.f;
DS_DEVINL float ql_gate_near(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }
DS_DEVINL float ql_gate_far(float g, float u) {
    const float t = __expf(0.5f * g);
    return (g * t) * (u * t);
}
DS_DEVINL float ql_gate(float g, float u) { return g < kQlFar ? ql_gate_far(g, u) : ql_gate_near(g, u); }
// An infinity as NaN, for the codes: E4M3 has no infinity, and what a row with one stands for is not finite.
DS_DEVINL float ql_inf_to_nan(float x) { return fabsf(x) == INFINITY ? __uint_as_float(0x7fffffffu) : x; }

// mbar_drain for what has nearly always come: reading the timer first would cost more than the look.
DS_DEVINL void ql_drain(uint64_t *bar, uint32_t parity) {
    if (!mbar_try_wait(bar, parity)) mbar_drain(bar, parity);
}
// One lane of the warp; a branch on it is known to hold a single thread.
DS_DEVINL bool ql_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A whole warp waits, and stays whole: every turn of the loop ends in a vote, on which all lanes leave it together. What
// follows reads tensor memory, whose instructions want all 32 lanes converged.
DS_DEVINL bool ql_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    unsigned long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
        if (__all_sync(~0u, mbar_try_wait(bar, parity))) return true;
        if ((i & 255u) == 255u) {
            const unsigned long long t = __shfl_sync(~0u, globaltimer(), 0);
            if (t0 == 0) t0 = t;
            if (__any_sync(~0u, *abort != 0)) return false;
            if (t - t0 > kWaitLimitNs) {
                *abort = 1;
                return false;
            }
        }
    }
}
// 32 columns of the warp's lanes and the wait for them in one statement: apart, with the registers tied to the wait, each
// may cost a move.
DS_DEVINL void tmem_ld32_now(uint32_t addr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(addr)
        : "memory");
}
DS_DEVINL void tmem_ld16_now(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}

// Four bytes into shared memory; the barrier's arrival when all that this thread has requested is there.
DS_DEVINL void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
DS_DEVINL void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Clusters of `cluster` CTAs that fit on the current device at once (0: it holds none); asked once per kernel, size and device,
// and again where the question failed.
template <typename Kernel>
class ClusterRoom {
    static constexpr int kDevices = 64, kMost = 8;
    std::atomic<int> known_[kDevices][kMost + 1] = {};  // answer + 1

  public:
    cudaError_t operator()(Kernel kern, int cluster, int threads, int smem, int *n) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const bool kept = dev >= 0 && dev < kDevices && cluster <= kMost;
        if (kept && (*n = known_[dev][cluster].load(std::memory_order_relaxed) - 1) >= 0) return cudaSuccess;
        carveout_max((const void *)kern);  // as every launch has it
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)cluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(cluster);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(n, kern, &cfg);
        if (e == cudaSuccess && kept) known_[dev][cluster].store(*n + 1, std::memory_order_relaxed);
        return e;
    }
};

// How either kernel would divide a call.
struct QlPlan {
    int split;           // few: CTAs that share a tile's blocks of k; many: 1 or 2 halves of 128 outputs a tile
    long long tiles;
    int room;            // many: pairs on the device at once
    float time;          // many: about how long, in us
    cudaError_t error;
};
QlPlan plan_qgemm(const QlParams &p, bool gated);
QlPlan plan_qgemm_few(const QlParams &p, bool gated);
cudaError_t launch_qgemm(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                         const QlPlan &plan, cudaStream_t st);
cudaError_t launch_qgemm_few(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0,
                             const dspark_qweight_t &w1, const QlPlan &plan, cudaStream_t st);

}  // namespace ds
