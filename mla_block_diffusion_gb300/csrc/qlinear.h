// Internal declarations of the 8-bit layers (qlinear.cu, qgemm.cu, qgemm_few.cu).
#pragma once

#include "e4m3.cuh"
#include "internal.h"
#include "qcache.h"

namespace ds {

constexpr int kQlBlock = 128;     // inputs (and, for weights, outputs) that share a scale
constexpr int kQlEmin = -100;     // the least exponent of a scale that the quantiser writes

// A product of quantised rows and one weight matrix, or (gated) two of the same shape.
struct QlParams {
    int M, N, KB;                 // rows, outputs (of one matrix), blocks of k
    const float *sx;              // [KB, M], row stride sx_stride
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
// silu(g) * u
DS_DEVINL float ql_gate(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }
// An infinity as NaN, for the codes: E4M3 has no infinity, and what a row with one stands for is not finite.
DS_DEVINL float ql_inf_to_nan(float x) { return fabsf(x) == INFINITY ? __uint_as_float(0x7fffffffu) : x; }

// One lane of the warp; a branch on it is known to hold a single thread.
DS_DEVINL bool ql_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
DS_DEVINL bool ql_warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort));
}
// acc (a pair of floats) += (a, b) * f
DS_DEVINL void fma2(unsigned long long &acc, uint32_t a, uint32_t b, unsigned long long f) {
    asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}" : "+l"(acc) : "r"(a), "r"(b), "l"(f));
}
DS_DEVINL unsigned long long pack2(float f) {
    unsigned long long d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(f));
    return d;
}
DS_DEVINL float2 unpack2(unsigned long long d) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(d));
    return f;
}

cudaError_t launch_qgemm(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0, const dspark_qweight_t &w1,
                         int num_sms, cudaStream_t st);
cudaError_t launch_qgemm_few(const QlParams &p, bool gated, const dspark_qrows_t &x, const dspark_qweight_t &w0,
                             const dspark_qweight_t &w1, int num_sms, cudaStream_t st);

}  // namespace ds
