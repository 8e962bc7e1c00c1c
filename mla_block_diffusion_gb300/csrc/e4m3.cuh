// E4M3 on the tensor core and in registers: the kind::f8f6f4 MMA, conversions
// between fp32 / f16 pairs and E4M3 codes, and the residual of a two-term split.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ds {

// Instruction descriptor, kind::f8f6f4: E4M3 A and B, fp32 accumulator, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

DS_DEVINL void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Two floats to an f16 pair (round to nearest even): `even` in the low half.
DS_DEVINL uint32_t f32x2_to_f16x2(float even, float odd) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(odd), "f"(even));
    return d;
}
// An f16 pair to two E4M3 codes (round to nearest even, saturating), low half
// to the low byte.
DS_DEVINL uint32_t f16x2_to_e4m3x2(uint32_t h) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h));
    return d;
}
// Two E4M3 codes (low byte first) to an f16 pair.
DS_DEVINL uint32_t e4m3x2_to_f16x2_(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
// (a - b) * 16 on f16 pairs.
DS_DEVINL uint32_t f16x2_sub_x16(uint32_t a, uint32_t b) {
    const __half2 d = __hmul2(__hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b)),
                              __floats2half2_rn(16.f, 16.f));
    return *reinterpret_cast<const uint32_t *>(&d);
}

}  // namespace ds
