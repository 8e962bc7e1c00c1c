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

// Shared-memory matrix descriptor of a swizzled operand, as two words (type 2:
// 128-byte rows and swizzle, 4: 64-byte). K-major: sbo is the distance of 8-row
// groups. MN-major (rows of MN elements, one per k): sbo is the distance of
// groups of 8 k. The operands used here are one swizzle row wide, so the other
// offset is unused. Moving by n bytes adds n >> 4 to the low word.
DS_DEVINL uint32_t sdesc_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | 1u << 16; }
__host__ __device__ constexpr uint32_t sdesc_hi(uint32_t sbo, uint32_t type) { return (sbo >> 4) | 1u << 14 | type << 29; }

// Block-scaled MMA, kind::mxf8f6f4, descriptors as words (one 32-bit addition is
// all that an operand costs the issuing thread): E4M3 A [M x 32] and B [N x 32], one E8M0
// scale 2^(byte - 127) per row and 32 k. Scale words lie in tensor memory: row r
// at lane r % 32 of column r / 32 (the same in all four lane quarters), byte k of
// the word for the k-block that the instruction descriptor selects (here: sfb; A's
// byte 0). Both operands K-major, or with kIdescBothMN both MN-major.
__host__ __device__ constexpr uint32_t idesc_mx_e4m3(int M, int N, int sfb) {
    return ((uint32_t)sfb << 4) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdescBothMN = 1u << 15 | 1u << 16;
DS_DEVINL void mma_mx_e4m3_w(uint32_t d_tmem, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi, uint32_t idesc,
                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %8, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], a, b, %5, [%6], [%7], p;\n\t}" ::"r"(
            d_tmem),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
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
