// Internal declarations of the 8-bit latent cache (qcache.cu, qattn.cu, qattn_tc.cu).
#pragma once

#include "common.cuh"

namespace ds {

constexpr int kQcPage = 64;       // tokens per page
constexpr int kQcEmax = 60;       // scale exponents lie in [-kQcEmax, kQcEmax]
constexpr int kQcMaxBs = 1024;
constexpr int kQaTile = 64;       // query rows (token, head) per work item
constexpr int kQaChunk = 128;     // cached tokens per unit of work: two pages
constexpr int kQaThreads = 384;    // of an attention CTA
constexpr int kQaMaxGrid = 512;   // CTAs of an attention launch at most
constexpr size_t kQcCtlBytes = 1024;  // error word, zero-filled by the caller

// Exponent of a page scale: whether it is 2^e with e in range.
DS_DEVINL bool qc_scale_exponent(float s, int *e) {
    const uint32_t u = __float_as_uint(s);
    const int x = (int)(u >> 23) - 127;  // a negative, zero, subnormal or non-finite scale falls out of range
    const bool ok = (u & 0x7fffffu) == 0 && x >= -kQcEmax && x <= kQcEmax;
    *e = ok ? x : 0;
    return ok;
}
DS_DEVINL float qc_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

struct QaSplit {
    int q0, r0, rows;  // the item: its request's first query token, its first row, rows from there to the request's end
    int lo_slot;     // partial slot of the item's first CTA
    int c_hi;        // its last CTA (slots 2c beyond the first); < 0: none
};

struct QaParams {
    const __nv_bfloat16 *q;
    long long q_stride;
    const int32_t *cu_q, *length;
    int H, bs, total_q, causal;
    uint32_t h_mul;                  // r / H = r * h_mul >> h_shift for r < 2^31
    int h_shift;
    float scale_log2;                // softmax scale * log2(e)
    __nv_bfloat16 *o;
    long long o_stride;
    float *lse;
    const uint8_t *codes;            // [n_pages, 64, D]
    const float *scales;             // [n_pages]
    const int32_t *page_table;
    int n_pages, max_pages;
    float *part_o;                   // [2 * grid, kQaTile, DV] weights times codes, not normalised
    float2 *part_ml;                 // [2 * grid, kQaTile] (log2 reference, sum)
    QaSplit *split;                  // [grid] the item that starts in this CTA and goes on in later ones
    int *err;
};

cudaError_t launch_qattn_tc(const QaParams &p, int kv_lora, int grid, cudaStream_t st);
cudaError_t launch_qattn(const QaParams &p, int kv_lora, int num_sms, cudaStream_t st);

}  // namespace ds
