// 8-bit layers with a scale for each block of 128: host entry points and the
// quantisers (include/dspark.h, calls 10 to 13).
#include <math.h>
#include <string.h>

#include "overlap.h"
#include "qlinear.h"

using namespace ds;

namespace ds {

// ---------------------------------------------------------------------------
// Quantising rows: 16 lanes hold a block of 128 elements, eight each.
//
// e = the least exponent >= -100 with amax <= 448 * 2^e; codes are RN(x 2^-e),
// one rounding since 2^-e is a power of two. Bound: HBM (2 or 4 bytes read and
// one written per element). A CTA takes 8 rows x 2 PER blocks, each half-warp PER
// blocks that it requests together; the scales of 8 rows are one full sector of
// their [block, row] matrix. Measured, inputs in turn: 4000 x 7168 bf16 17.4 us (5.0 TB/s, 63 % of the
// issue slots), fp32 27.1 (5.3 TB/s).
// ---------------------------------------------------------------------------
constexpr int kQrThreads = 256, kQrRows = 8;

// Eight consecutive elements, as they lie in memory.
template <typename T>
struct Eight {
    static constexpr bool kWide = sizeof(T) == 4;
    uint4 v[kWide ? 2 : 1];
    DS_DEVINL void load(const T *p) {
        v[0] = __ldg((const uint4 *)p);
        if (kWide) v[kWide] = __ldg((const uint4 *)p + 1);
    }
    DS_DEVINL void zero() {
        v[0] = make_uint4(0, 0, 0, 0);
        if (kWide) v[kWide] = v[0];
    }
    DS_DEVINL float at(int i) const {
        const uint32_t *w = (const uint32_t *)v;
        return __uint_as_float(kWide ? w[i] : (i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    // Largest magnitude, as the bits of an fp32 number (an infinity or NaN is above every number).
    DS_DEVINL uint32_t amax() const {
        const uint32_t *w = (const uint32_t *)v;
        if (kWide) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        }
        const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        return max(m << 16, m & 0xffff0000u);
    }
    DS_DEVINL uint32_t amax_finite() const {
        uint32_t m = 0;
        for (int i = 0; i < 8; ++i) {
            const uint32_t u = __float_as_uint(at(i)) & 0x7fffffffu;
            if (u < 0x7f800000u) m = max(m, u);
        }
        return m;
    }
    DS_DEVINL uint2 codes(float inv) const {
        return make_uint2(ql_e4m3x2(at(0) * inv, at(1) * inv) | ql_e4m3x2(at(2) * inv, at(3) * inv) << 16,
                          ql_e4m3x2(at(4) * inv, at(5) * inv) | ql_e4m3x2(at(6) * inv, at(7) * inv) << 16);
    }
    DS_DEVINL uint2 codes_nan(float inv) const {  // some are not finite
        uint32_t c[4];
        for (int i = 0; i < 4; ++i) c[i] = ql_e4m3x2(ql_inf_to_nan(at(2 * i)) * inv, ql_inf_to_nan(at(2 * i + 1)) * inv);
        return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
};
constexpr uint32_t kQlInf = 0x7f800000u;

template <typename T, int PER>
__global__ void __launch_bounds__(kQrThreads, sizeof(T) == 2 ? 8 : 5) quantise_rows_kernel(const T *__restrict__ x, long long x_stride, int M, int K,
                                                                   uint8_t *__restrict__ codes, float *__restrict__ scales,
                                                                   long long s_stride) {
    const int tid = threadIdx.x, lane16 = tid & 15, half = tid >> 4;
    const int row0 = blockIdx.x * kQrRows, first = blockIdx.y * (2 * PER);
    const int r = row0 + (half & 7), k = (first + (half >> 3)) * kQlBlock + 8 * lane16;
    const int left = r < M ? K - k : 0;  // elements from this thread's first to the row's end
    __shared__ float s_scale[2 * PER][kQrRows];
    pdl_trigger();
    pdl_wait();
    const T *from = x + (long long)r * x_stride + k;
    uint8_t *to = codes + (long long)r * K + k;
    Eight<T> v[PER];
    uint32_t m[PER], all = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (2 * i * kQlBlock < left) v[i].load(from + 2 * i * kQlBlock);
        else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        m[i] = v[i].amax();
        all = max(all, m[i]);
    }
    const bool bad = __any_sync(~0u, all >= kQlInf);  // some are not finite
    if (bad) {
#pragma unroll
        for (int i = 0; i < PER; ++i) m[i] = v[i].amax_finite();
    }
    const uint32_t peers = 0xffffu << (tid & 16);
    float scale[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = ql_exponent(__reduce_max_sync(peers, m[i]));
        scale[i] = qc_pow2(e);
        m[i] = (uint32_t)(127 - e) << 23;  // 2^-e
    }
    if (!bad) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (2 * i * kQlBlock < left) *(uint2 *)(to + 2 * i * kQlBlock) = v[i].codes(__uint_as_float(m[i]));
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (2 * i * kQlBlock < left) *(uint2 *)(to + 2 * i * kQlBlock) = v[i].codes_nan(__uint_as_float(m[i]));
    }
    if (lane16 == 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) s_scale[(half >> 3) + 2 * i][half & 7] = scale[i];
    }
    __syncthreads();
    if (tid < 2 * PER * kQrRows) {
        const int b = first + tid / kQrRows, rr = row0 + tid % kQrRows;
        if (rr < M && b * kQlBlock < K) scales[(long long)b * s_stride + rr] = s_scale[tid / kQrRows][tid % kQrRows];
    }
}

// The same over blocks of 128 x 128, one CTA each; the block waits in registers for its maximum.
// Bound: HBM; 7168 x 14336 bf16 55.8 us (5.5 TB/s), fp32 107.9 (4.8 TB/s).
constexpr int kQwThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kQwThreads, sizeof(T) == 2 ? 3 : 2)
    quantise_weight_kernel(const T *__restrict__ w, long long stride, int N, int K, uint8_t *__restrict__ codes, float *__restrict__ scales) {
    constexpr int kPer = kQlBlock / (kQwThreads / 16), kStep = kQlBlock / kPer;  // rows of a half-warp
    __shared__ uint32_t s_max;
    const int tid = threadIdx.x, across = (K + kQlBlock - 1) / kQlBlock;
    const int r0 = blockIdx.x / across * kQlBlock + (tid >> 4), k = blockIdx.x % across * kQlBlock + 8 * (tid & 15);
    pdl_trigger();
    if (tid == 0) s_max = 0;
    pdl_wait();
    Eight<T> v[kPer];
    const T *at = w + (long long)r0 * stride + k;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (r0 + kStep * i < N && k < K) v[i].load(at + (long long)(kStep * i) * stride);
        else v[i].zero();
    }
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m = max(m, v[i].amax());
    const bool bad = m >= kQlInf;
    if (bad) {
        m = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) m = max(m, v[i].amax_finite());
    }
    m = __reduce_max_sync(~0u, m);
    if ((tid & 31) == 0) atomicMax(&s_max, m);
    __syncthreads();
    const int e = ql_exponent(s_max);
    uint8_t *to = codes + (long long)r0 * K + k;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (r0 + kStep * i < N && k < K)
            *(uint2 *)(to + (long long)(kStep * i) * K) = bad ? v[i].codes_nan(qc_pow2(-e)) : v[i].codes(qc_pow2(-e));
    }
    if (tid == 0) scales[blockIdx.x] = qc_pow2(e);
}

template <typename T>
static cudaError_t launch_rows(const void *x, long long stride, const dspark_qrows_t &o, int sms, cudaStream_t st) {
    const int kb = (o.k + kQlBlock - 1) / kQlBlock, rb = (o.rows + kQrRows - 1) / kQrRows;
    // Two blocks a half-warp for long calls of bf16, whose loads are half as long, else one. us, one against two, inputs in
    // turn, rows of 7168: bf16, 7 rows 1.2 and 1.4, 256 2.7 and 3.4, 512 4.1 and 3.9, 1024 6.6 and 6.0, 4000 20.2 and 17.4;
    // fp32, 1024 8.7 and 9.4, 4000 27.1 and 29.1.
    if constexpr (sizeof(T) == 2) {
        if ((long long)rb * kb >= 20ll * sms)
            return launch_pdl(quantise_rows_kernel<T, 2>, dim3(rb, (kb + 3) / 4), dim3(kQrThreads), 0, st, (const T *)x, stride, o.rows,
                              o.k, (uint8_t *)o.codes, o.scales, (long long)o.scale_stride);
    }
    return launch_pdl(quantise_rows_kernel<T, 1>, dim3(rb, (kb + 1) / 2), dim3(kQrThreads), 0, st, (const T *)x, stride, o.rows,
                      o.k, (uint8_t *)o.codes, o.scales, (long long)o.scale_stride);
}
template <typename T>
static cudaError_t launch_weight(const void *w, long long stride, const dspark_qweight_t &o, cudaStream_t st) {
    const int kb = (o.k + kQlBlock - 1) / kQlBlock, nb = (o.n + kQlBlock - 1) / kQlBlock;
    return launch_pdl(quantise_weight_kernel<T>, dim3(kb * nb), dim3(kQwThreads), 0, st, (const T *)w, stride, o.n, o.k,
                      (uint8_t *)o.codes, o.scales);
}

}  // namespace ds

namespace {

bool ok16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
// 2^24 rows of them, 4 bytes each, count within 64 bits; no memory holds two.
constexpr int64_t kMaxStride = 1ll << 36;
bool ok4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool ok_dim(int d) { return d >= 16 && d <= DSPARK_QLINEAR_MAX_DIM && d % 16 == 0; }

// SMs of the current device; 0: the runtime does not say.
int current_sms() {
    constexpr int kDevices = 64;  // devices past these: asked on every call
    static std::atomic<int> known[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool kept = dev >= 0 && dev < kDevices;
    if (kept && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (kept) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

dspark_status done(cudaError_t e) {
    if (e == cudaSuccess) return DSPARK_OK;
    (void)cudaGetLastError();
    return DSPARK_ERR_CUDA;
}

dspark_status check_rows(const dspark_qrows_t *x) {
    if (!x) return DSPARK_ERR_NULL;
    if (x->rows < 0 || x->rows > DSPARK_QLINEAR_MAX_ROWS || !ok_dim(x->k) || x->scale_stride < x->rows || x->scale_stride > kMaxStride) return DSPARK_ERR_SHAPE;
    if (x->rows == 0) return DSPARK_OK;
    if (!x->codes || !x->scales) return DSPARK_ERR_NULL;
    return ok16(x->codes) && ok4(x->scales) ? DSPARK_OK : DSPARK_ERR_ALIGN;
}
dspark_status check_weight(const dspark_qweight_t *w) {
    if (!w) return DSPARK_ERR_NULL;
    if (!ok_dim(w->n) || !ok_dim(w->k)) return DSPARK_ERR_SHAPE;
    if (!w->codes || !w->scales) return DSPARK_ERR_NULL;
    return ok16(w->codes) && ok4(w->scales) ? DSPARK_OK : DSPARK_ERR_ALIGN;
}
// A matrix that the quantiser writes: any number of rows.
dspark_status check_matrix(const dspark_qweight_t &w) {
    if (w.n < 1 || w.n > DSPARK_QLINEAR_MAX_DIM || !ok_dim(w.k)) return DSPARK_ERR_SHAPE;
    if (!w.codes || !w.scales) return DSPARK_ERR_NULL;
    return ok16(w.codes) && ok4(w.scales) ? DSPARK_OK : DSPARK_ERR_ALIGN;
}
dspark_status check_source(const void *x, int type, int64_t stride, int k) {
    if (type != DSPARK_ENTRY_BF16 && type != DSPARK_ENTRY_FP32) return DSPARK_ERR_UNSUPPORTED;
    if (stride < k || stride > kMaxStride) return DSPARK_ERR_SHAPE;
    if (!x) return DSPARK_ERR_NULL;
    return ok16(x) && stride % (type == DSPARK_ENTRY_BF16 ? 8 : 4) == 0 ? DSPARK_OK : DSPARK_ERR_ALIGN;
}

Span codes_of(const dspark_qrows_t &x) { return {x.codes, (unsigned)x.k, (unsigned)x.k, (unsigned)x.rows}; }
Span codes_of(const dspark_qweight_t &w) { return {w.codes, (unsigned)w.k, (unsigned)w.k, (unsigned)w.n}; }
unsigned long long blocks(int d) { return (d + kQlBlock - 1) / kQlBlock; }
Span scales_of(const dspark_qrows_t &x) { return {x.scales, 4ull * x.rows, 4ull * x.scale_stride, blocks(x.k)}; }
Span scales_of(const dspark_qweight_t &w) { return {w.scales, 4 * blocks(w.k), 4 * blocks(w.k), blocks(w.n)}; }
template <typename T>
bool overlaps(const Span &a, const T &x) {  // either part of x
    return overlap(a, codes_of(x)) || overlap(a, scales_of(x));
}

Span source(const void *at, int type, int64_t stride, int rows, int k) {
    const unsigned long long size = type == DSPARK_ENTRY_BF16 ? 2 : 4;
    return {at, k * size, stride * size, (unsigned)rows};
}

dspark_status quantise_matrix(const void *w, int type, int64_t stride, const dspark_qweight_t &out, cudaStream_t st) {
    dspark_status s = check_matrix(out);
    if (s == DSPARK_OK) s = check_source(w, type, stride, out.k);
    if (s != DSPARK_OK) return s;
    if (overlaps(source(w, type, stride, out.n, out.k), out) || overlap(codes_of(out), scales_of(out))) return DSPARK_ERR_SHAPE;
    return done(type == DSPARK_ENTRY_BF16 ? launch_weight<__nv_bfloat16>(w, stride, out, st) : launch_weight<float>(w, stride, out, st));
}

// Up to 64 rows the weights stream past the rows, above the rows are the tensor core's lanes. 64 rows, one against the
// other, us: 12288 outputs x 576 inputs 5.4 and 9.3, 1808 x 720 6.1 and 7.1, 1024 x 512 4.9 and 6.3, 576 x 14336 9.2 and 33.1,
// 14336 x 7168 21.2 and 30.2. What the rule does not know: with few outputs and long rows, where pairs of CTAs are idle,
// calls of 64 rows each would be faster up to 192 rows (576 x 14336, us, as it is and in such calls: 65 rows 35.2 and
// 16.1, 128 35.3 and 19.0, 192 34.9 and 27.9, 256 35.0 and 37.0).
dspark_status product(const QlParams &p, bool gated, const dspark_qrows_t *x, const dspark_qweight_t *w0,
                      const dspark_qweight_t *w1, cudaStream_t st) {
    const QlPlan plan = p.M <= 64 ? plan_qgemm_few(p, gated) : plan_qgemm(p, gated);
    if (plan.error != cudaSuccess) return done(plan.error);
    return done(p.M <= 64 ? launch_qgemm_few(p, gated, *x, *w0, *w1, plan, st) : launch_qgemm(p, gated, *x, *w0, *w1, plan, st));
}

}  // namespace

extern "C" {

dspark_status dspark_qlinear_quantise(const void *x, int x_type, int64_t x_stride, const dspark_qrows_t *out, void *stream) {
    dspark_status s = check_rows(out);
    if (s != DSPARK_OK || out->rows == 0) return s;
    s = check_source(x, x_type, x_stride, out->k);
    if (s != DSPARK_OK) return s;
    if (overlaps(source(x, x_type, x_stride, out->rows, out->k), *out) || overlap(codes_of(*out), scales_of(*out))) return DSPARK_ERR_SHAPE;
    const int sms = current_sms();
    if (sms < 1) return DSPARK_ERR_CUDA;
    return done(x_type == DSPARK_ENTRY_BF16 ? launch_rows<__nv_bfloat16>(x, x_stride, *out, sms, (cudaStream_t)stream)
                                            : launch_rows<float>(x, x_stride, *out, sms, (cudaStream_t)stream));
}

dspark_status dspark_qlinear_quantise_weight(const void *w, int w_type, int64_t w_stride, const dspark_qweight_t *out,
                                             void *stream) {
    const dspark_status s = check_weight(out);
    return s == DSPARK_OK ? quantise_matrix(w, w_type, w_stride, *out, (cudaStream_t)stream) : s;
}

dspark_status dspark_qlinear_quantise_matrix(const void *w, int w_type, int64_t w_stride, int n, int k, void *codes, float *scales,
                                             void *stream) {
    return quantise_matrix(w, w_type, w_stride, dspark_qweight_t{n, k, codes, scales}, (cudaStream_t)stream);
}

dspark_status dspark_qlinear_matmul(const dspark_qrows_t *x, const dspark_qweight_t *w, const float *add, int64_t add_stride,
                                    void *y, int y_type, int64_t y_stride, void *ws, size_t ws_bytes, void *stream) {
    dspark_status s = check_rows(x);
    if (s == DSPARK_OK) s = check_weight(w);
    if (s != DSPARK_OK) return s;
    if (y_type != DSPARK_ENTRY_BF16 && y_type != DSPARK_ENTRY_FP32) return DSPARK_ERR_UNSUPPORTED;
    if (x->k != w->k || y_stride < w->n || y_stride > kMaxStride || (add && (add_stride < w->n || add_stride > kMaxStride)))
        return DSPARK_ERR_SHAPE;
    if (!ws || ws_bytes < DSPARK_QLINEAR_WS_BYTES) return DSPARK_ERR_WORKSPACE;
    if (!ok16(ws)) return DSPARK_ERR_ALIGN;
    if (x->rows == 0) return DSPARK_OK;
    if (!y) return DSPARK_ERR_NULL;
    if (!ok16(y) || !ok16(add) || y_stride % (y_type == DSPARK_ENTRY_BF16 ? 8 : 4) || (add && add_stride % 4)) return DSPARK_ERR_ALIGN;
    const Span out = source(y, y_type, y_stride, x->rows, w->n);
    if (overlaps(out, *x) || overlaps(out, *w)) return DSPARK_ERR_SHAPE;
    // the residual may be y itself, element for element, and nothing else that overlaps it
    if (add && !((const void *)add == y && y_type == DSPARK_ENTRY_FP32 && add_stride == y_stride) &&
        overlap(out, source(add, DSPARK_ENTRY_FP32, add_stride, x->rows, w->n)))
        return DSPARK_ERR_SHAPE;
    QlParams p;
    memset(&p, 0, sizeof(p));
    p.M = x->rows;
    p.N = w->n;
    p.KB = (int)blocks(x->k);
    p.sx = x->scales;
    p.sx_stride = x->scale_stride;
    p.sw[0] = p.sw[1] = w->scales;
    p.add = add;
    p.add_stride = add_stride;
    p.y = y;
    p.y_fp32 = y_type == DSPARK_ENTRY_FP32;
    p.y_stride = y_stride;
    p.err = (int *)ws;
    return product(p, false, x, w, w, (cudaStream_t)stream);
}

dspark_status dspark_qlinear_gated(const dspark_qrows_t *x, const dspark_qweight_t *gate, const dspark_qweight_t *up,
                                   const dspark_qrows_t *h, void *ws, size_t ws_bytes, void *stream) {
    dspark_status s = check_rows(x);
    if (s == DSPARK_OK) s = check_weight(gate);
    if (s == DSPARK_OK) s = check_weight(up);
    if (s == DSPARK_OK) s = check_rows(h);
    if (s != DSPARK_OK) return s;
    if (x->k != gate->k || x->k != up->k || gate->n != up->n || h->k != gate->n || h->rows != x->rows) return DSPARK_ERR_SHAPE;
    if (!ws || ws_bytes < DSPARK_QLINEAR_WS_BYTES) return DSPARK_ERR_WORKSPACE;
    if (!ok16(ws)) return DSPARK_ERR_ALIGN;
    if (x->rows == 0) return DSPARK_OK;
    const Span hc = codes_of(*h), hs = scales_of(*h);
    if (overlap(hc, hs) || overlaps(hc, *x) || overlaps(hs, *x) || overlaps(hc, *gate) || overlaps(hs, *gate) || overlaps(hc, *up) ||
        overlaps(hs, *up))
        return DSPARK_ERR_SHAPE;
    QlParams p;
    memset(&p, 0, sizeof(p));
    p.M = x->rows;
    p.N = gate->n;
    p.KB = (int)blocks(x->k);
    p.sx = x->scales;
    p.sx_stride = x->scale_stride;
    p.sw[0] = gate->scales;
    p.sw[1] = up->scales;
    p.h = (uint8_t *)h->codes;
    p.sh = h->scales;
    p.sh_stride = h->scale_stride;
    p.err = (int *)ws;
    return product(p, true, x, gate, up, (cudaStream_t)stream);
}

}  // extern "C"
