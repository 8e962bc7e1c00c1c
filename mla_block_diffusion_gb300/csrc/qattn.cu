// Attention over the 8-bit latent cache (include/dspark.h, call 9): the kernel
// for the smaller latent widths, and the combine of split items.
#include <math.h>

#include "e4m3.cuh"
#include "qattn.cuh"

namespace ds {

DS_DEVINL void ldsm4(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
DS_DEVINL void ldsm4t(uint32_t (&r)[4], const void *p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p)));
}
DS_DEVINL void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DS_DEVINL float qa_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------
// The smaller widths (256 + 32, 128 + 32, 64 + 16), mma.sync m16n8k16 in f16.
//
// A CTA of 8 warps holds 64 query rows: warp (w & 3) 16 of them, w >> 2 one half
// of the output columns (both halves compute the scores of their rows). E4M3
// codes are exact in f16; a query row is scaled by a power of two so that its
// largest magnitude lies in [2^7, 2^8), where a bf16 significand is exact in
// f16 down to 2^-22 of it. Online softmax in the log2 domain: the weight that
// meets a code is w = 2^(s + e - m) with e the page scale's exponent and m the
// row's running maximum of s + e, so that codes are used as they are; the row
// sum adds w * 2^-e. Weights are rounded to f16 (2^-12), sums are fp32.
// ---------------------------------------------------------------------------
template <int D, int DV>
struct QgCfg {
    static constexpr int kThreads = 256;
    static constexpr int kRow = D * 2 + 16;                 // bytes per shared row: an odd number of 16-byte pieces
    static constexpr int kStages = 4;                       // pages of raw codes in flight
    static constexpr int kRaw = kQcPage * D;
    static constexpr int kSmem = (64 + kQcPage) * kRow + kStages * kRaw + 64 * 8;
    static constexpr int kCtas = DV < 256 ? 2 : 1;          // resident per SM
    static constexpr int kPieces = kQcPage * D / 16;        // 16-byte pieces of a page
    static constexpr int kPer = (kPieces + kThreads - 1) / kThreads;
    static_assert((kRow / 16) % 2 == 1, "conflict-free row stride");
    static_assert(kSmem >= QaWork<64, 64>::kScratch, "scratch of the work division");
};

template <int D, int DV>
__global__ void __launch_bounds__(QgCfg<D, DV>::kThreads, QgCfg<D, DV>::kCtas) qattn_any_kernel(const QaParams p) {
    using C = QgCfg<D, DV>;
    using W = QaWork<kQaTile, kQcPage>;
    extern __shared__ __align__(16) uint8_t qg_smem[];
    uint8_t *sQ = qg_smem, *sK = sQ + 64 * C::kRow, *sR = sK + kQcPage * C::kRow;
    float *s_c = (float *)(sR + C::kStages * C::kRaw);  // score factor of every row (NaN: a non-finite query)
    int *s_lim = (int *)(s_c + 64);                  // tokens every row sees
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rg = warp & 3, half = warp >> 2;
    const int cta = blockIdx.x, grid = gridDim.x;
    constexpr int NV = DV / 2 / 8;                   // output column tiles of a warp

    pdl_trigger();
    pdl_wait();
    W wk;
    wk.find(p, cta, grid, qg_smem);
    long long left = wk.end - wk.begin, unit = wk.begin;
    QaSplit sp;
    sp.q0 = sp.r0 = sp.rows = sp.lo_slot = 0;
    sp.c_hi = -1;
    int slot = 2 * cta;
    for (; left > 0; slot = 2 * cta + 1) {
        const QaItem it = wk.item;
        const int take = (int)min((long long)(it.chunks - wk.off), left);
        const bool first = wk.off == 0, whole = first && take == it.chunks;
        if (first && !whole) {
            sp.q0 = it.q0;
            sp.r0 = it.t * kQaTile;
            sp.rows = it.nq * p.H - sp.r0;
            sp.lo_slot = slot;
            sp.c_hi = wk.last_cta(unit);
        }
        const int r0 = it.t * kQaTile, R = it.nq * p.H;
        __syncthreads();
        // query rows as f16
        for (int r = warp; r < 64; r += 8) {
            const bool in = r0 + r < R;
            const int tok = in ? (int)W::token(p, r0 + r) : 0, hd = in ? r0 + r - tok * p.H : 0;
            const __nv_bfloat16 *src = p.q + (size_t)(it.q0 + tok) * p.q_stride + (size_t)hd * D;
            uint32_t mx = 0;
            uint4 v[(D / 8 + 31) / 32];
#pragma unroll
            for (int j = 0; j < (D / 8 + 31) / 32; ++j) {
                const int k = lane + 32 * j;
                v[j] = in && k < D / 8 ? __ldg((const uint4 *)src + k) : make_uint4(0, 0, 0, 0);
                const uint32_t *u = (const uint32_t *)&v[j];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx = max(mx, max((u[i] << 16) & 0x7fffffffu, u[i] & 0x7fff0000u));
            }
            mx = __reduce_max_sync(~0u, mx);
            const bool bad = mx >= 0x7f800000u;
            // 2^a times the largest magnitude lies in [2^7, 2^8)
            int a = mx < 0x00800000u ? 0 : 7 - ((int)(mx >> 23) - 127);
            a = min(a, 100);
            const float f = qc_pow2(a);
#pragma unroll
            for (int j = 0; j < (D / 8 + 31) / 32; ++j) {
                const int k = lane + 32 * j;
                if (k < D / 8) {
                    const uint32_t *u = (const uint32_t *)&v[j];
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        h[i] = bad ? 0u : f32x2_to_f16x2(__uint_as_float(u[i] << 16) * f, __uint_as_float(u[i] & 0xffff0000u) * f);
                    *(uint4 *)(sQ + r * C::kRow + k * 16) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            if (lane == 0) {
                s_c[r] = bad ? __uint_as_float(0x7fffffffu) : qc_pow2(-a) * p.scale_log2;
                s_lim[r] = in ? W::sees(p, it.nq, it.len, tok) : 0;
                if (bad && first) set_error(p.err, DSPARK_ERR_BAD_INPUT);
            }
        }
        float oacc[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) oacc[i][j] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        // Pages: every thread copies its pieces of the raw codes into a ring three pages ahead, and
        // decodes the same pieces for all, so the copies need no barrier of their own. Page numbers
        // and scales: 32 pages at a time in the lanes of every warp, one block ahead.
        const int npages = min((it.len + kQcPage - 1) / kQcPage, wk.off + take);
        const int32_t *row = p.page_table + (size_t)it.b * p.max_pages;
        auto page = [&](int c) {
            int pg = c < npages ? row[c] : 0;
            if (pg < 0 || pg >= p.n_pages) {
                set_error(p.err, DSPARK_ERR_OOB);
                pg = 0;
            }
            return pg;
        };
        auto exponent = [&](int c, int pg) {
            int x = 0;
            if (c < npages && !qc_scale_exponent(p.scales[pg], &x)) set_error(p.err, DSPARK_ERR_BAD_INPUT);
            return x;
        };
        int pg_l = page(wk.off + lane), pg_n = 0, ex = exponent(wk.off + lane, pg_l), ex_n = 0;  // loads run ahead: pg_l is their block
        auto load = [&](int i) {  // page wk.off + i into stage i % kStages
            if (i > 0 && (i & 31) == 0) pg_l = pg_n;
            const int c = wk.off + i, pg = __shfl_sync(~0u, pg_l, i & 31);
            if (c < npages) {
                const uint4 *src = (const uint4 *)(p.codes + (size_t)pg * kQcPage * D);
                const int used = min(kQcPage, it.len - c * kQcPage) * (D / 16);  // pieces of cached tokens
                const uint32_t dst = smem_u32(sR + (i % C::kStages) * C::kRaw);
#pragma unroll
                for (int j = 0; j < C::kPer; ++j) {
                    const int k = tid + j * C::kThreads;
                    if (k < C::kPieces)  // zeros past the cached tokens
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + k * 16), "l"(src + (k < used ? k : 0)),
                                     "r"(k < used ? 16 : 0)
                                     : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int i = 0; i < C::kStages - 1; ++i) load(i);
#pragma unroll 1
        for (int i = 0; i < take; ++i) {
            const int c = wk.off + i, base = c * kQcPage;
            if ((i & 31) == 0) {
                if (i > 0) ex = ex_n;
                pg_n = page(wk.off + i + 32 + lane);
            }
            if ((i & 31) == 16) ex_n = exponent(wk.off + i + 16 + lane, pg_n);
            const int e = __shfl_sync(~0u, ex, i & 31);
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
            __syncthreads();  // the page before has been read
            if (base < it.len) {
                const uint8_t *raw = sR + (i % C::kStages) * C::kRaw;
#pragma unroll
                for (int j = 0; j < C::kPer; ++j) {
                    const int k = tid + j * C::kThreads;
                    if (k < C::kPieces) {
                        const uint4 v = *(const uint4 *)(raw + k * 16);
                        const uint32_t *u = (const uint32_t *)&v;
                        uint8_t *dst = sK + (k / (D / 16)) * C::kRow + (k % (D / 16)) * 32;
                        uint32_t h[8];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            h[2 * x] = e4m3x2_to_f16x2_(u[x] & 0xffffu);
                            h[2 * x + 1] = e4m3x2_to_f16x2_(u[x] >> 16);
                        }
                        *(uint4 *)dst = make_uint4(h[0], h[1], h[2], h[3]);
                        *(uint4 *)(dst + 16) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                }
            }
            load(i + C::kStages - 1);
            __syncthreads();
            if (base >= it.len) continue;
            // scores of 16 rows x 64 tokens
            float s[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                ldsm4(a, sQ + (16 * rg + (lane & 15)) * C::kRow + k * 32 + (lane >> 4) * 16);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    uint32_t b[4];
                    ldsm4(b, sK + (16 * n + (lane & 7) + ((lane >> 4) << 3)) * C::kRow + k * 32 + ((lane >> 3) & 1) * 16);
                    mma_f16_16816(s[2 * n], a, b[0], b[1]);
                    mma_f16_16816(s[2 * n + 1], a, b[2], b[3]);
                }
            }
            const float fe = (float)e, scale = qc_pow2(e), unscale = qc_pow2(-e);
            uint32_t pr[8][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // rows lane / 4 and lane / 4 + 8
                const int row = 16 * rg + (lane >> 2) + 8 * h;
                const float cf = s_c[row] * scale;
                const int lim = s_lim[row] - base;
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < 8; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = 8 * n + 2 * (lane & 3) + j;
                        float &x = s[n][2 * h + j];
                        x = col < lim ? x * cf + fe : -INFINITY;
                        mx = fmaxf(mx, x);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                const float mn = fmaxf(m[h], mx), mb = mn == -INFINITY ? 0.f : mn;
                const float corr = qa_ex2(m[h] - mb);
                m[h] = mn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float w0 = qa_ex2(s[n][2 * h] - mb), w1 = qa_ex2(s[n][2 * h + 1] - mb);
                    sum += w0 + w1;
                    pr[n][h] = f32x2_to_f16x2(w0, w1);
                }
                l[h] = l[h] * corr + sum * unscale;
                if (__any_sync(~0u, corr != 1.f)) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        oacc[i][2 * h] *= corr;
                        oacc[i][2 * h + 1] *= corr;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a[4] = {pr[2 * k][0], pr[2 * k][1], pr[2 * k + 1][0], pr[2 * k + 1][1]};
#pragma unroll
                for (int n = 0; n < NV / 2; ++n) {
                    uint32_t b[4];
                    ldsm4t(b, sK + (16 * k + (lane & 15)) * C::kRow + (half * (DV / 2) + 16 * n) * 2 + (lane >> 4) * 16);
                    mma_f16_16816(oacc[2 * n], a, b[0], b[1]);
                    mma_f16_16816(oacc[2 * n + 1], a, b[2], b[3]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(~0u, l[h], 1);
            l[h] += __shfl_xor_sync(~0u, l[h], 2);
            const int row = 16 * rg + (lane >> 2) + 8 * h, r = r0 + row;
            if (whole) {
                if (r < R) {
                    const bool bad = isnan(s_c[row]);
                    const float inv = bad ? __uint_as_float(0x7fffffffu) : l[h] > 0.f ? 1.f / l[h] : 0.f;
                    const int tk = (int)W::token(p, r), tok = it.q0 + tk, hd = r - tk * p.H;
                    __nv_bfloat16 *dst = p.o + (size_t)tok * p.o_stride + (size_t)hd * DV + half * (DV / 2) + 2 * (lane & 3);
#pragma unroll
                    for (int n = 0; n < NV; ++n)
                        *(__nv_bfloat162 *)(dst + 8 * n) = __floats2bfloat162_rn(oacc[n][2 * h] * inv, oacc[n][2 * h + 1] * inv);
                    if (p.lse && half == 0 && (lane & 3) == 0)
                        p.lse[(size_t)tok * p.H + hd] = bad ? __uint_as_float(0x7fffffffu)
                                                      : l[h] > 0.f ? (m[h] + log2f(l[h])) * 0.6931471805599453f : -INFINITY;
                }
            } else {
                const bool bad = isnan(s_c[row]);
                float *dst = p.part_o + ((size_t)slot * kQaTile + row) * DV + half * (DV / 2) + 2 * (lane & 3);
#pragma unroll
                for (int n = 0; n < NV; ++n) *(float2 *)(dst + 8 * n) = make_float2(oacc[n][2 * h], oacc[n][2 * h + 1]);
                if (half == 0 && (lane & 3) == 0)
                    p.part_ml[slot * kQaTile + row] = make_float2(bad ? 0.f : m[h], bad ? __uint_as_float(0x7fffffffu) : l[h]);
            }
        }
        left -= take;
        unit += it.chunks - wk.off;
        if (left > 0) wk.next(p);
    }
    if (tid == 0) p.split[cta] = sp;
}

// ---------------------------------------------------------------------------
// Combine: the rows of items that were split, one warp per two rows and 128
// columns (all columns at the narrower widths), partials in CTA order. The warp's
// lanes hold the partials' weights; sixteen partials are in flight, the first of
// them requested together with the weights. Bound: latency and L2 (the
// partials were just written).
// ---------------------------------------------------------------------------
constexpr int kQaCombineThreads = 256;

template <int DV>
__global__ void __launch_bounds__(kQaCombineThreads) qattn_combine_kernel(const QaParams p, int ctas) {
    __shared__ QaSplit s_list[kQaMaxGrid];
    __shared__ int s_first[kQaMaxGrid];
    __shared__ unsigned s_mask[kQaMaxGrid / 32];
    constexpr int kCols = DV < 128 ? DV : 128, kSub = DV / kCols;
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_trigger();
    pdl_wait();
    // the split items in CTA order (every block lists them alike)
    QaSplit sp_own[kQaMaxGrid / kQaCombineThreads];
#pragma unroll
    for (int i = 0; i < kQaMaxGrid / kQaCombineThreads; ++i) {
        const int c = tid + i * kQaCombineThreads;
        sp_own[i].c_hi = -1;
        if (c < ctas) sp_own[i] = p.split[c];
        const unsigned mask = __ballot_sync(~0u, sp_own[i].c_hi >= 0);
        if (lane == 0) s_mask[c / 32] = mask;
    }
    __syncthreads();
    int n_split = 0;
    for (int w = 0; w < kQaMaxGrid / 32; ++w) {
        const unsigned mask = s_mask[w];
#pragma unroll
        for (int i = 0; i < kQaMaxGrid / kQaCombineThreads; ++i) {
            const int c = tid + i * kQaCombineThreads;
            if (c / 32 == w && sp_own[i].c_hi >= 0) {
                const int at = n_split + __popc(mask & ((1u << lane) - 1u));
                s_list[at] = sp_own[i];
                s_first[at] = c;
            }
        }
        n_split += __popc(mask);
    }
    __syncthreads();
    constexpr int kRows = 2, kDeep = 16;  // rows of a task, partials in flight (of both rows, or of one when there are many)
    const int tasks = n_split * (kQaTile / kRows) * kSub, warps = gridDim.x * (kQaCombineThreads / 32);
    const bool on = 4 * lane < kCols;
    for (int task = blockIdx.x * (kQaCombineThreads / 32) + (tid >> 5); task < tasks; task += warps) {
        const int sub = task % kSub, row0 = task / kSub % (kQaTile / kRows) * kRows, li = task / kSub / (kQaTile / kRows);
        const QaSplit sp = s_list[li];
        const int left = sp.rows - row0;
        if (left <= 0) continue;
        const int c = s_first[li], n = sp.c_hi - c + 1;
        auto slot = [&](int k) { return (size_t)(k == 0 ? sp.lo_slot : 2 * (c + k)); };
        const float *src = p.part_o + (size_t)row0 * DV + sub * kCols + 4 * lane;
        auto fetch = [&](int k, int i) {
            return on && k < n ? __ldcg((const float4 *)(src + slot(k) * (kQaTile * DV) + i * DV)) : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        // reference and sum, lane = partial
        auto stats = [&](int k0, int i) {
            return k0 + lane < n ? __ldcg(&p.part_ml[slot(k0 + lane) * kQaTile + row0 + i]) : make_float2(-INFINITY, 0.f);
        };
        auto store = [&](int i, const float4 &o, float m, float l) {
            const float sum = warp_sum(l);
            const float inv = isnan(sum) ? sum : sum > 0.f ? 1.f / sum : 0.f;
            const int r = sp.r0 + row0 + i, tq = (int)QaWork<kQaTile, kQcPage>::token(p, r), hd = r - tq * p.H, tok = sp.q0 + tq;
            if (on) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
                uint2 u;
                u.x = *(const uint32_t *)&lo;
                u.y = *(const uint32_t *)&hi;
                *(uint2 *)(p.o + (size_t)tok * p.o_stride + (size_t)hd * DV + sub * kCols + 4 * lane) = u;
            }
            if (p.lse && sub == 0 && lane == 0)
                p.lse[(size_t)tok * p.H + hd] = isnan(sum) ? sum : sum > 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        };
        auto reference = [&](float m) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
            return m == -INFINITY ? 0.f : m;
        };
        auto add = [&](float4 &o, float w, const float4 &v) {
            o.x += w * v.x;
            o.y += w * v.y;
            o.z += w * v.z;
            o.w += w * v.w;
        };
        float4 v[kDeep];
        if (n <= kDeep / 2) {  // both rows at once, everything requested together
            const float2 ml[kRows] = {stats(0, 0), stats(0, 1)};
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j] = fetch(j >> 1, j & 1);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float m = reference(ml[i].x), w = qa_ex2(ml[i].x - m);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kDeep / 2; ++j) add(o, __shfl_sync(~0u, w, j), v[2 * j + i]);
                if (i < left) store(i, o, m, w * ml[i].y);
            }
            continue;
        }
#pragma unroll 1
        for (int i = 0; i < min(kRows, left); ++i) {
            float2 ml = stats(0, i);
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j] = fetch(j, i);
            float m = ml.x;
            for (int k0 = 32; k0 < n; k0 += 32) m = fmaxf(m, stats(k0, i).x);
            m = reference(m);
            float w = qa_ex2(ml.x - m), l = w * ml.y;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < n; k += kDeep) {
                if (k > 0) {
#pragma unroll
                    for (int j = 0; j < kDeep; ++j) v[j] = fetch(k + j, i);
                    if ((k & 31) == 0) {
                        ml = stats(k, i);
                        w = qa_ex2(ml.x - m);
                        l += w * ml.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < kDeep; ++j) add(o, __shfl_sync(~0u, w, (k + j) & 31), v[j]);
            }
            store(i, o, m, l);
        }
    }
}

template <int DV>
static cudaError_t combine(const QaParams &p, int grid, int num_sms, cudaStream_t st) {
    return launch_pdl(qattn_combine_kernel<DV>, dim3(2 * num_sms), dim3(kQaCombineThreads), 0, st, p, grid);
}

template <int D, int DV>
static cudaError_t any_width(const QaParams &p, int num_sms, cudaStream_t st) {
    using C = QgCfg<D, DV>;
    static bool attr = false;
    if (!attr) {
        const cudaError_t e = cudaFuncSetAttribute(qattn_any_kernel<D, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        attr = true;
    }
    const int grid = min(num_sms * C::kCtas, kQaMaxGrid);
    const cudaError_t e = launch_pdl(qattn_any_kernel<D, DV>, dim3(grid), dim3(C::kThreads), (size_t)C::kSmem, st, p);
    return e != cudaSuccess ? e : combine<DV>(p, grid, num_sms, st);
}

cudaError_t launch_qattn(const QaParams &p, int kv_lora, int, int num_sms, cudaStream_t st) {
    switch (kv_lora) {
        case 512: {
            const int grid = min(num_sms, kQaMaxGrid);
            const cudaError_t e = launch_qattn_tc(p, grid, st);
            return e != cudaSuccess ? e : combine<512>(p, grid, num_sms, st);
        }
        case 256: return any_width<288, 256>(p, num_sms, st);
        case 128: return any_width<160, 128>(p, num_sms, st);
        case 64: return any_width<80, 64>(p, num_sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ds
