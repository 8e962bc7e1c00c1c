// Attention over the 8-bit latent cache (include/dspark.h, call 9): the combine of
// split items, and the launches.
#include <math.h>

#include "qattn.cuh"

namespace ds {

DS_DEVINL float qa_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------------------
// Combine: the rows of items that were split, one warp per two rows and 128
// columns (all columns at the narrower widths), partials in CTA order. The warp's
// lanes hold the partials' weights; sixteen partials are in flight, the first of
// them requested together with the weights. Bound: latency and L2 (the
// partials were just written): 15 MB of partials (a block of 7 x 64 rows in 16
// pieces each) add about 5 us to the attention.
// ---------------------------------------------------------------------------
constexpr int kQaCombineThreads = 256;
// Partials are weighed by 2^(their reference - the largest + 20). A piece's sum may lie 2^60 above its reference
// (scores that rose behind its first chunk) or below it (pages of scale 2^60), so a piece whose reference is 2^-126 of
// the largest one can still count; with 2^20 more a flushed weight stands for less than 2^-25 of the row's sum a token.
// The most that a sum can reach is then 2^(70 + 31 + 20), an element of O over 2^31 tokens.
constexpr float kQaHeadroom = 20.f;

// A task of the combine: a pair of rows and up to 128 columns of one split item.
template <int DV>
struct QaTask {
    static constexpr int kCols = DV < 128 ? DV : 128, kSub = DV / kCols, kRows = 2;
    const QaParams &p;
    const QaSplit sp;
    const int c, n, sub, row0, lane;  // the item's first CTA and its pieces
    const bool on;
    const float *src;
    DS_DEVINL QaTask(const QaParams &p_, const QaSplit *list, const int *first, int task, int lane_)
        : p(p_), sp(list[task / kSub / (kQaTile / kRows)]), c(first[task / kSub / (kQaTile / kRows)]), n(sp.c_hi - c + 1),
          sub(task % kSub), row0(task / kSub % (kQaTile / kRows) * kRows), lane(lane_), on(4 * lane_ < kCols),
          src(p_.part_o + (size_t)row0 * DV + sub * kCols + 4 * lane_) {}
    DS_DEVINL size_t slot(int k) const { return (size_t)(k == 0 ? sp.lo_slot : 2 * (c + k)); }
    DS_DEVINL float4 fetch(int k, int i) const {
        return on && k < n ? __ldcg((const float4 *)(src + slot(k) * (kQaTile * DV) + i * DV)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // reference and sum, lane = partial
    DS_DEVINL float2 stats(int k0, int i) const {
        return k0 + lane < n ? __ldcg(&p.part_ml[slot(k0 + lane) * kQaTile + row0 + i]) : make_float2(-INFINITY, 0.f);
    }
    // l: to be summed over the lanes
    DS_DEVINL void store(int i, const float4 &o, float m, float l) const {
        const float sum = warp_sum(l);
        const float inv = isnan(sum) ? sum : sum > 0.f ? 1.f / sum : 0.f;
        const int r = sp.r0 + row0 + i, tq = (int)QaWork::token(p, r), hd = r - tq * p.H, tok = sp.q0 + tq;
        if (on) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
            uint2 u;
            u.x = *(const uint32_t *)&lo;
            u.y = *(const uint32_t *)&hi;
            *(uint2 *)(p.o + (size_t)tok * p.o_stride + (size_t)hd * DV + sub * kCols + 4 * lane) = u;
        }
        if (p.lse && sub == 0 && lane == 0)
            p.lse[(size_t)tok * p.H + hd] = isnan(sum) ? sum : sum > 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    static DS_DEVINL float reference(float m) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
        return m == -INFINITY ? 0.f : m - kQaHeadroom;
    }
    static DS_DEVINL void add(float4 &o, float w, const float4 &v) {
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
    }
};

// Few items, many pieces each: 2, 4 or 8 warps of a block share a task's partials and add up in shared memory, in
// order, over the lists, which `smem` holds.
template <int DV>
DS_DEVINL void qattn_combine_shared(const QaParams &p, const QaSplit *s_list, const int *s_first, int tasks,
                                                  int share_log2, void *smem) {
    constexpr int kRows = QaTask<DV>::kRows, kDeep = 16, kWarps = kQaCombineThreads / 32;
    float4(*s_o)[kRows][32] = (float4(*)[kRows][32])smem;
    float(*s_l)[kRows] = (float(*)[kRows])(s_o + kWarps);
    float *s_m = (float *)(s_l + kWarps);
    static_assert(kWarps * (kRows * 32 * 16 + kRows * 4 + 4) <= sizeof(QaSplit) * kQaMaxGrid, "in the list's place");
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int share = 1 << share_log2, part = wid & (share - 1), task = blockIdx.x * (kWarps >> share_log2) + (wid >> share_log2);
    const QaTask<DV> t(p, s_list, s_first, min(task, tasks - 1), lane);
    const int left = task < tasks ? t.sp.rows - t.row0 : 0;
    __syncthreads();  // the lists have been read
    const int k0 = t.n * part >> share_log2, k1 = t.n * (part + 1) >> share_log2;
#pragma unroll 1
    for (int i = 0; i < min(kRows, left); ++i) {
        float4 v[kDeep], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kDeep; ++j) v[j] = t.fetch(k0 + j < k1 ? k0 + j : t.n, i);
        float mx = -INFINITY, l = 0.f;
        for (int k = 0; k < t.n; k += 32) mx = fmaxf(mx, t.stats(k, i).x);
        const float m = t.reference(mx);
        for (int k = k0; k < k1; k += kDeep) {
            if (k > k0) {
#pragma unroll
                for (int j = 0; j < kDeep; ++j) v[j] = t.fetch(k + j < k1 ? k + j : t.n, i);
            }
            const float2 ml = lane < kDeep && k + lane < k1 ? t.stats(k, i) : make_float2(-INFINITY, 0.f);
            const float w = qa_ex2(ml.x - m);
            l += w * ml.y;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) t.add(o, __shfl_sync(~0u, w, j), v[j]);
        }
        s_o[wid][i][lane] = o;
        l = warp_sum(l);
        if (lane == 0) s_l[wid][i] = l;
        if (part == i) s_m[wid] = m;
    }
    __syncthreads();
    if (part < min(kRows, left)) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
        for (int w = wid - part; w < wid - part + share; ++w) {
            t.add(o, 1.f, s_o[w][part][lane]);
            l += s_l[w][part];
        }
        t.store(part, o, s_m[wid], lane == 0 ? l : 0.f);
    }
}

template <int DV, bool FEW>
__global__ void __launch_bounds__(kQaCombineThreads) qattn_combine_kernel(const QaParams p, int ctas) {
    __shared__ alignas(16) QaSplit s_list[kQaMaxGrid];
    __shared__ int s_first[kQaMaxGrid];
    __shared__ unsigned s_mask[kQaMaxGrid / 32];
    constexpr int kSub = QaTask<DV>::kSub;
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
    constexpr int kRows = QaTask<DV>::kRows, kDeep = 16;  // partials in flight (of both rows, or of one when there are many)
    const int tasks = n_split * (kQaTile / kRows) * kSub, warps = gridDim.x * (kQaCombineThreads / 32);
    if constexpr (FEW) {
        int most = 0, share_log2 = 0;  // about a flight of partials a warp
        for (int i = 0; i < n_split; ++i) most = max(most, s_list[i].c_hi - s_first[i] + 1);
        while (share_log2 < 3 && most > kDeep << share_log2 && tasks << (share_log2 + 1) <= warps) ++share_log2;
        if (share_log2 > 0) {
            qattn_combine_shared<DV>(p, s_list, s_first, tasks, share_log2, s_list);
            return;
        }
    }
    for (int task = blockIdx.x * (kQaCombineThreads / 32) + (tid >> 5); task < tasks; task += warps) {
        const QaTask<DV> t(p, s_list, s_first, task, lane);
        const int left = t.sp.rows - t.row0, n = t.n;
        if (left <= 0) continue;
        float4 v[kDeep];
        if (n <= kDeep / 2) {  // both rows at once, everything requested together
            const float2 ml[kRows] = {t.stats(0, 0), t.stats(0, 1)};
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j] = t.fetch(j >> 1, j & 1);
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const float m = t.reference(ml[i].x), w = qa_ex2(ml[i].x - m);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kDeep / 2; ++j) t.add(o, __shfl_sync(~0u, w, j), v[2 * j + i]);
                if (i < left) t.store(i, o, m, w * ml[i].y);
            }
            continue;
        }
#pragma unroll 1
        for (int i = 0; i < min(kRows, left); ++i) {
            float2 ml = t.stats(0, i);
#pragma unroll
            for (int j = 0; j < kDeep; ++j) v[j] = t.fetch(j, i);
            float m = ml.x;
            for (int k0 = 32; k0 < n; k0 += 32) m = fmaxf(m, t.stats(k0, i).x);
            m = t.reference(m);
            float w = qa_ex2(ml.x - m), l = w * ml.y;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < n; k += kDeep) {
                if (k > 0) {
#pragma unroll
                    for (int j = 0; j < kDeep; ++j) v[j] = t.fetch(k + j, i);
                    if ((k & 31) == 0) {
                        ml = t.stats(k, i);
                        w = qa_ex2(ml.x - m);
                        l += w * ml.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < kDeep; ++j) t.add(o, __shfl_sync(~0u, w, (k + j) & 31), v[j]);
            }
            t.store(i, o, m, l);
        }
    }
}

template <int DV>
static cudaError_t combine(const QaParams &p, int grid, int num_sms, cudaStream_t st) {
    // A bound on the items, and one on an item's pieces: with up to four items of more than sixteen pieces, warps share a
    // task (one token of 64 heads over 40000 tokens 45 -> 27 us, two requests 38 -> 30, four of 30000 tokens 38 either
    // way). The form without that is the faster one for everything else (32 requests 57 against 60 us, a block of 7 tokens
    // over 4096 21.2 against 22). The lengths are on the device: a short request under a table of more than 32 pages pays for
    // the first form (one token over 100 tokens: 16.3 us, under a narrower table 14.1).
    const long long rows = (long long)p.total_q * p.H, items = (rows + (long long)min(p.bs, p.total_q) * (kQaTile - 1)) / kQaTile;
    const bool few = items <= 4 && p.max_pages > 2 * 16;
    return few ? launch_pdl(qattn_combine_kernel<DV, true>, dim3(2 * num_sms), dim3(kQaCombineThreads), 0, st, p, grid)
               : launch_pdl(qattn_combine_kernel<DV, false>, dim3(2 * num_sms), dim3(kQaCombineThreads), 0, st, p, grid);
}

cudaError_t launch_qattn(const QaParams &p, int kv_lora, int num_sms, cudaStream_t st) {
    const int grid = min(num_sms, kQaMaxGrid);
    const cudaError_t e = launch_qattn_tc(p, kv_lora, grid, st);
    if (e != cudaSuccess) return e;
    switch (kv_lora) {
        case 512: return combine<512>(p, grid, num_sms, st);
        case 256: return combine<256>(p, grid, num_sms, st);
        case 128: return combine<128>(p, grid, num_sms, st);
        default: return combine<64>(p, grid, num_sms, st);
    }
}

}  // namespace ds
