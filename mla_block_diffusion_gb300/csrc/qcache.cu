// The 8-bit latent cache: host entry points, the page plan and the quantising
// append (include/dspark.h, calls 7 and 8).
#include <math.h>
#include <string.h>

#include "e4m3.cuh"
#include "internal.h"
#include "per_device.h"
#include "qcache.h"

using namespace ds;

namespace ds {

// ---------------------------------------------------------------------------
// Page plan.
//
// Per request: pages it needs, its new tokens, the pages those touch, and the
// pages it gives back; running sums of the four over the requests give every
// place. A growing request is served if its inclusive sums fit, and then all
// growing requests before it are served too, so the exclusive sums of a served
// request are the same whether those not served are counted or not: one scan.
// Sums saturate at 2^30 + 1 (saturating addition of non-negative numbers is
// associative), which no capacity reaches.
//
// Bound: latency (a dependent chain of two loads, a block scan and the search
// of a token's request in shared memory) until the slot maps are long, then
// their stores. Every CTA repeats the scan (up to 1024 requests, four a
// thread) and fills its share of the outputs, so no CTA waits for another. In a graph
// over eight plans in turn: one request 3.6 us, 32 4.6, 500 of 1 to 8192 tokens 7.9, 64
// prompts 5.9 (with L2 flushed before: 5.1, 7.1, 10.5, 7.3); the host call takes 8 to 9.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256;
constexpr int kPlanPer = kQcMaxBs / kPlanThreads;
constexpr unsigned kPlanSat = (1u << 30) + 1;

struct PlanParams {
    dspark_qplan_t p;
    int32_t *page_table;
    int n_pages, max_pages, bs, max_new, max_seg;
    int *err;
};

DS_DEVINL unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kPlanSat); }

struct Sums {
    unsigned need, fresh, seg, give;
};
DS_DEVINL Sums operator+(const Sums &a, const Sums &b) {
    return Sums{sat_add(a.need, b.need), sat_add(a.fresh, b.fresh), sat_add(a.seg, b.seg), sat_add(a.give, b.give)};
}
DS_DEVINL Sums shfl_up(const Sums &a, int d) {
    return Sums{__shfl_up_sync(~0u, a.need, d), __shfl_up_sync(~0u, a.fresh, d), __shfl_up_sync(~0u, a.seg, d),
                __shfl_up_sync(~0u, a.give, d)};
}

// The request whose range of the running sums cu[0 .. bs] holds i < cu[bs].
DS_DEVINL int find_request(const unsigned *cu, int bs, unsigned i) {
    int lo = 0, hi = bs;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) qcache_plan_kernel(const PlanParams a) {
    __shared__ unsigned s_need[kQcMaxBs + 1], s_new[kQcMaxBs + 1], s_seg[kQcMaxBs + 1], s_give[kQcMaxBs + 1];
    __shared__ int s_len[kQcMaxBs], s_want[kQcMaxBs];
    __shared__ Sums s_warp[kPlanThreads / 32];
    __shared__ unsigned s_tot[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first_cta = blockIdx.x == 0;
    pdl_trigger();
    if (tid < 4) s_tot[tid] = 0;
    pdl_wait();

    int head = a.p.ring_state[0], count = a.p.ring_state[1];
    if (head < 0 || head >= a.n_pages || count < 0 || count > a.n_pages) {
        if (first_cta && tid == 0) set_error(a.err, DSPARK_ERR_OOB);
        head = 0;
        count = 0;
    }
    const long long cap = (long long)a.max_pages * kQcPage;
    int len[kPlanPer], want[kPlanPer];
    const int b0 = tid * kPlanPer;
#pragma unroll
    for (int j = 0; j < kPlanPer; ++j) {
        len[j] = b0 + j < a.bs ? a.p.length[b0 + j] : 0;
        want[j] = b0 + j < a.bs ? a.p.want[b0 + j] : 0;
    }
    Sums own[kPlanPer], sum = Sums{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kPlanPer; ++j) {
        if (len[j] < 0 || len[j] > cap || want[j] < 0 || want[j] > cap) {
            if (first_cta) set_error(a.err, DSPARK_ERR_OOB);
            want[j] = len[j];  // stays as it is
        }
        Sums s{0, 0, 0, 0};
        if (want[j] > len[j]) {
            s.need = (unsigned)((want[j] + kQcPage - 1) / kQcPage - (len[j] + kQcPage - 1) / kQcPage);
            s.fresh = min((unsigned)(want[j] - len[j]), kPlanSat);
            s.seg = (unsigned)((want[j] + kQcPage - 1) / kQcPage - len[j] / kQcPage);
        } else if (want[j] < len[j]) {
            s.give = (unsigned)((len[j] + kQcPage - 1) / kQcPage - (want[j] + kQcPage - 1) / kQcPage);
        }
        own[j] = s;
        sum = sum + s;
    }
    Sums inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = shfl_up(inc, d);
        if (lane >= d) inc = inc + o;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    Sums run = Sums{0, 0, 0, 0};
    for (int w = 0; w < warp; ++w) run = run + s_warp[w];
    {
        const Sums o = shfl_up(inc, 1);  // of the lanes before this one
        if (lane > 0) run = run + o;
    }
    Sums last = Sums{0, 0, 0, 0};  // sums up to this thread's last served request
    bool any = false;
#pragma unroll
    for (int j = 0; j < kPlanPer; ++j) {
        const int b = b0 + j;
        if (b < a.bs) {
            s_need[b] = run.need;
            s_new[b] = run.fresh;
            s_seg[b] = run.seg;
            s_give[b] = run.give;
            run = run + own[j];
            bool served = false;
            if (want[j] > len[j]) {
                served = run.need <= (unsigned)count && run.fresh <= (unsigned)a.max_new && run.seg <= (unsigned)a.max_seg;
                if (served) {
                    last = run;
                    any = true;
                }
            }
            s_len[b] = len[j];
            s_want[b] = want[j] > len[j] && !served ? len[j] : want[j];
            if (first_cta) a.p.length_out[b] = s_want[b];
        }
    }
    if (any) {
        atomicMax(&s_tot[0], last.need);
        atomicMax(&s_tot[1], last.fresh);
        atomicMax(&s_tot[2], last.seg);
    }
    if (b0 < a.bs) atomicMax(&s_tot[3], run.give);
    __syncthreads();
    const unsigned t_need = s_tot[0], t_new = s_tot[1], t_seg = s_tot[2], t_give = s_tot[3];
    // places past the served requests hold the totals (a request that is not served spans nothing)
    for (int b = tid; b <= a.bs; b += kPlanThreads) {
        s_need[b] = b < a.bs ? min(s_need[b], t_need) : t_need;
        s_new[b] = b < a.bs ? min(s_new[b], t_new) : t_new;
        s_seg[b] = b < a.bs ? min(s_seg[b], t_seg) : t_seg;
        if (b == a.bs) s_give[b] = t_give;
    }
    __syncthreads();

    const int gt = blockIdx.x * kPlanThreads + tid, gn = gridDim.x * kPlanThreads;
    auto free_page = [&](unsigned i) {  // i-th page from the ring's front
        unsigned at = (unsigned)head + i;
        if (at >= (unsigned)a.n_pages) at -= (unsigned)a.n_pages;
        return a.p.ring[at];
    };
    if (first_cta) {
        for (int b = tid; b <= a.bs; b += kPlanThreads) a.p.cu_new[b] = (int)s_new[b];
        if (tid == 0) {
            const unsigned left = (unsigned)count - t_need;
            unsigned kept = t_give, h = (unsigned)head + t_need;
            if ((unsigned)count + t_give > (unsigned)a.n_pages) {
                set_error(a.err, DSPARK_ERR_OOB);  // more pages given back than the ring lacks
                kept = (unsigned)(a.n_pages - count);
            }
            if (h >= (unsigned)a.n_pages) h -= (unsigned)a.n_pages;
            a.p.ring_state_out[0] = (int)h;
            a.p.ring_state_out[1] = (int)(left + kept);
        }
    }
    // page-table entries of new pages
    for (unsigned i = gt; i < t_need; i += gn) {
        const int b = find_request(s_need, a.bs, i);
        const int at = (s_len[b] + kQcPage - 1) / kQcPage + (int)(i - s_need[b]);
        const int pg = free_page(i);
        if (pg < 0 || pg >= a.n_pages) set_error(a.err, DSPARK_ERR_OOB);
        a.page_table[(size_t)b * a.max_pages + at] = pg;
    }
    // pages given back go behind the ring's last free page
    for (unsigned i = gt; i < t_give; i += gn) {
        if ((unsigned)count + i >= (unsigned)a.n_pages) break;
        const int b = find_request(s_give, a.bs, i);
        const int at = (s_want[b] + kQcPage - 1) / kQcPage + (int)(i - s_give[b]);
        unsigned to = (unsigned)head + (unsigned)count + i;
        if (to >= (unsigned)a.n_pages) to -= (unsigned)a.n_pages;
        const int pg = a.page_table[(size_t)b * a.max_pages + at];
        if (pg < 0 || pg >= a.n_pages) set_error(a.err, DSPARK_ERR_OOB);
        a.p.ring[to] = pg;
    }
    // slots and positions, four tokens a thread
    for (int i0 = 4 * gt; i0 < a.max_new; i0 += 4 * gn) {
        int slot[4], pos[4];
        int b = (unsigned)i0 < t_new ? find_request(s_new, a.bs, (unsigned)i0) : 0;
        int last_at = -1, last_b = -1, pg = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned i = (unsigned)i0 + j;
            slot[j] = -1;
            pos[j] = -1;
            if (i < t_new) {
                while (s_new[b + 1] <= i) ++b;
                pos[j] = s_len[b] + (int)(i - s_new[b]);
                const int at = pos[j] / kQcPage, held = (s_len[b] + kQcPage - 1) / kQcPage;
                if (at != last_at || b != last_b) {
                    pg = at < held ? a.page_table[(size_t)b * a.max_pages + at] : free_page(s_need[b] + (unsigned)(at - held));
                    last_at = at;
                    last_b = b;
                }
                if (pg >= 0 && pg < a.n_pages) slot[j] = pg * kQcPage + pos[j] % kQcPage;
                else set_error(a.err, DSPARK_ERR_OOB);
            }
        }
        if (i0 + 4 <= a.max_new) {
            *(int4 *)(a.p.slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *(int4 *)(a.p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int j = 0; i0 + j < a.max_new; ++j) {
                a.p.slots[i0 + j] = slot[j];
                a.p.positions[i0 + j] = pos[j];
            }
        }
    }
    // first row of every touched page
    for (int s = gt; s <= a.max_seg; s += gn) {
        int row = (int)t_new;
        if ((unsigned)s < t_seg) {
            const int b = find_request(s_seg, a.bs, (unsigned)s);
            const int k = s - (int)s_seg[b];
            row = (int)s_new[b] + (k == 0 ? 0 : (s_len[b] / kQcPage + k) * kQcPage - s_len[b]);
        }
        a.p.seg_row[s] = row;
    }
}

// ---------------------------------------------------------------------------
// Quantising append: one CTA per touched page and layer.
//
// e = the least exponent with amax <= 448 * 2^e over the page's new rows, and
// at least the page's present one if it holds earlier tokens; codes are
// RN(x * 2^-e), exact but for the rounding since 2^-e is a power of two.
// Earlier codes move by whole binades: exact unless they fall below 2^-6.
// Bound: HBM (2 or 4 bytes read and one written per element). Bulk copies bring
// the page's rows into shared memory, where they wait for their maximum: the bytes
// in flight are bounded by shared memory (three bf16 pages of the full width an
// SM), not by registers, and each element is read once. 24 prompts of 700 to 8192
// tokens, bf16: 30 us, 5.4 TB/s of 6.8 (with the rows held in registers 38.6 us,
// read twice 49 us); the narrower widths 19, 12 and 11 us. fp32: 62 us at the full
// width, 4.4 TB/s (a page is 147 KB, one an SM, whose load waits for the conversion of
// the one before), 25, 17 and 12 at the others.
// ---------------------------------------------------------------------------
constexpr int kAppThreads = 384;

struct AppendParams {
    uint8_t *codes[DSPARK_MAX_LAYERS];
    float *scales[DSPARK_MAX_LAYERS];
    const void *entries;
    long long row_stride, layer_stride;
    const int32_t *slots, *seg_row;
    int rows, n_pages;
    int *err;
};

// Elements 2i and 2i + 1 of a 16-byte piece as fp32.
DS_DEVINL float2 pair_of(const uint4 &u, int i, const __nv_bfloat16 *) {
    const uint32_t w = ((const uint32_t *)&u)[i];
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
DS_DEVINL float2 pair_of(const uint4 &u, int i, const float *) {
    const float *f = (const float *)&u;
    return make_float2(f[2 * i], f[2 * i + 1]);
}
// Largest magnitude of a piece, as the bits of an fp32 number (a NaN is above every number).
DS_DEVINL uint32_t amax_of(const uint4 &u, const __nv_bfloat16 *) {
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}
DS_DEVINL uint32_t amax_of(const uint4 &u, const float *) {
    return max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
}
// Two floats to two E4M3 codes (round to nearest even, saturating), even low.
DS_DEVINL uint32_t f32x2_to_e4m3x2(float even, float odd) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(odd), "f"(even));
    return d;
}

// The least e with bits <= 448 * 2^e (448 = 1.75 * 2^8), clamped.
DS_DEVINL int amax_exponent(uint32_t bits) {
    if (bits < 0x00800000u) return -kQcEmax;  // zero or subnormal
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-kQcEmax, min(kQcEmax, e));
}

// n 16-byte pieces of a page's codes move to a scale 2^-d times theirs (d < 0), rounded to nearest even. All
// of a thread's pieces are requested at once: one trip to memory and back, not one for each (32 requests x 5 layers,
// one token each, every page's scale growing: 6.3 us against 7.9; 4.5 when none grows).
template <int D>
DS_DEVINL void move_codes(uint8_t *codes, int n, int d) {
    constexpr int kPer = ((kQcPage - 1) * (D / 16) + kAppThreads - 1) / kAppThreads;
    const float f = qc_pow2(d);
    uint4 v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = threadIdx.x + k * kAppThreads;
        v[k] = i < n ? *(const uint4 *)(codes + (size_t)i * 16) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = threadIdx.x + k * kAppThreads;
        if (i >= n) break;
        uint32_t *w = (uint32_t *)&v[k];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h[2] = {e4m3x2_to_f16x2_(w[j] & 0xffffu), e4m3x2_to_f16x2_(w[j] >> 16)};
            const float2 x = __half22float2(*(const __half2 *)&h[0]), y = __half22float2(*(const __half2 *)&h[1]);
            w[j] = f32x2_to_e4m3x2(x.x * f, x.y * f) | f32x2_to_e4m3x2(y.x * f, y.y * f) << 16;
        }
        *(uint4 *)(codes + (size_t)i * 16) = v[k];
    }
}

// Bulk copy of bytes (16-byte aligned, a multiple of 16) into shared memory.
DS_DEVINL void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppThreads, 2) qcache_append_kernel(const AppendParams a) {
    constexpr int kRow = D * sizeof(T), kPer = kRow / 16;  // bytes and 16-byte pieces of a row
    constexpr int kPairs = 8 / sizeof(T);                  // element pairs of a piece
    extern __shared__ __align__(128) uint8_t ap_smem[];
    __shared__ uint64_t s_bar;
    __shared__ uint32_t s_amax;
    __shared__ volatile int s_abort;
    const int layer = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    pdl_trigger();
    if (tid == 0) {
        s_amax = 0;
        s_abort = 0;
        mbar_init(&s_bar, 1);
        fence_mbar_init();
    }
    pdl_wait();
    const int r0 = a.seg_row[blockIdx.x], r1 = a.seg_row[blockIdx.x + 1];
    if (r1 == r0) return;  // no rows (padding)
    if (r0 < 0 || r1 > a.rows || r1 < r0) {
        if (tid == 0) set_error(a.err, DSPARK_ERR_OOB);
        return;
    }
    const int nr = r1 - r0, slot = a.slots[r0], mine = a.slots[r0 + min(tid, nr - 1)];
    if (slot == -1) {  // skipped, which has to hold for every row of the span
        bool skip = true;
        for (int i = tid; i < nr; i += kAppThreads) skip = skip && a.slots[r0 + i] == -1;
        if (!__syncthreads_and(skip) && tid == 0) set_error(a.err, DSPARK_ERR_OOB);
        return;
    }
    const int page = slot / kQcPage, off = slot % kQcPage;
    if (slot < 0 || page >= a.n_pages || off + nr > kQcPage) {
        if (tid == 0) set_error(a.err, DSPARK_ERR_OOB);
        return;
    }
    const uint8_t *src = (const uint8_t *)a.entries + ((long long)layer * a.layer_stride + (long long)r0 * a.row_stride) * sizeof(T);
    uint8_t *dst = a.codes[layer] + (size_t)page * kQcPage * D;
    if (tid < 32) {
        if (lane == 0) mbar_arrive_expect_tx(&s_bar, (uint32_t)(nr * kRow));
        __syncwarp();
        if (a.row_stride == D) {
            if (lane == 0) bulk_load(ap_smem, src, (uint32_t)(nr * kRow), &s_bar);
        } else {
            for (int r = lane; r < nr; r += 32) bulk_load(ap_smem + r * kRow, src + (long long)r * a.row_stride * sizeof(T), kRow, &s_bar);
        }
    }
    const float old = off > 0 ? a.scales[layer][page] : 1.f;
    const bool run = __syncthreads_and(tid >= nr || mine == slot + tid);  // (and the barrier is set up)
    if (!mbar_wait_bounded(&s_bar, 0, &s_abort)) {
        if (tid == 0) {
            set_error(a.err, DSPARK_ERR_TIMEOUT);
            mbar_drain(&s_bar, 0);
        }
    }
    __syncthreads();
    if (s_abort) return;
    if (!run) {  // the rows' slots do not follow one another
        if (tid == 0) set_error(a.err, DSPARK_ERR_OOB);
        return;
    }
    const int n = nr * kPer;
    uint32_t mx = 0;
    bool bad = false;
    const T *tag = nullptr;  // picks the type
    for (int i = tid; i < n; i += kAppThreads) {
        const uint4 u = *(const uint4 *)(ap_smem + i * 16);
        const uint32_t m = amax_of(u, tag);
        if (m >= 0x7f800000u) {  // an infinity or NaN: the finite ones count
            bad = true;
#pragma unroll
            for (int x = 0; x < kPairs; ++x) {
                const float2 f = pair_of(u, x, tag);
                const uint32_t u0 = __float_as_uint(f.x) & 0x7fffffffu, u1 = __float_as_uint(f.y) & 0x7fffffffu;
                if (u0 < 0x7f800000u) mx = max(mx, u0);
                if (u1 < 0x7f800000u) mx = max(mx, u1);
            }
        } else {
            mx = max(mx, m);
        }
    }
    mx = __reduce_max_sync(~0u, mx);
    if (lane == 0) atomicMax(&s_amax, mx);
    bad = __syncthreads_or(bad);
    mx = s_amax;
    if (mx > __float_as_uint(448.f * qc_pow2(kQcEmax))) bad = true;
    int e = amax_exponent(mx);
    if (off > 0) {
        int eo;
        if (!qc_scale_exponent(old, &eo)) {
            bad = true;
            eo = e;
        }
        if (eo >= e) e = eo;
        else move_codes<D>(dst, off * (D / 16), eo - e);
    }
    const float inv = qc_pow2(-e);
    uint8_t *to = dst + (size_t)off * D;  // a row's pieces are its codes in order, and the rows follow one another
    for (int i = tid; i < n; i += kAppThreads) {
        const uint4 u = *(const uint4 *)(ap_smem + i * 16);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < kPairs; ++x) {
            float2 f = pair_of(u, x, tag);
            if (bad) f = make_float2(isnan(f.x) ? 0.f : f.x, isnan(f.y) ? 0.f : f.y);
            w[x / 2] |= f32x2_to_e4m3x2(f.x * inv, f.y * inv) << (16 * (x & 1));
        }
        if (kPairs == 4) *(uint2 *)(to + (size_t)i * 8) = make_uint2(w[0], w[1]);
        else *(uint32_t *)(to + (size_t)i * 4) = w[0];
    }
    if (tid == 0) {
        a.scales[layer][page] = qc_pow2(e);
        if (bad) set_error(a.err, DSPARK_ERR_BAD_INPUT);
    }
}

template <typename T, int D>
static cudaError_t launch_append_width(const AppendParams &a, int n_seg, int layers, cudaStream_t st) {
    constexpr int kSmem = kQcPage * D * (int)sizeof(T);
    static OncePerDevice once;
    const cudaError_t e =
        once([] { return cudaFuncSetAttribute(qcache_append_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return e;
    return launch_pdl(qcache_append_kernel<T, D>, dim3(n_seg, layers), dim3(kAppThreads), (size_t)kSmem, st, a);
}

template <typename T>
static cudaError_t launch_append(const AppendParams &a, int n_seg, int layers, int D, cudaStream_t st) {
    switch (D) {
        case 576: return launch_append_width<T, 576>(a, n_seg, layers, st);
        case 288: return launch_append_width<T, 288>(a, n_seg, layers, st);
        case 160: return launch_append_width<T, 160>(a, n_seg, layers, st);
        case 80: return launch_append_width<T, 80>(a, n_seg, layers, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ds

namespace {

bool ok16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool latent_supported(int kv, int rope) {
    return (kv == 512 && rope == 64) || (kv == 256 && rope == 32) || (kv == 128 && rope == 32) || (kv == 64 && rope == 16);
}

dspark_status check_cache(const dspark_qcache_t *c, bool plan) {
    if (!c) return DSPARK_ERR_NULL;
    if (!latent_supported(c->kv_lora, c->d_rope) || c->page_size != kQcPage) return DSPARK_ERR_UNSUPPORTED;
    if (c->n_layers < 0 || c->n_layers > DSPARK_MAX_LAYERS || c->n_pages < 1 || c->n_pages >= (1 << 25) ||
        c->max_pages < 1 || c->max_pages >= (1 << 25))
        return DSPARK_ERR_SHAPE;
    if (!c->page_table) return DSPARK_ERR_NULL;
    if (!ok16(c->page_table)) return DSPARK_ERR_ALIGN;
    if (plan) return DSPARK_OK;
    if (c->n_layers < 1) return DSPARK_ERR_SHAPE;
    for (int l = 0; l < c->n_layers; ++l) {
        if (!c->codes[l] || !c->scales[l]) return DSPARK_ERR_NULL;
        if (!ok16(c->codes[l]) || ((uintptr_t)c->scales[l] & 3u)) return DSPARK_ERR_ALIGN;
    }
    return DSPARK_OK;
}

int current_sms() {
    static int sms[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms[dev];
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct QaLayout {
    size_t split, ml, o, total;
};
QaLayout attend_layout(int kv) {
    QaLayout L;
    L.split = kQcCtlBytes;
    L.ml = up(L.split + sizeof(QaSplit) * kQaMaxGrid);
    L.o = up(L.ml + sizeof(float2) * 2 * kQaMaxGrid * kQaTile);
    L.total = up(L.o + sizeof(float) * 2 * kQaMaxGrid * (size_t)kQaTile * kv);
    return L;
}

dspark_status done(cudaError_t e) {
    if (e == cudaSuccess) return DSPARK_OK;
    (void)cudaGetLastError();
    return DSPARK_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t dspark_qcache_workspace_bytes(const dspark_qcache_t *c, int max_heads) {
    if (!c || !latent_supported(c->kv_lora, c->d_rope) || max_heads < 0 || max_heads > 1024) return 0;
    return max_heads ? attend_layout(c->kv_lora).total : kQcCtlBytes;
}

dspark_status dspark_qcache_plan(const dspark_qcache_t *c, const dspark_qplan_t *p, int bs, int max_new, int max_seg,
                                 void *ws, size_t ws_bytes, void *stream) {
    const dspark_status st = check_cache(c, true);
    if (st != DSPARK_OK) return st;
    if (!p || !p->length || !p->want || !p->ring || !p->ring_state || !p->length_out || !p->ring_state_out ||
        !p->cu_new || !p->seg_row)
        return DSPARK_ERR_NULL;
    if (bs < 1 || bs > kQcMaxBs || max_new < 0 || max_new > (1 << 30) || max_seg < 0 || max_seg > (1 << 30))
        return DSPARK_ERR_SHAPE;
    if (max_new > 0 && (!p->slots || !p->positions)) return DSPARK_ERR_NULL;
    const void *all[] = {p->length, p->want, p->ring, p->ring_state, p->length_out, p->ring_state_out,
                         p->cu_new, p->slots, p->positions, p->seg_row, ws};
    for (const void *x : all)
        if (!ok16(x)) return DSPARK_ERR_ALIGN;
    if (p->length_out == p->length || p->length_out == p->want || p->ring_state_out == p->ring_state) return DSPARK_ERR_SHAPE;
    if (!ws || ws_bytes < kQcCtlBytes) return DSPARK_ERR_WORKSPACE;
    PlanParams a;
    a.p = *p;
    a.page_table = c->page_table;
    a.n_pages = c->n_pages;
    a.max_pages = c->max_pages;
    a.bs = bs;
    a.max_new = max_new;
    a.max_seg = max_seg;
    a.err = (int *)ws;
    const int sms = current_sms();
    if (sms < 1) return DSPARK_ERR_CUDA;
    // about 2048 tokens of the slot map a CTA
    int grid = max_new / 2048 + 1;
    if (grid > 2 * sms) grid = 2 * sms;
    return done(launch_pdl(qcache_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, (cudaStream_t)stream, a));
}

dspark_status dspark_qcache_append(const dspark_qcache_t *c, const void *entries, int entry_type, int64_t row_stride,
                                   int64_t layer_stride, const int32_t *slots, int rows, const int32_t *seg_row,
                                   int n_seg, void *ws, size_t ws_bytes, void *stream) {
    const dspark_status st = check_cache(c, false);
    if (st != DSPARK_OK) return st;
    if (entry_type != DSPARK_ENTRY_BF16 && entry_type != DSPARK_ENTRY_FP32) return DSPARK_ERR_UNSUPPORTED;
    if (rows < 0 || n_seg < 0) return DSPARK_ERR_SHAPE;
    if (!ws || ws_bytes < kQcCtlBytes) return DSPARK_ERR_WORKSPACE;
    if (!ok16(ws)) return DSPARK_ERR_ALIGN;
    if (rows == 0 || n_seg == 0) return DSPARK_OK;
    if (!entries || !slots || !seg_row) return DSPARK_ERR_NULL;
    if (!ok16(entries) || !ok16(slots) || !ok16(seg_row)) return DSPARK_ERR_ALIGN;
    const int D = c->kv_lora + c->d_rope, quantum = entry_type == DSPARK_ENTRY_BF16 ? 8 : 4;
    if (row_stride < D || (c->n_layers > 1 && layer_stride < 0)) return DSPARK_ERR_SHAPE;
    if (row_stride % quantum || (c->n_layers > 1 && layer_stride % quantum)) return DSPARK_ERR_ALIGN;
    AppendParams a;
    memset(&a, 0, sizeof(a));
    for (int l = 0; l < c->n_layers; ++l) {
        a.codes[l] = (uint8_t *)c->codes[l];
        a.scales[l] = c->scales[l];
    }
    a.entries = entries;
    a.row_stride = row_stride;
    a.layer_stride = c->n_layers > 1 ? layer_stride : 0;
    a.slots = slots;
    a.seg_row = seg_row;
    a.rows = rows;
    a.n_pages = c->n_pages;
    a.err = (int *)ws;
    return done(entry_type == DSPARK_ENTRY_BF16 ? launch_append<__nv_bfloat16>(a, n_seg, c->n_layers, D, (cudaStream_t)stream)
                                                : launch_append<float>(a, n_seg, c->n_layers, D, (cudaStream_t)stream));
}

dspark_status dspark_qcache_attend(const dspark_qcache_t *c, int layer, const dspark_qattn_t *q, int bs, void *ws,
                                   size_t ws_bytes, void *stream) {
    const dspark_status st = check_cache(c, false);
    if (st != DSPARK_OK) return st;
    if (!q || !q->cu_q || !q->length) return DSPARK_ERR_NULL;
    const int D = c->kv_lora + c->d_rope;
    if (layer < 0 || layer >= c->n_layers || bs < 1 || bs > kQcMaxBs || q->n_heads < 1 || q->n_heads > 1024 ||
        q->total_q < 0 || (long long)q->total_q * q->n_heads >= (1ll << 31) - kQaTile * 1024ll ||
        !(q->scale > 0.f) || !isfinite(q->scale) || q->q_stride < (int64_t)q->n_heads * D ||
        q->o_stride < (int64_t)q->n_heads * c->kv_lora || (q->causal != 0 && q->causal != 1))
        return DSPARK_ERR_SHAPE;
    if (q->total_q > 0 && (!q->q || !q->o)) return DSPARK_ERR_NULL;
    if (!ok16(q->q) || !ok16(q->o) || !ok16(q->lse) || !ok16(q->cu_q) || !ok16(q->length) || !ok16(ws) ||
        q->q_stride % 8 || q->o_stride % 8)
        return DSPARK_ERR_ALIGN;
    const QaLayout L = attend_layout(c->kv_lora);
    if (!ws || ws_bytes < L.total) return DSPARK_ERR_WORKSPACE;
    if (q->total_q == 0) return DSPARK_OK;
    const int sms = current_sms();
    if (sms < 1) return DSPARK_ERR_CUDA;
    QaParams p;
    memset(&p, 0, sizeof(p));
    p.q = (const __nv_bfloat16 *)q->q;
    p.q_stride = q->q_stride;
    p.cu_q = q->cu_q;
    p.length = q->length;
    p.H = q->n_heads;
    // with 2^s >= H: ceil(2^(31 + s) / H) < 2^32, and the product errs by less than 1 / H for r < 2^31
    int hs = 0;
    while ((1 << hs) < q->n_heads) ++hs;
    p.h_shift = 31 + hs;
    p.h_mul = (uint32_t)(((1ull << (31 + hs)) + q->n_heads - 1) / (uint64_t)q->n_heads);
    p.bs = bs;
    p.total_q = q->total_q;
    p.causal = q->causal;
    p.scale_log2 = q->scale * 1.4426950408889634f;
    p.o = (__nv_bfloat16 *)q->o;
    p.o_stride = q->o_stride;
    p.lse = q->lse;
    p.codes = (const uint8_t *)c->codes[layer];
    p.scales = c->scales[layer];
    p.page_table = c->page_table;
    p.n_pages = c->n_pages;
    p.max_pages = c->max_pages;
    p.split = (QaSplit *)((char *)ws + L.split);
    p.part_ml = (float2 *)((char *)ws + L.ml);
    p.part_o = (float *)((char *)ws + L.o);
    p.err = (int *)ws;
    return done(launch_qattn(p, c->kv_lora, sms, (cudaStream_t)stream));
}

dspark_status dspark_qcache_check(void *ws, void *stream) {
    if (!ws) return DSPARK_ERR_NULL;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return DSPARK_ERR_CUDA;
    int err = 0;
    if (cudaMemcpy(&err, ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return DSPARK_ERR_CUDA;
    if (err) {
        const int zero = 0;
        if (cudaMemcpy(ws, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return DSPARK_ERR_CUDA;
    }
    return (dspark_status)err;
}

}  // extern "C"
