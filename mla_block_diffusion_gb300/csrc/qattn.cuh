// Work division of the attention over the 8-bit latent cache, shared by its
// kernels.
//
// An item is one tile of TILE query rows (token-major, heads inside) of one
// request; its units are the chunks of CH cached tokens that its last query
// sees (one unit if none: the item still writes its outputs). The units of all
// items, in order, are cut into one equal range per CTA whatever the requests'
// lengths, so ragged batches leave no CTA idle. An item that lies in one
// range is finished there; one that is cut leaves a partial per CTA (fp32
// output, reference and sum per row) for the combine kernel, which adds them in
// CTA order: the result does not depend on timing. A CTA cuts at most the items
// at its two ends: slot 2c holds its first piece, slot 2c + 1 a later one.
//
// Lengths live on the device, so every CTA finds its own range: a scan of the
// requests' tile counts, then of the units of all tiles dealt out to the
// threads in equal runs (a few instructions a tile, against the matrix work of
// at least one chunk that every tile brings).
#pragma once

#include "qcache.h"

namespace ds {

struct QaItem {
    int b, t;            // request and tile
    int q0, nq, len;     // the request's first query token, its query tokens and cached tokens
    int chunks;          // units
};

template <int TILE, int CH>
struct QaWork {
    // Request b's queries and length; out of range: no queries (reported by `report`).
    static DS_DEVINL void request(const QaParams &p, int b, int *q0, int *nq, int *len, bool report = false) {
        const int a = p.cu_q[b], z = p.cu_q[b + 1], n = p.length[b];
        const bool ok = a >= 0 && z >= a && z <= p.total_q && n >= 0 && n <= (long long)p.max_pages * kQcPage;
        if (!ok && report) set_error(p.err, DSPARK_ERR_OOB);
        *q0 = ok ? a : 0;
        *nq = ok ? z - a : 0;
        *len = ok ? n : 0;
    }
    static DS_DEVINL int tiles(const QaParams &p, int nq) { return (int)(((long long)nq * p.H + TILE - 1) / TILE); }
    // Tokens that query i of nq sees.
    static DS_DEVINL int sees(const QaParams &p, int nq, int len, int i) {
        return p.causal ? max(0, len - nq + i + 1) : len;
    }
    static DS_DEVINL int chunks(const QaParams &p, int nq, int len, int t) {
        const int last = min(nq - 1, (int)((((long long)t + 1) * TILE - 1) / p.H));
        return max(1, (int)(((long long)sees(p, nq, len, last) + CH - 1) / CH));
    }

    long long begin, end;  // this CTA's units
    long long total;
    int parts;             // CTAs with units: never more than there are units, so that no range is empty
    QaItem item;           // the item that holds `begin`
    int off;               // units of it before `begin`

    // Block-wide exclusive sum; *sum gets the total. scratch: one word per warp.
    static DS_DEVINL long long scan(long long v, long long *scratch, long long *sum) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        long long inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long o = __shfl_up_sync(~0u, inc, d);
            if (lane >= d) inc += o;
        }
        __syncthreads();
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        long long base = 0, all = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) base += scratch[w];
            all += scratch[w];
        }
        *sum = all;
        return base + inc - v;
    }

    static constexpr int kScratch = (32 + 4) * 8 + (kQcMaxBs + 2) * 4;  // bytes of shared memory that find() uses

    // All threads of the block. cta of grid.
    DS_DEVINL void find(const QaParams &p, int cta, int grid, void *smem) {
        long long *s_scan = (long long *)smem;
        int *s_item = (int *)(s_scan + 32);  // b, t, off
        int *s_tiles = (int *)(s_scan + 36);
        const int nt = blockDim.x, tid = threadIdx.x;
        // first tile of every request
        const int per = (p.bs + nt - 1) / nt;
        long long mine = 0, all_tiles;
        for (int j = 0; j < per; ++j) {
            const int b = tid * per + j;
            if (b >= p.bs) break;
            int q0, nq, len;
            request(p, b, &q0, &nq, &len, cta == 0);
            mine += tiles(p, nq);
        }
        long long at = scan(mine, s_scan, &all_tiles);
        for (int j = 0; j < per; ++j) {
            const int b = tid * per + j;
            if (b >= p.bs) break;
            int q0, nq, len;
            request(p, b, &q0, &nq, &len);
            s_tiles[b] = (int)at;
            at += tiles(p, nq);
        }
        if (tid == 0) s_tiles[p.bs] = (int)all_tiles;
        __syncthreads();
        // units of this thread's run of tiles
        const int i0 = (int)((long long)tid * all_tiles / nt), i1 = (int)((long long)(tid + 1) * all_tiles / nt);
        auto walk = [&](long long from, bool seek) -> long long {
            if (i0 >= i1) return from;
            int lo = 0, hi = p.bs;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_tiles[mid] <= i0) lo = mid;
                else hi = mid;
            }
            int b = lo, q0, nq, len;
            request(p, b, &q0, &nq, &len);
            for (int i = i0; i < i1; ++i) {
                while (i >= s_tiles[b + 1]) {
                    ++b;
                    request(p, b, &q0, &nq, &len);
                }
                const int n = chunks(p, nq, len, i - s_tiles[b]);
                if (seek && from <= begin && begin < from + n) {
                    s_item[0] = b;
                    s_item[1] = i - s_tiles[b];
                    s_item[2] = (int)(begin - from);
                }
                from += n;
            }
            return from;
        };
        const long long start = scan(walk(0, false), s_scan, &total);
        parts = (int)(total < grid ? total : grid);
        begin = cta < parts ? (long long)cta * total / parts : total;
        end = cta < parts ? (long long)(cta + 1) * total / parts : total;
        walk(start, true);
        __syncthreads();
        if (begin < end) {
            item.b = s_item[0];
            item.t = s_item[1];
            off = s_item[2];
            request(p, item.b, &item.q0, &item.nq, &item.len);
            item.chunks = chunks(p, item.nq, item.len, item.t);
        }
        __syncthreads();
    }
    // The next item (there is one while units of this CTA are left).
    DS_DEVINL void next(const QaParams &p) {
        off = 0;
        if (++item.t >= tiles(p, item.nq)) {
            item.t = 0;
            do {
                ++item.b;
                request(p, item.b, &item.q0, &item.nq, &item.len);
            } while (item.nq == 0 && item.b + 1 < p.bs);
        }
        item.chunks = chunks(p, item.nq, item.len, item.t);
    }
    // The CTA whose range holds unit u.
    DS_DEVINL int owner(long long u) const { return (int)(((u + 1) * parts - 1) / total); }
};

}  // namespace ds
