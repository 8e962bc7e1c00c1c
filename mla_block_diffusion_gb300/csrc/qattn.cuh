// Work division of the attention over the 8-bit latent cache.
//
// An item is one tile of TILE = 64 query rows (token-major, heads inside) of one
// request; its units are the chunks of CH = 128 cached tokens that its last query
// sees (one unit if none: the item still writes its outputs). Two ways to divide
// them, whatever the requests' lengths:
//   - pieces: an item of n units is cut into ceil(n / per) equal pieces, one per
//     CTA, with the least `per` that the grid holds by either of two estimates;
//   - ranges: the units of all items, in order, are cut into one equal range per
//     CTA, which leaves no CTA idle but gives many of them two or more items.
// Ranges cost a CTA about QaWork::kItemCost units for its further items (queries
// in, output out, the pipeline drained and refilled, partials written and read), so
// pieces are taken unless they leave a CTA that many more units than an equal range:
// when items are fewer than CTAs and not of too different sizes. Measured with costs
// of 1, 4, 8, 14 and 24: 64 requests of 1K to 8K tokens 79, 66, 65, 65, 65 us; 100 of
// 1K to 4K -, 76, 67, 67, 66; 140 of 1K to 4K 91, 91, 91, 82, 82; 20 blocks of 5
// tokens over 500 to 9000 -, -, 101, 84, 81; 64 requests of 200 to 16K tokens, whose
// longest is three times an equal range, -, -, 103, 102, 122.
// An item that one CTA holds whole is finished there; one that is cut leaves a
// partial per CTA (fp32 output, reference and sum per row) for the combine
// kernel, which adds them in CTA order: the result does not depend on timing. A
// range cuts at most the items at its two ends: slot 2c holds CTA c's first
// piece, slot 2c + 1 a later one.
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

struct QaWork {
    static constexpr int TILE = kQaTile, CH = kQaChunk;
    static_assert((TILE & (TILE - 1)) == 0 && (CH & (CH - 1)) == 0, "powers of two");
    // Request b's queries and length; out of range: no queries (reported by `report`).
    static DS_DEVINL void request(const QaParams &p, int b, int *q0, int *nq, int *len, bool report = false) {
        const int a = p.cu_q[b], z = p.cu_q[b + 1], n = p.length[b];
        const bool ok = a >= 0 && z >= a && z <= p.total_q && n >= 0 && (unsigned)n <= (unsigned)p.max_pages * kQcPage;
        if (!ok && report) set_error(p.err, DSPARK_ERR_OOB);
        *q0 = ok ? a : 0;
        *nq = ok ? z - a : 0;
        *len = ok ? n : 0;
    }
    // Query token of row r of a request: r / H by the reciprocal (exact below 2^31).
    static DS_DEVINL unsigned token(const QaParams &p, unsigned r) {
        return (unsigned)(((unsigned long long)r * p.h_mul) >> p.h_shift);
    }
    // total_q * H < 2^31 - TILE * 1024
    static DS_DEVINL int tiles(const QaParams &p, int nq) { return (int)(((unsigned)nq * (unsigned)p.H + TILE - 1) / TILE); }
    // Tokens that query i of nq sees.
    static DS_DEVINL int sees(const QaParams &p, int nq, int len, int i) {
        return p.causal ? max(0, len - nq + i + 1) : len;
    }
    static DS_DEVINL int chunks(const QaParams &p, int nq, int len, int t) {
        unsigned seen = (unsigned)len;
        if (p.causal) seen = (unsigned)sees(p, nq, len, min(nq - 1, (int)token(p, ((unsigned)t + 1u) * TILE - 1u)));
        return max(1, (int)((seen + CH - 1) / CH));
    }

    static constexpr int kItemCost = 14;
    long long begin, end;  // this CTA's units
    long long total;
    int parts;             // CTAs with units: never more than there are units, so that no range is empty
    int piece_hi;          // pieces: the item's last CTA; ranges: -1
    QaItem item;           // the item that holds `begin`
    int off;               // units of it before `begin`

    // Block-wide exclusive sum; *sum gets the total. scratch: one word per warp.
    template <typename T>
    static DS_DEVINL T scan(T v, T *scratch, T *sum) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        T inc = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T o = __shfl_up_sync(~0u, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) scratch[warp] = inc;
        __syncthreads();
        T base = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kQaThreads / 32; ++w) {
            const T x = scratch[w];
            if (w < warp) base += x;
            all += x;
        }
        *sum = all;
        return base + inc - v;
    }

    struct Scratch {  // shared memory that find() uses
        long long units[32];
        int tiles[32];
        int at[4];                          // request, tile, units before `begin`, last CTA
        int first[kQcMaxBs + 1];            // first tile of every request
        int q0[kQcMaxBs], nq[kQcMaxBs], len[kQcMaxBs];
    };
    static constexpr int kScratch = sizeof(Scratch);

    // The request of tile i of all, and its units.
    static DS_DEVINL int request_of(const QaParams &p, const Scratch &s, int i) {
        int lo = 0, hi = p.bs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s.first[mid] <= i) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    static DS_DEVINL int units_of(const QaParams &p, const Scratch &s, int i) {
        const int b = request_of(p, s, i);
        return chunks(p, s.nq[b], s.len[b], i - s.first[b]);
    }

    // n / d for 0 <= n < 2^23, 0 < d < 2^23: the approximate quotient (2 ulp, each at most 1/2) is off by one at most.
    // Half the latency of the integer division; six of them stand between a call's start and its first load.
    static DS_DEVINL int div24(int n, int d) {
        int q = (int)__fdividef((float)n, (float)d);
        const int r = n - q * d;
        if (r < 0) --q;
        if (r >= d) ++q;
        return q;
    }
    // Pieces, if their estimate is the better one. Every warp works it out for itself, a lane an item.
    static constexpr int kPieceItems = 160, kPieceRounds = kPieceItems / 32;
    DS_DEVINL bool find_piece(const QaParams &p, const Scratch &s, int cta, int grid, int items) {
        const int lane = threadIdx.x & 31;
        int u[kPieceRounds], T = 0, longest = 0;
#pragma unroll
        for (int r = 0; r < kPieceRounds; ++r) {
            u[r] = 0;
            if (32 * r < items) {
                u[r] = 32 * r + lane < items ? units_of(p, s, 32 * r + lane) : 0;
                T += min(u[r], 1 << 14);
                longest = max(longest, u[r]);
            }
        }
        T = (int)__reduce_add_sync(~0u, (unsigned)T);
        longest = (int)__reduce_max_sync(~0u, (unsigned)longest);
        if (longest >= 1 << 14) return false;  // (the counts below stay within 32 bits)
        // tight: would do if items wasted half a piece each; loose: always does
        const int loose = div24(T + grid - items - 1, grid - items);
        const int tight = div24(2 * T + 2 * grid - items - 1, 2 * grid - items);
        int n = 0;
#pragma unroll
        for (int r = 0; r < kPieceRounds; ++r)
            if (32 * r < items) n += div24(u[r] + tight - 1, tight);
        const int cut = (int)__reduce_add_sync(~0u, (unsigned)n) <= grid ? tight : loose;
        if (min(cut, longest) > div24(T + grid - 1, grid) + kItemCost) return false;
        int base = 0;
#pragma unroll
        for (int r = 0; r < kPieceRounds; ++r) {
            if (32 * r >= items) break;
            const int w = div24(u[r] + cut - 1, cut);
            int inc = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(~0u, inc, d);
                if (lane >= d) inc += o;
            }
            const int k = cta - (base + inc - w);
            const unsigned hit = __ballot_sync(~0u, k >= 0 && k < w);
            if (hit) {
                const int src = __ffs(hit) - 1, i = 32 * r + src;
                const int units = __shfl_sync(~0u, u[r], src), of = __shfl_sync(~0u, w, src), kk = __shfl_sync(~0u, k, src);
                item.b = request_of(p, s, i);
                item.t = i - s.first[item.b];
                item.q0 = s.q0[item.b];
                item.nq = s.nq[item.b];
                item.len = s.len[item.b];
                item.chunks = units;
                off = div24(kk * units, of);
                begin = off;
                end = div24((kk + 1) * units, of);
                piece_hi = cta - kk + of - 1;
            }
            base += __shfl_sync(~0u, inc, 31);
        }
        return true;
    }

    // All threads of the block: this CTA's part of the work.
    DS_DEVINL void find(const QaParams &p, int cta, int grid, void *smem) {
        Scratch &s = *(Scratch *)smem;
        constexpr int nt = kQaThreads;
        const int tid = threadIdx.x;
        // requests: their tiles, and the first tile of each
        const int per = (p.bs + nt - 1) / nt, b0 = tid * per, b1 = min(p.bs, b0 + per);
        int mine = 0, all_tiles;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            int q0, nq, len;
            request(p, b, &q0, &nq, &len, cta == 0);
            s.q0[b] = q0;
            s.nq[b] = nq;
            s.len[b] = len;
            mine += tiles(p, nq);
        }
        int at = scan(mine, s.tiles, &all_tiles);
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            s.first[b] = at;
            at += tiles(p, s.nq[b]);
        }
        if (tid == 0) s.first[p.bs] = all_tiles;
        __syncthreads();
        piece_hi = -1;
        parts = 0;
        begin = end = 0;
        total = 0;
        if (all_tiles < min(grid, kPieceItems) && find_piece(p, s, cta, grid, all_tiles)) {
            __syncthreads();  // the scratch is free
            return;
        }
        // ranges: units of this thread's run of tiles
        const int run = (all_tiles + nt - 1) / nt, i0 = min(all_tiles, tid * run), i1 = min(all_tiles, i0 + run);
        long long start = 0;
#pragma unroll 1
        for (int seek = 0; seek < 2; ++seek) {
            long long from = start;
            if (i0 < i1) {
                int b = request_of(p, s, i0);
#pragma unroll 1
                for (int i = i0; i < i1; ++i) {
                    while (i >= s.first[b + 1]) ++b;
                    const int n = chunks(p, s.nq[b], s.len[b], i - s.first[b]);
                    if (seek && from <= begin && begin < from + n) {
                        s.at[0] = b;
                        s.at[1] = i - s.first[b];
                        s.at[2] = (int)(begin - from);
                    }
                    from += n;
                }
            }
            if (seek) break;
            start = scan(from, s.units, &total);
            parts = (int)(total < grid ? total : grid);
            if (total < (1ll << 22)) {  // grid <= 512: 32-bit divisions
                const unsigned T = (unsigned)total, P = max(1u, (unsigned)parts);
                begin = cta < parts ? (unsigned)cta * T / P : T;
                end = cta < parts ? (unsigned)(cta + 1) * T / P : T;
            } else {
                begin = cta < parts ? (long long)cta * total / parts : total;
                end = cta < parts ? (long long)(cta + 1) * total / parts : total;
            }
        }
        __syncthreads();
        if (begin < end) {
            item.b = s.at[0];
            item.t = s.at[1];
            off = s.at[2];
            item.q0 = s.q0[item.b];
            item.nq = s.nq[item.b];
            item.len = s.len[item.b];
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
    // The last CTA that holds units of the item that starts at unit u (of this CTA's counting).
    DS_DEVINL int last_cta(long long u) const {
        return piece_hi >= 0 ? piece_hi : (int)(((u + item.chunks) * parts - 1) / total);
    }
};

}  // namespace ds
