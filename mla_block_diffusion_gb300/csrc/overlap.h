// Whether matrices in memory share a byte (host code).
#pragma once

#include <stdint.h>

namespace ds {

// `rows` rows of `width` bytes, `pitch` bytes from one to the next (pitch >= width).
struct Span {
    const void *at;
    unsigned long long width, pitch, rows;
};

// For overlap() below: of matrices whose ranges from the first byte to the last have bytes in common.
inline bool overlap_by_rows(Span a, Span b) {
    typedef __int128 wide;
    for (Span *s : {&a, &b})
        if (s->rows == 1 || s->pitch == s->width) {  // one row
            s->width *= s->rows;
            s->rows = 1;
        }
    const wide d = (wide)(uintptr_t)b.at - (wide)(uintptr_t)a.at;
    const wide wa = a.width, wb = b.width, la = a.rows - 1, lb = b.rows - 1;
    if (!la && !lb) return true;
    if (la && lb && a.pitch != b.pitch) return true;
    // Row i of a and row j of b share a byte where, with t = i - j and the pitch p, t p < d + wb and d < t p + wa; t goes from
    // -lb to la.
    const wide p = la ? a.pitch : b.pitch;
    auto below = [](wide x, wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };  // floor(x / y)
    const wide lo = below(d - wa, p) + 1, hi = -below(-(d + wb), p) - 1;
    return (lo > -lb ? lo : -lb) <= (hi < la ? hi : la);
}

// Exact where a matrix is contiguous or the pitches are equal (columns of one buffer); of two others, the bytes between the
// rows count as well. Sizes and ends fit 64 bits.
inline bool overlap(const Span &a, const Span &b) {
    if (!a.rows || !b.rows || !a.width || !b.width) return false;
    const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    if (x >= y + ((b.rows - 1) * b.pitch + b.width) || y >= x + ((a.rows - 1) * a.pitch + a.width)) return false;
    return overlap_by_rows(a, b);
}

}  // namespace ds
