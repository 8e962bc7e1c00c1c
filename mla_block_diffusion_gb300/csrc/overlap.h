// Whether matrices in memory share a byte (host code).
#pragma once

#include <stdint.h>

namespace ds {

// `rows` rows of `width` bytes, `pitch` bytes from one to the next (pitch >= width).
struct Span {
    const void *at;
    unsigned long long width, pitch, rows;
};

// Exact where a matrix is contiguous or the pitches are equal (columns of one buffer); of two others, the bytes between the
// rows count as well.
inline bool overlap(Span a, Span b) {
    typedef __int128 wide;
    if (!a.rows || !b.rows || !a.width || !b.width) return false;
    for (Span *s : {&a, &b})
        if (s->rows == 1 || s->pitch == s->width) {  // one row
            s->width *= s->rows;
            s->rows = 1;
        }
    const wide d = (wide)(uintptr_t)b.at - (wide)(uintptr_t)a.at;
    const wide wa = a.width, wb = b.width, la = a.rows - 1, lb = b.rows - 1;
    if (d >= la * a.pitch + wa || -d >= lb * b.pitch + wb) return false;
    if (!la && !lb) return true;
    if (la && lb && a.pitch != b.pitch) return true;
    // Row i of a and row j of b share a byte where, with t = i - j and the pitch p, t p < d + wb and d < t p + wa; t goes from
    // -lb to la.
    const wide p = la ? a.pitch : b.pitch;
    auto below = [](wide x, wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };  // floor(x / y)
    const wide lo = below(d - wa, p) + 1, hi = -below(-(d + wb), p) - 1;
    return (lo > -lb ? lo : -lb) <= (hi < la ? hi : la);
}

}  // namespace ds
