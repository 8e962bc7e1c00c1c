"""Whether matrices in memory share a byte (csrc/overlap.h), compiled for the host, against a count of their bytes: every pair
of small matrices at every distance, and addresses and strides near the ends of 64 bits (no GPU)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <stdio.h>
#include <initializer_list>
#include "overlap.h"
using namespace ds;
typedef unsigned long long u64;
static bool in(const Span &s, u64 x) {  // byte x of memory
    const u64 at = (u64)(uintptr_t)s.at;
    return x >= at && (x - at) / s.pitch < s.rows && (x - at) % s.pitch < s.width;
}
int main(void) {
    long cases = 0, shared = 0, exact = 0;
    for (u64 ra = 1; ra <= 3; ++ra) for (u64 rb = 1; rb <= 4; ++rb)
    for (u64 wa = 1; wa <= 4; ++wa) for (u64 wb = 1; wb <= 5; ++wb)
    for (u64 pa = wa; pa <= 7; ++pa) for (u64 pb = wb; pb <= 7; ++pb)
    for (u64 at = 60; at < 140; ++at) {
        const Span a = {(void *)100, wa, pa, ra}, b = {(void *)at, wb, pb, rb};
        bool want = false;
        for (u64 x = 50; x < 200 && !want; ++x) want = in(a, x) && in(b, x);
        const bool got = overlap(a, b), solid = ra == 1 || pa == wa || rb == 1 || pb == wb || pa == pb;
        if (got != overlap(b, a) || (want && !got) || (solid && got != want)) {
            printf("%llu x %llu of %llu, %llu x %llu of %llu at %lld: %d for %d\n", ra, wa, pa, rb, wb, pb, (long long)at - 100, got, want);
            return 1;
        }
        ++cases, shared += want, exact += solid;
    }
    if (!shared || shared == cases || exact < cases / 2) return 2;
    // 2^24 rows, 2^38 bytes apart: columns of one buffer, and the far end
    const u64 far = 1ull << 38, rows = 1ull << 24;
    const Span y = {(void *)4096, 64, far, rows};
    if (overlap(y, {(void *)(4096 + 64), 64, far, rows})) return 3;
    if (!overlap(y, {(void *)(4096 + 63), 64, far, rows})) return 4;
    if (!overlap(y, {(void *)(4096 + far * (rows - 1) + 63), 1, 1, 1})) return 5;
    if (overlap(y, {(void *)(4096 + far * (rows - 1) + 64), 1, 1, 1})) return 6;
    if (overlap(y, {(void *)(4096 + far * rows), 64, far, rows})) return 7;
    if (overlap({0, 0, 1, 9}, {0, 4, 4, 4}) || overlap({0, 4, 4, 0}, {0, 4, 4, 4})) return 8;  // nothing
    printf("ok\n");
    return 0;
}
"""


def test_overlap_is_a_shared_byte(tmp_path):
    (tmp_path / "p.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "mla_block_diffusion_gb300", "csrc"), str(tmp_path / "p.cpp"), "-o",
                    str(tmp_path / "p")], check=True)
    r = subprocess.run([str(tmp_path / "p")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stdout)
