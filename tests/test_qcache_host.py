"""Host checks of the 8-bit latent cache: each refusal returns its status with nothing launched (no GPU needed)."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest

import mla_block_diffusion_gb300 as M
from mla_block_diffusion_gb300 import build as B
from mla_block_diffusion_gb300 import dspark as D

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


def P(k):
    """An aligned address that is never dereferenced."""
    return 0x100000 + 0x1000 * k


def cache(**kw):
    c = D.QCacheStruct(kv_lora=512, d_rope=64, page_size=64, n_layers=2, n_pages=8, page_table=P(0), max_pages=4)
    for l in range(2):
        c.codes[l], c.scales[l] = P(1 + l), P(3 + l)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def plan_args(**kw):
    a = D.QPlanArgs(*[P(10 + i) for i in range(10)])
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attn_args(**kw):
    a = D.QAttnArgs(P(20), 64 * 576, P(21), P(22), 64, 7, 0, 0.1, P(23), 64 * 512, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_struct_layout(L):
    probe = r"""
#include <stdio.h>
#include <stddef.h>
#include "dspark.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\n", sizeof(dspark_qcache_t), offsetof(dspark_qcache_t, max_pages), sizeof(dspark_qplan_t),
         sizeof(dspark_qattn_t), offsetof(dspark_qattn_t, scale), offsetof(dspark_qattn_t, lse));
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(src, "w").write(probe)
        subprocess.run(["gcc", "-I", HEADER, src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(D.QCacheStruct), D.QCacheStruct.max_pages.offset, C.sizeof(D.QPlanArgs),
                   C.sizeof(D.QAttnArgs), D.QAttnArgs.scale.offset, D.QAttnArgs.lse.offset]


@pytest.mark.parametrize("kw,want", [
    (dict(kv_lora=512, d_rope=32), UNSUPPORTED), (dict(page_size=32), UNSUPPORTED), (dict(n_pages=0), SHAPE),
    (dict(n_pages=1 << 25), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 25), SHAPE),
    (dict(n_layers=17), SHAPE), (dict(n_layers=-1), SHAPE), (dict(page_table=None), NULL), (dict(page_table=P(0) + 8), ALIGN),
])
def test_cache_struct(L, kw, want):
    c = C.byref(cache(**kw))
    assert L.dspark_qcache_plan(c, C.byref(plan_args()), 1, 8, 8, P(50), 1024, None) == want
    assert L.dspark_qcache_append(c, P(30), 0, 576, 0, P(31), 4, P(32), 2, P(50), 1024, None) == want
    assert L.dspark_qcache_attend(c, 0, C.byref(attn_args()), 1, P(50), 1 << 40, None) == want


@pytest.mark.parametrize("name", [f for f, _ in D.QPlanArgs._fields_])
def test_plan_null_and_misaligned(L, name):
    c = C.byref(cache())
    assert L.dspark_qcache_plan(c, C.byref(plan_args(**{name: None})), 1, 8, 8, P(50), 1024, None) == NULL
    assert L.dspark_qcache_plan(c, C.byref(plan_args(**{name: P(60) + 4})), 1, 8, 8, P(50), 1024, None) == ALIGN


@pytest.mark.parametrize("bs,new,seg,ws,size,want", [
    (0, 8, 8, P(50), 1024, SHAPE), (1025, 8, 8, P(50), 1024, SHAPE), (1, -1, 8, P(50), 1024, SHAPE),
    (1, (1 << 30) + 1, 8, P(50), 1024, SHAPE), (1, 8, -1, P(50), 1024, SHAPE), (1, 8, 8, None, 1024, WORKSPACE),
    (1, 8, 8, P(50), 1023, WORKSPACE), (1, 8, 8, P(50) + 4, 1024, ALIGN),
])
def test_plan_sizes(L, bs, new, seg, ws, size, want):
    assert L.dspark_qcache_plan(C.byref(cache()), C.byref(plan_args()), bs, new, seg, ws, size, None) == want


def test_plan_aliases(L):
    c = C.byref(cache())
    assert L.dspark_qcache_plan(c, None, 1, 8, 8, P(50), 1024, None) == NULL
    assert L.dspark_qcache_plan(None, C.byref(plan_args()), 1, 8, 8, P(50), 1024, None) == NULL
    for kw in (dict(length_out=P(10)), dict(length_out=P(11)), dict(ring_state_out=P(13))):
        assert L.dspark_qcache_plan(c, C.byref(plan_args(**kw)), 1, 8, 8, P(50), 1024, None) == SHAPE


@pytest.mark.parametrize("kw,want", [
    (dict(entries=None), NULL), (dict(slots=None), NULL), (dict(seg=None), NULL), (dict(entries=P(30) + 8), ALIGN),
    (dict(slots=P(31) + 4), ALIGN), (dict(seg=P(32) + 4), ALIGN), (dict(kind=2), UNSUPPORTED), (dict(row=575), SHAPE),
    (dict(row=580), ALIGN), (dict(layer=-8), SHAPE), (dict(layer=4), ALIGN), (dict(rows=-1), SHAPE), (dict(n=-1), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(size=1000), WORKSPACE), (dict(ws=P(50) + 4), ALIGN),
    (dict(kind=1, row=578), ALIGN), (dict(kind=1, layer=2), ALIGN),
])
def test_append(L, kw, want):
    a = dict(entries=P(30), kind=0, row=576, layer=5760, slots=P(31), rows=4, seg=P(32), n=2, ws=P(50), size=1024) | kw
    assert L.dspark_qcache_append(C.byref(cache()), a["entries"], a["kind"], a["row"], a["layer"], a["slots"], a["rows"],
                                  a["seg"], a["n"], a["ws"], a["size"], None) == want


def test_append_layers(L):
    ok = (P(30), 0, 576, 5760, P(31), 4, P(32), 2, P(50), 1024, None)
    assert L.dspark_qcache_append(C.byref(cache(n_layers=0)), *ok) == SHAPE
    c = cache()
    c.codes[1] = None
    assert L.dspark_qcache_append(C.byref(c), *ok) == NULL
    c.codes[1] = P(2) + 8
    assert L.dspark_qcache_append(C.byref(c), *ok) == ALIGN
    c = cache()
    c.scales[1] = P(4) + 2
    assert L.dspark_qcache_append(C.byref(c), *ok) == ALIGN
    # nothing to do is no error
    assert L.dspark_qcache_append(C.byref(cache()), None, 0, 576, 0, None, 0, None, 0, P(50), 1024, None) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(cu_q=None), NULL), (dict(length=None), NULL), (dict(q=P(20) + 2), ALIGN),
    (dict(o=P(23) + 2), ALIGN), (dict(lse=P(24) + 4), ALIGN), (dict(cu_q=P(21) + 4), ALIGN), (dict(length=P(22) + 4), ALIGN),
    (dict(n_heads=0), SHAPE), (dict(n_heads=1025), SHAPE), (dict(total_q=-1), SHAPE), (dict(total_q=1 << 30), SHAPE),
    (dict(causal=2), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(q_stride=64 * 576 - 8), SHAPE), (dict(o_stride=64 * 512 - 8), SHAPE), (dict(q_stride=64 * 576 + 4), ALIGN),
    (dict(o_stride=64 * 512 + 4), ALIGN),
])
def test_attend(L, kw, want):
    size = L.dspark_qcache_workspace_bytes(C.byref(cache()), 64)
    assert L.dspark_qcache_attend(C.byref(cache()), 0, C.byref(attn_args(**kw)), 1, P(50), size, None) == want


def test_attend_sizes(L):
    c, a = C.byref(cache()), C.byref(attn_args())
    size = L.dspark_qcache_workspace_bytes(c, 64)
    assert size > 1024 and L.dspark_qcache_workspace_bytes(c, 0) == 1024
    assert L.dspark_qcache_workspace_bytes(c, -1) == 0 and L.dspark_qcache_workspace_bytes(c, 1025) == 0
    assert L.dspark_qcache_workspace_bytes(C.byref(cache(d_rope=16)), 1) == 0
    assert L.dspark_qcache_workspace_bytes(None, 1) == 0
    for layer, bs, ws, n, want in ((-1, 1, P(50), size, SHAPE), (2, 1, P(50), size, SHAPE), (0, 0, P(50), size, SHAPE),
                                   (0, 1025, P(50), size, SHAPE), (0, 1, None, size, WORKSPACE),
                                   (0, 1, P(50), size - 1, WORKSPACE), (0, 1, P(50) + 8, size, ALIGN)):
        assert L.dspark_qcache_attend(c, layer, a, bs, ws, n, None) == want
    assert L.dspark_qcache_attend(c, 0, None, 1, P(50), size, None) == NULL
    assert L.dspark_qcache_attend(c, 0, C.byref(attn_args(total_q=0, q=None, o=None)), 1, P(50), size, None) == 0
    assert L.dspark_qcache_check(None, None) == NULL
