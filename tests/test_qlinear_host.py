"""Host checks of the 8-bit layers: each refusal returns its status with nothing launched, and the binding's checks of its
tensors (no GPU needed)."""
import ctypes as C
import os
import subprocess
import tempfile

import pytest
import torch

import mla_block_diffusion_gb300 as M
from mla_block_diffusion_gb300 import build as B
from mla_block_diffusion_gb300 import dspark as D

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 6
BF16, FP32 = 0, 1


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


def P(k):
    """An aligned address that is never dereferenced."""
    return 0x10000000 + 0x1000000 * k


def rows(**kw):
    return D.QRowsStruct(**(dict(rows=7, k=512, codes=P(0), scales=P(1), scale_stride=7) | kw))


def weight(**kw):
    return D.QWeightStruct(**(dict(n=272, k=512, codes=P(2), scales=P(3)) | kw))


def test_struct_layout(L):
    probe = r"""
#include <stdio.h>
#include <stddef.h>
#include "dspark.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu\n", sizeof(dspark_qrows_t), offsetof(dspark_qrows_t, codes), offsetof(dspark_qrows_t, scale_stride),
         sizeof(dspark_qweight_t), offsetof(dspark_qweight_t, scales));
  printf("%d %d %d\n", DSPARK_QLINEAR_MAX_DIM, DSPARK_QLINEAR_MAX_ROWS, DSPARK_QLINEAR_WS_BYTES);
  return 0;
}
"""
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        open(src, "w").write(probe)
        subprocess.run(["gcc", "-I", HEADER, src, "-o", exe], check=True)
        got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got[:5] == [C.sizeof(D.QRowsStruct), D.QRowsStruct.codes.offset, D.QRowsStruct.scale_stride.offset,
                       C.sizeof(D.QWeightStruct), D.QWeightStruct.scales.offset]
    assert got[5:] == [1 << 20, 1 << 24, 1024]


BAD_ROWS = [(dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1, scale_stride=1 << 25), SHAPE), (dict(k=0), SHAPE), (dict(k=520), SHAPE),
            (dict(k=(1 << 20) + 16), SHAPE), (dict(scale_stride=6), SHAPE), (dict(codes=None), NULL), (dict(scales=None), NULL),
            (dict(codes=P(0) + 8), ALIGN), (dict(scales=P(1) + 2), ALIGN)]
BAD_WEIGHT = [(dict(n=0), SHAPE), (dict(n=264), SHAPE), (dict(n=-16), SHAPE), (dict(n=(1 << 20) + 16), SHAPE), (dict(k=8), SHAPE),
              (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(codes=P(2) + 4), ALIGN), (dict(scales=P(3) + 1), ALIGN)]


@pytest.mark.parametrize("kw,status", BAD_ROWS + [(dict(x=None), NULL), (dict(x=P(9) + 2), ALIGN), (dict(kind=2), UNSUPPORTED),
                                                  (dict(kind=-1), UNSUPPORTED), (dict(stride=511), SHAPE), (dict(stride=516), ALIGN),
                                                  (dict(kind=FP32, stride=514), ALIGN), (dict(x=P(0)), SHAPE),
                                                  (dict(x=P(0) + 7 * 512 - 16), SHAPE)])
def test_quantise_refusals(L, kw, status):
    a = dict(x=P(9), kind=BF16, stride=512)
    a |= {k: v for k, v in kw.items() if k in a}
    r = rows(**{k: v for k, v in kw.items() if k not in a})
    assert L.dspark_qlinear_quantise(a["x"], a["kind"], a["stride"], C.byref(r), None) == status


@pytest.mark.parametrize("kw,status", BAD_WEIGHT + [(dict(w=None), NULL), (dict(w=P(9) + 2), ALIGN), (dict(kind=2), UNSUPPORTED),
                                                    (dict(stride=511), SHAPE), (dict(stride=516), ALIGN), (dict(w=P(2) + 16), SHAPE)])
def test_quantise_weight_refusals(L, kw, status):
    a = dict(w=P(9), kind=BF16, stride=512)
    a |= {k: v for k, v in kw.items() if k in a}
    w = weight(**{k: v for k, v in kw.items() if k not in a})
    assert L.dspark_qlinear_quantise_weight(a["w"], a["kind"], a["stride"], C.byref(w), None) == status


def matmul(L, r=None, w=None, add=None, add_stride=272, y=P(5), kind=BF16, stride=272, ws=P(6), ws_bytes=1024):
    return L.dspark_qlinear_matmul(C.byref(r or rows()), C.byref(w or weight()), add, add_stride, y, kind, stride, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), NULL), (dict(y=P(5) + 8), ALIGN), (dict(kind=2), UNSUPPORTED), (dict(stride=271), SHAPE), (dict(stride=276), ALIGN),
    (dict(kind=FP32, stride=274), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws_bytes=1023), WORKSPACE), (dict(ws=P(6) + 8), ALIGN),
    (dict(add=P(7) + 4), ALIGN), (dict(add=P(7), add_stride=271), SHAPE), (dict(add=P(7), add_stride=274), ALIGN),
    (dict(y=P(0)), SHAPE), (dict(y=P(0) + 7 * 512 - 16), SHAPE),                       # y over the rows
    (dict(add=P(5)), SHAPE), (dict(add=P(5), kind=FP32, add_stride=276), SHAPE),        # add over y, but not y itself
    (dict(add=P(5) + 16, kind=FP32), SHAPE)])
def test_matmul_refusals(L, kw, status):
    assert matmul(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_matmul_refuses_rows(L, kw, status):
    assert matmul(L, r=rows(**kw)) == status


@pytest.mark.parametrize("kw,status", BAD_WEIGHT + [(dict(k=528), SHAPE)])
def test_matmul_refuses_weights(L, kw, status):
    assert matmul(L, w=weight(**kw)) == status


def gated(L, r=None, g=None, u=None, h=None, ws=P(6), ws_bytes=1024):
    h = h or rows(k=272, codes=P(10), scales=P(11))
    return L.dspark_qlinear_gated(C.byref(r or rows()), C.byref(g or weight()), C.byref(u or weight(codes=P(8))), C.byref(h), ws, ws_bytes,
                                  None)


def test_gated_refusals(L):
    assert gated(L, u=weight(n=288)) == SHAPE
    assert gated(L, u=weight(k=528)) == SHAPE
    assert gated(L, g=weight(k=528), u=weight(k=528)) == SHAPE
    assert gated(L, h=rows(k=288, codes=P(10), scales=P(11))) == SHAPE
    assert gated(L, h=rows(rows=6, k=272, codes=P(10), scales=P(11))) == SHAPE
    assert gated(L, h=rows(k=272, codes=P(0), scales=P(11))) == SHAPE       # h over the rows
    assert gated(L, h=rows(k=272, codes=P(10), scales=P(1) + 64)) == SHAPE  # its scales over theirs
    assert gated(L, ws=None) == WORKSPACE and gated(L, ws_bytes=8) == WORKSPACE and gated(L, ws=P(6) + 4) == ALIGN
    for kw, status in BAD_ROWS:
        assert gated(L, r=rows(**kw)) == status
    for kw, status in BAD_WEIGHT:
        assert gated(L, g=weight(**kw)) == status


def test_null_structs(L):
    r, w = rows(), weight()
    assert L.dspark_qlinear_quantise(P(9), 0, 512, None, None) == NULL
    assert L.dspark_qlinear_quantise_weight(P(9), 0, 512, None, None) == NULL
    assert L.dspark_qlinear_matmul(None, C.byref(w), None, 0, P(5), 0, 272, P(6), 1024, None) == NULL
    assert L.dspark_qlinear_matmul(C.byref(r), None, None, 0, P(5), 0, 272, P(6), 1024, None) == NULL
    assert L.dspark_qlinear_gated(C.byref(r), C.byref(w), None, C.byref(r), P(6), 1024, None) == NULL


def test_no_rows_are_no_work(L):
    none = dict(rows=0, codes=None, scales=None, scale_stride=0)
    assert L.dspark_qlinear_quantise(None, 0, 512, C.byref(rows(**none)), None) == 0
    assert matmul(L, r=rows(**none), y=None) == 0
    assert gated(L, r=rows(**none), h=rows(k=272, **none)) == 0


class Stand:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=torch.uint8, device=0, stride=None):
        self.shape, self.dtype, self.at, self.strides = torch.Size(shape), dtype, device, stride
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.at

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self, i=None):
        s = self.strides or tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))
        return s if i is None else s[i]

    def is_contiguous(self):
        return self.strides is None

    def data_ptr(self):
        return 0x100000


class Library:
    calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def reach(monkeypatch):
    lib, current = Library(), [0]
    monkeypatch.setattr(D, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0])
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    return lib, current


F32, BF = torch.float32, torch.bfloat16


def linear(n=272, k=512, device=0):
    return M.QLinear(Stand(n, k, device=device), Stand(-(-n // 128), -(-k // 128), dtype=F32, device=device),
                     workspace=Stand(1024, device=device))


def test_binding_passes_good_calls(reach):
    lib, current = reach
    for device in (0, 1):
        current[0] = device
        at = dict(device=device)
        m = linear(device=device)
        x, sx = Stand(7, 512, **at), Stand(4, 7, dtype=F32, **at)
        M.quantise_rows(Stand(7, 512, dtype=BF, **at), x, sx)
        M.quantise_rows(Stand(7, 512, dtype=F32, stride=(700, 1), **at), x, sx)
        M.quantise_weight(Stand(272, 512, dtype=F32, **at), Stand(272, 512, **at), Stand(3, 4, dtype=F32, **at))
        m.matmul(x, sx, Stand(7, 272, dtype=BF, **at))
        m.matmul(x, Stand(4, 7, dtype=F32, stride=(20, 1), **at), Stand(7, 272, dtype=F32, **at), add=Stand(7, 272, dtype=F32, **at))
        M.QGated(m, linear(device=device)).forward(x, sx, Stand(7, 272, **at), Stand(3, 7, dtype=F32, **at))
        assert m.check() == 0
    assert lib.calls == 14


@pytest.mark.parametrize("make", [
    lambda: M.QLinear(Stand(272, 512, dtype=F32), Stand(3, 4, dtype=F32)),
    lambda: M.QLinear(Stand(272, 512), Stand(2, 4, dtype=F32)),
    lambda: M.QLinear(Stand(272, 512), Stand(3, 4, dtype=BF)),
    lambda: M.QLinear(Stand(264, 512), Stand(3, 4, dtype=F32)),
    lambda: M.QLinear(Stand(272, 520), Stand(3, 5, dtype=F32)),
    lambda: M.QLinear(Stand(272, 512, stride=(600, 1)), Stand(3, 4, dtype=F32)),
    lambda: M.QLinear(Stand(272, 512, device=-1), Stand(3, 4, dtype=F32)),
    lambda: M.QLinear(Stand(272, 512), Stand(3, 4, dtype=F32, device=1)),
    lambda: M.QLinear(Stand(272, 512), Stand(3, 4, dtype=F32), workspace=Stand(1024, dtype=F32)),
    lambda: M.QGated(linear(), linear(n=288)),
    lambda: M.QGated(linear(), linear(device=1))])
def test_binding_refuses_weights(reach, make):
    with pytest.raises(ValueError):
        make()
    assert reach[0].calls == 0


@pytest.mark.parametrize("kw", [dict(x=Stand(7, 528)), dict(x=Stand(7, 512, dtype=F32)), dict(x=Stand(7, 512, stride=(600, 1))),
                                dict(sx=Stand(4, 6, dtype=F32)), dict(sx=Stand(7, 4, dtype=F32)), dict(sx=Stand(4, 7, dtype=BF)),
                                dict(sx=Stand(4, 7, dtype=F32, stride=(1, 4))), dict(sx=Stand(4, 7, dtype=F32, stride=(5, 1))),
                                dict(y=Stand(7, 288, dtype=BF)), dict(y=Stand(6, 272, dtype=BF)), dict(y=Stand(7, 272, dtype=torch.float16)),
                                dict(y=Stand(7, 272, dtype=BF, stride=(1, 7))), dict(add=Stand(7, 272, dtype=BF)),
                                dict(add=Stand(7, 271, dtype=F32)), dict(x=Stand(7, 512, device=1)), dict(y=Stand(7, 272, dtype=BF, device=1)),
                                dict(add=Stand(7, 272, dtype=F32, device=1))])
def test_binding_refuses_products(reach, kw):
    lib, _ = reach
    m = linear()
    a = dict(x=Stand(7, 512), sx=Stand(4, 7, dtype=F32), y=Stand(7, 272, dtype=BF), add=None) | kw
    with pytest.raises(ValueError):
        m.matmul(a["x"], a["sx"], a["y"], add=a["add"])
    assert lib.calls == 0


def test_binding_refuses_another_device(reach):
    lib, current = reach
    m = linear()
    current[0] = 1
    with pytest.raises(ValueError):
        m.matmul(Stand(7, 512), Stand(4, 7, dtype=F32), Stand(7, 272, dtype=BF))
    with pytest.raises(ValueError):
        M.QGated(m, linear()).forward(Stand(7, 512), Stand(4, 7, dtype=F32), Stand(7, 272), Stand(3, 7, dtype=F32))
    with pytest.raises(ValueError):
        m.check()
    with pytest.raises(ValueError):
        M.quantise_rows(Stand(7, 512, dtype=BF), Stand(7, 512), Stand(4, 7, dtype=F32))
    assert lib.calls == 0


WIDE = 1 << 41  # elements from one row to the next: byte counts of such a matrix do not fit 64 bits at 2^24 rows


def test_results_overlap_nothing(L):
    end = 7 * 512 - 16  # the last 16 bytes of the rows' codes
    # quantisers: scales over the source, over the codes
    assert L.dspark_qlinear_quantise(P(1), BF16, 512, C.byref(rows()), None) == SHAPE
    assert L.dspark_qlinear_quantise(P(9), BF16, 512, C.byref(rows(scales=P(0) + end)), None) == SHAPE
    assert L.dspark_qlinear_quantise_weight(P(3), BF16, 512, C.byref(weight()), None) == SHAPE
    assert L.dspark_qlinear_quantise_weight(P(9), BF16, 512, C.byref(weight(scales=P(2) + 64)), None) == SHAPE
    # products: over the rows' scales, the weights' codes and scales
    for y in (P(1), P(2), P(2) + 272 * 512 - 16, P(3)):
        assert matmul(L, y=y) == SHAPE
    # gated: h's codes or scales over any input, or over each other
    for at in (P(0), P(1), P(2), P(3), P(8), P(2) + 272 * 512 - 16):
        assert gated(L, h=rows(k=272, codes=at, scales=P(11))) == SHAPE
        assert gated(L, h=rows(k=272, codes=P(10), scales=at)) == SHAPE
    assert gated(L, h=rows(k=272, codes=P(10), scales=P(10) + 64)) == SHAPE


def test_strides_beyond_any_memory(L):
    assert matmul(L, stride=WIDE) == SHAPE
    assert matmul(L, add=P(7), add_stride=WIDE) == SHAPE
    assert matmul(L, r=rows(scale_stride=WIDE)) == SHAPE
    assert L.dspark_qlinear_quantise(P(9), BF16, WIDE, C.byref(rows()), None) == SHAPE
    assert L.dspark_qlinear_quantise_weight(P(9), FP32, WIDE, C.byref(weight()), None) == SHAPE
    assert gated(L, h=rows(k=272, codes=P(10), scales=P(11), scale_stride=WIDE)) == SHAPE
