"""Every call that the cases' ranges can make passes the host's checks, and matrices of any number of rows are quantised (no GPU
needed: without one, a call that passes them ends with the runtime's error)."""
import ctypes as C
import random

import pytest
import torch

import mla_block_diffusion_gb300 as M
from mla_block_diffusion_gb300 import build as B
from mla_block_diffusion_gb300 import dspark as D
from perf import more_operators as cases
from tests.test_qlinear_host import P, Stand

NULL, ALIGN, SHAPE, UNSUPPORTED, CUDA = 1, 2, 3, 4, 5
BF16, FP32 = 0, 1
F32, BF = torch.float32, torch.bfloat16
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not a GPU's")


@pytest.fixture(scope="module")
def L():
    B.build()
    return M.lib()


class At(Stand):
    """A stand-in at an address of its own, 16 GB from the next: never read."""
    made = 0

    def __init__(self, *shape, **kw):
        super().__init__(*shape, **kw)
        At.made += 1
        self.address = (At.made % 1000 + 1) << 34

    def data_ptr(self):
        return self.address


def blocks(n):
    return -(-n // 128)


def calls(case):
    """The calls of the framework that a pass of the case makes."""
    m, k = case["rows"], case["k"]
    rows = lambda m, k: (At(m, k), At(blocks(k), m, dtype=F32))  # noqa: E731
    weight = lambda n, k: (At(n, k), At(blocks(n), blocks(k), dtype=F32))  # noqa: E731
    linear = lambda n, k: M.QLinear(*weight(n, k), workspace=At(1024))  # noqa: E731
    if case["op"] == "quantise":
        x = At(m, k, dtype=BF if case["dtype"] == "bf16" else F32)
        return [lambda: M.quantise_weight(x, *weight(m, k))] if case["weight"] else [lambda: M.quantise_rows(x, *rows(m, k))]
    if case["op"] == "matmul":
        y = At(m, case["n"], dtype=BF if case["out"] == "bf16" else F32)
        add = At(m, case["n"], dtype=F32) if case["add"] else None
        return [lambda: linear(case["n"], k).matmul(*rows(m, k), y, add=add)]
    i = case["inter"]
    return [lambda: M.quantise_rows(At(m, k, dtype=BF), *rows(m, k)),
            lambda: M.QGated(linear(i, k), linear(i, k)).forward(*rows(m, k), *rows(m, i)),
            lambda: linear(k, i).matmul(*rows(m, i), At(m, k, dtype=BF), add=At(m, k, dtype=F32))]


@needs_no_gpu
@pytest.mark.parametrize("seed", range(4))
def test_every_case_passes_the_checks(L, monkeypatch, seed):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    rng = random.Random(seed)
    for case in cases.listed() + [cases.draw(rng) for _ in range(1000)]:
        for call in calls(case):
            with pytest.raises(M.DSparkError) as e:
                call()
            assert e.value.status == CUDA, case


def matrix(L, w=P(9), kind=BF16, stride=512, n=264, k=512, codes=P(2), scales=P(3)):
    return L.dspark_qlinear_quantise_matrix(w, kind, stride, n, k, codes, scales, None)


@needs_no_gpu
@pytest.mark.parametrize("n", [1, 2, 15, 17, 129, 264, 1234, 4999, (1 << 20) - 1, 1 << 20])
def test_matrices_of_any_number_of_rows(L, n):
    assert matrix(L, w=At(1).data_ptr(), n=n, codes=At(1).data_ptr(), scales=At(1).data_ptr()) == CUDA


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), SHAPE), (dict(n=-16), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(k=8), SHAPE), (dict(k=520, stride=520), SHAPE),
    (dict(k=0), SHAPE), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(codes=P(2) + 4), ALIGN), (dict(scales=P(3) + 1), ALIGN),
    (dict(w=None), NULL), (dict(w=P(9) + 2), ALIGN), (dict(kind=2), UNSUPPORTED), (dict(stride=511), SHAPE), (dict(stride=516), ALIGN),
    (dict(stride=1 << 41), SHAPE), (dict(w=P(2) + 263 * 512), SHAPE), (dict(w=P(3)), SHAPE), (dict(scales=P(2) + 263 * 512), SHAPE)])
def test_refusals(L, kw, status):
    assert matrix(L, **kw) == status


def test_the_binding_passes_any_number_of_rows(monkeypatch):
    got = []

    class Library:
        def dspark_qlinear_quantise_matrix(self, *a):
            got.append(a[1:5])
            return 0
    monkeypatch.setattr(D, "lib", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    for n in (1, 15, 129, 1234):
        M.quantise_weight(Stand(n, 512, dtype=BF, stride=(700, 1)), Stand(n, 512), Stand(blocks(n), 4, dtype=F32))
    assert got == [(BF16, 700 if n > 1 else 512, n, 512) for n in (1, 15, 129, 1234)]
    with pytest.raises(ValueError):  # scales of another shape
        M.quantise_weight(Stand(129, 512, dtype=BF), Stand(129, 512), Stand(1, 4, dtype=F32))
