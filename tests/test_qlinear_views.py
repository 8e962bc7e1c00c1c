"""Results and inputs of the 8-bit layers that are columns of one buffer: told apart by their bytes (no GPU needed: without one,
a call that passes the host's checks ends with the runtime's error)."""
import ctypes as C

import pytest
import torch

from tests.test_qlinear_host import BF16, FP32, P, SHAPE, L, gated, matmul, rows, weight  # noqa: F401

CUDA = 5
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not a GPU's")


@needs_no_gpu
def test_columns_of_one_buffer(L):  # noqa: F811
    # y and the residual side by side, of one type and of two (rows 4 x 600 bytes apart), either one first
    assert matmul(L, y=P(5), kind=FP32, stride=600, add=P(5) + 4 * 272, add_stride=600) == CUDA
    assert matmul(L, y=P(5) + 4 * 272, kind=FP32, stride=600, add=P(5), add_stride=600) == CUDA
    assert matmul(L, y=P(5), kind=BF16, stride=1200, add=P(5) + 2 * 272, add_stride=600) == CUDA
    # y around contiguous inputs: the rows' codes (7 x 512 bytes) between its first two rows
    assert matmul(L, y=P(0) - 4 * 272, kind=FP32, stride=4096) == CUDA
    # the scales of the rows and of h in one buffer [blocks, 20]
    x, h = rows(scale_stride=20), rows(k=272, codes=P(10), scales=P(1) + 4 * 7, scale_stride=20)
    assert gated(L, r=x, h=h) == CUDA
    # a source between the rows of its own scales
    assert L.dspark_qlinear_quantise(P(1) + 7 * 4 + 4, BF16, 512, C.byref(rows(scale_stride=4096)), None) == CUDA


def test_shared_bytes_are_refused(L):  # noqa: F811
    assert matmul(L, y=P(5), kind=FP32, stride=600, add=P(5) + 4 * 268, add_stride=600) == SHAPE     # four columns in common
    assert matmul(L, y=P(5), kind=FP32, stride=600, add=P(5) + 4 * 332, add_stride=600) == SHAPE     # the next row's first ones
    assert matmul(L, y=P(5), kind=FP32, stride=600, add=P(5) + 4 * 272, add_stride=604) == SHAPE     # not told apart
    assert matmul(L, y=P(5), kind=BF16, stride=1200, add=P(5) + 2 * 264, add_stride=600) == SHAPE
    assert matmul(L, y=P(0) - 4 * 272, kind=FP32, stride=560) == SHAPE
    x = rows(scale_stride=20)
    assert gated(L, r=x, h=rows(k=272, codes=P(10), scales=P(1) + 4 * 6, scale_stride=20)) == SHAPE
    assert gated(L, r=x, h=rows(k=272, codes=P(10), scales=P(1) + 4 * 14, scale_stride=20)) == SHAPE
    assert gated(L, r=x, h=rows(k=272, codes=P(1) + 16, scales=P(11))) == SHAPE
    assert L.dspark_qlinear_quantise(P(1) + 32, BF16, 512, C.byref(rows(scale_stride=1024)), None) == SHAPE
