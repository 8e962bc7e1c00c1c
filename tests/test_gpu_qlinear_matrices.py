"""Matrices of any number of rows into E4M3 with a scale for each block of 128 x 128, bit for bit the oracle's."""
import ctypes as C

import numpy as np
import pytest
import torch

import mla_block_diffusion_gb300 as M
from mla_block_diffusion_gb300 import dspark as D
from oracle import qlinear as O

pytestmark = pytest.mark.gpu


def same(got, want):
    """Codes equal; NaN codes of either sign are one."""
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan)
    assert np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(1, 16), (15, 144), (31, 128), (129, 272), (264, 512), (1234, 720)])
def test_any_number_of_rows(n, k, dtype):
    rng = np.random.default_rng(n * 10007 + k)
    w = torch.from_numpy(rng.standard_normal((n, k)) * np.exp2(rng.integers(-8, 8, (n, k)))).to(dtype)
    wide = torch.full((n, k + 48), 1e30, dtype=dtype, device="cuda")  # rows of another stride; their neighbours are not read
    wide[:, 16:16 + k] = w.cuda()
    codes = torch.full((n + 2, k), 9, dtype=torch.uint8, device="cuda")
    flat = torch.full((-(-n // 128) * -(-k // 128) + 2,), 9.0, device="cuda")
    scales = flat[1:-1].view(-(-n // 128), -(-k // 128))
    M.quantise_weight(wide[:, 16:16 + k], codes[1:-1], scales)
    c, s = O.quantise_weight(w.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes[1:-1].cpu().numpy(), c)
    assert bool((codes[0] == 9).all() and (codes[-1] == 9).all()) and float(flat[0]) == 9 and float(flat[-1]) == 9


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_edges(dtype):
    """Blocks of zeros, of subnormals, of the largest numbers; NaN and infinities anywhere in a block."""
    rng = np.random.default_rng(5)
    w = np.ones((300, 400))
    w[:128, :128] = 0
    w[:128, 128:256] = rng.standard_normal((128, 128)) * 2.0 ** -130
    w[:128, 256:384] = rng.uniform(-1, 1, (128, 128)) * 2.0 ** 127
    w[3, 384:] = -2.0 ** -149
    w[200, 5], w[255, 127], w[130, 200], w[129, 300] = np.nan, np.inf, -np.inf, np.nan
    w[256:, 128:256] = np.nan
    w[299, 399] = np.inf
    w = torch.from_numpy(w).to(dtype)
    codes = torch.empty(300, 400, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 4, device="cuda")
    M.quantise_weight(w.cuda(), codes, scales)
    c, s = O.quantise_weight(w.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    same(codes.cpu().numpy(), c)


def test_both_calls_give_the_same():
    """The C call for a product's weights and the one for any matrix."""
    w = torch.randn(272, 528, device="cuda")
    out = [(torch.zeros(272, 528, dtype=torch.uint8, device="cuda"), torch.zeros(3, 5, device="cuda")) for _ in range(2)]
    M.quantise_weight(w, *out[0])
    a = D.QWeightStruct(272, 528, out[1][0].data_ptr(), out[1][1].data_ptr())
    assert M.lib().dspark_qlinear_quantise_weight(w.data_ptr(), 1, 528, C.byref(a), D._stream()) == 0
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_rows_of_zeros_make_a_products_weight():
    """A matrix of 100 rows in a product: its codes with 12 rows of zeros behind them, the same scales."""
    g = torch.Generator(device="cuda").manual_seed(2)
    w, x = torch.randn(100, 272, device="cuda", generator=g), torch.randn(70, 272, device="cuda", generator=g)
    codes = torch.zeros(112, 272, dtype=torch.uint8, device="cuda")
    scales = torch.empty(1, 3, device="cuda")
    M.quantise_weight(w, codes[:100], scales)
    xq = torch.empty(70, 272, dtype=torch.uint8, device="cuda"), torch.empty(3, 70, device="cuda")
    M.quantise_rows(x, *xq)
    y = torch.empty(70, 112, device="cuda")
    lin = M.QLinear(codes, scales)
    lin.matmul(*xq, y)
    assert lin.check() == 0
    xv, wv = (f(*(t.cpu().numpy() for t in q)) for f, q in ((O.rows_values, xq), (O.weight_values, (codes, scales))))
    want, mag = O.matmul(xv, wv)
    # three blocks of four additions in the tensor core, each off by 2^-21 of what it has seen, and their fp32 sums
    assert (np.abs(y.cpu().numpy() - want) <= mag * (4 * 2.0 ** -21 + 13 * 2.0 ** -24)).all()
    assert not y[:, 100:].any()
