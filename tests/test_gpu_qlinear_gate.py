"""The gate over the whole range of gates, against the oracle in 64 bits: each block of 128 outputs has one gate, its up values
are large where the gate is far below zero."""
import numpy as np
import pytest
import torch

import mla_block_diffusion_gb300 as M
from oracle import qlinear as O
from tests.test_gpu_qlinear import dev, host

pytestmark = pytest.mark.gpu
GATES = [-1.0, -20.0, -60.0, -80.0, -88.0, -96.0, -104.0, -128.0, -160.0, 0.25, 20.0, 88.0, 320.0]


@pytest.mark.parametrize("m", [5, 70])
def test_gates_of_every_size(m):
    """Row r multiplies both factors by its scale, from 0.98 to 1.01: gates from -86.2 to -88.9, where 1 + exp(-gate) leaves
    the range of fp32, are among them."""
    k, n = 16, 128 * len(GATES)
    x = np.zeros((m, k), np.uint8)
    x[:, 0] = 0x38  # 1.0
    sx = (0.98 + 0.03 * np.arange(m, dtype=np.float32) / (m - 1))[None].astype(np.float32)
    wg, wu = np.zeros((n, k), np.uint8), np.zeros((n, k), np.uint8)
    wg[:, 0] = O.codes_of(np.repeat(np.array(GATES), 128))
    wu[:, 0] = 0x38 + np.arange(n) % 64  # 1 to 240
    wu[1::2, 0] |= 0x80
    sg = np.ones((len(GATES), 1), np.float32)
    su = np.where(np.array(GATES) < 0, 2.0 ** 118, 1.0).astype(np.float32)[:, None]
    xv = O.rows_values(x, sx)
    g, u = xv @ O.weight_values(wg, sg).T, xv @ O.weight_values(wu, su).T
    want = O.gated(g, u)
    # Of the value: the gate is off by two roundings, 2^-23 of it, which the exponential multiplies by |g|; the fast
    # exponential by 2 + 1.173 |x| units of 2^-23, twice at half the gate far below zero; division, products and u by six more.
    off = np.abs(want) * 2.0 ** -23 * (np.abs(g) + 4 + 1.173 * np.abs(g) + 6)
    hc = torch.empty(m, n, dtype=torch.uint8, device="cuda")
    hs = torch.empty(len(GATES), m, device="cuda")
    gate = M.QGated(M.QLinear(dev(wg), dev(sg)), M.QLinear(dev(wu), dev(su)))
    gate.forward(dev(x), dev(sx), hc, hs)
    assert gate.check() == 0
    scales = host(hs).astype(np.float64)
    for b in range(len(GATES)):
        at = np.s_[:, b * 128:(b + 1) * 128]
        low, high = (np.abs(want[at]) - off[at]).max(1), (np.abs(want[at]) + off[at]).max(1)
        assert (low <= 448 * scales[b]).all(), GATES[b]
        assert ((scales[b] == 2.0 ** -100) | (high > 224 * scales[b])).all(), GATES[b]
    s = np.repeat(scales.T, 128, 1)
    got = O.rows_values(host(hc), scales)
    # half a step: 2^-4 of the value, and 2^-10 scales below the normal numbers
    far = np.abs(got - want) - (off + np.maximum((np.abs(want) + off) * 2.0 ** -4, s * 2.0 ** -10))
    assert (far <= 0).all(), [GATES[b] for b in np.unique(np.nonzero(far > 0)[1] // 128)]
    assert np.abs(got).max(0).reshape(-1, 128).max(1).all()  # no block has vanished
