"""The 8-bit latent cache's oracle against hand-worked cases and torch's own conversion (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import qcache as Q
from oracle.formats import E4M3_TABLE


def test_encode_is_nearest_even_like_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, 1, 4000) * 2.0 ** rng.integers(-12, 9, 4000), E4M3_TABLE[:127], -E4M3_TABLE[:127],
                        (E4M3_TABLE[:126] + E4M3_TABLE[1:127]) / 2])  # every halfway point
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.e4m3_encode(x), want)
    assert Q.e4m3_encode(np.array([1e9, -np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x00]


@pytest.mark.parametrize("amax,e", [(0.0, -60), (448.0, 0), (448.0001, 1), (224.0, -1), (1.75, -8), (1.7501, -7),
                                    (448 * 2.0 ** 60, 60), (1e30, 60), (1e-30, -60)])
def test_page_exponent(amax, e):
    assert Q.page_exponent(amax) == e


def test_plan_by_hand():
    # request 0 grows over a page end, 1 ends, 2 asks for too many pages, 3 grows inside its page but comes after 2
    table = np.array([[7, 0, 0], [5, 6, 0], [0, 0, 0], [4, 0, 0]], dtype=np.int32)
    ring = np.array([1, 2, 0, 0, 0, 0, 0, 3], dtype=np.int32)
    out, state, cu, slots, pos, seg = Q.plan([63, 70, 0, 10], [66, 0, 192, 11], table, ring, (7, 3), 100, 9)
    assert out.tolist() == [66, 0, 0, 10] and state == (0, 4) and cu.tolist() == [0, 3, 3, 3, 3]
    assert slots[:4].tolist() == [7 * 64 + 63, 3 * 64, 3 * 64 + 1, -1] and pos[:4].tolist() == [63, 64, 65, -1]
    assert seg[:4].tolist() == [0, 1, 3, 3] and table[0].tolist() == [7, 3, 0]
    assert ring.tolist() == [1, 2, 5, 6, 0, 0, 0, 3]


def test_append_raises_a_page_scale_and_keeps_the_rest():
    codes, scales = np.zeros((2, 64, 2), dtype=np.uint8), np.ones(2, dtype=np.float32)
    slots = np.arange(3, dtype=np.int32) + 64
    Q.append(codes, scales, np.array([[1.0, -0.5], [1.75, 0], [0, 0]]), slots, np.array([0, 3]))
    assert scales.tolist() == [1.0, 2.0 ** -8] and E4M3_TABLE[codes[1, 0]].tolist() == [256.0, -128.0]
    Q.append(codes, scales, np.array([[7.0, 0.0]]), np.array([67]), np.array([0, 1]))
    assert scales[1] == 2.0 ** -6 and (E4M3_TABLE[codes[1, :4]] * scales[1]).tolist() == [[1, -.5], [1.75, 0], [0, 0], [7, 0]]
    Q.append(codes, scales, np.array([[1.0, 1.0]]), np.array([68]), np.array([0, 1]))
    assert scales[1] == 2.0 ** -6                      # a smaller row does not lower it
    Q.append(codes, scales, np.array([[1.0, 1.0]]), np.array([64]), np.array([0, 1]))
    assert scales[1] == 2.0 ** -8                      # a page that starts over does


def test_attend_by_hand():
    codes = Q.e4m3_encode(np.zeros((1, 64, 3)))
    codes[0, :2] = Q.e4m3_encode(np.array([[2.0, 0, 1], [0, 4.0, 1]]))
    q = np.array([[[np.log(3.0), 0, 0]], [[0, 0, 1.0]]])
    o, lse, _, _ = Q.attend(codes, np.array([0.5]), np.array([0]), 2, q, 2, False, 1.0)
    assert np.allclose(o[0, 0], [0.75, 0.5]) and np.allclose(o[1, 0], [0.5, 1.0])
    assert np.allclose(lse[:, 0], [np.log(4.0), 0.5 + np.log(2.0)])
    o, lse, _, _ = Q.attend(codes, np.array([0.5]), np.array([0]), 1, q, 2, True, 1.0)
    assert np.all(o[0] == 0) and lse[0, 0] == -np.inf and np.allclose(o[1, 0], [1.0, 0.0])
