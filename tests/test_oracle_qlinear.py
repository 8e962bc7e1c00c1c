"""The oracle of the 8-bit layers checks itself (no GPU): codes and values, the scale rule, both quantisers, values of edges."""
import numpy as np
import pytest
import torch

from oracle import qlinear as O


def test_values_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_values(), t, equal_nan=True)


def test_codes_are_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.integers(-12, 7, 20000)), O.e4m3_values()[:127], [0.0, -0.0, 448.0, -448.0]])
    # halves between neighbours: to the even code
    v = O.e4m3_values()[:127]
    x = np.clip(np.concatenate([x, (v[1:] + v[:-1]) / 2]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.codes_of(x.astype(np.float64)), want)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0000001, 1), (449.0, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -100),
                                    (2.0 ** -120, -100), (2.0 ** 127, 119), (1.76 * 2.0 ** 127, 120), (float("nan"), -100)])
def test_scale_rule(amax, e):
    assert O.scale_of(np.array([0.0, -amax, amax / 3])) == 2.0 ** e


def test_quantisers_keep_blocks_apart():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 272)) * np.repeat([1.0, 1000.0, 0.001], [128, 128, 16])
    c, s = O.quantise_rows(x)
    assert c.shape == (5, 272) and s.shape == (3, 5)
    err = np.abs(O.rows_values(c, s) - x)
    # half a step: 2^-4 of the element, or 2^-10 scales below the normal numbers
    assert (err <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s.T, 128, 1)[:, :272] * 2.0 ** -10)).all()
    w = rng.standard_normal((144, 272)) * np.repeat([1.0, 64.0], [128, 16])[:, None]
    c, s = O.quantise_weight(w)
    assert s.shape == (2, 3)
    per = np.repeat(np.repeat(s, 128, 0)[:144], 128, 1)[:, :272]
    assert (np.abs(O.weight_values(c, s) - w) <= np.maximum(np.abs(w) * 2.0 ** -4, per * 2.0 ** -10)).all()
    assert (np.log2(s) == np.round(np.log2(s))).all()


def test_not_finite():
    x = np.array([[np.nan, np.inf, -np.inf, 3.0] + [1.0] * 12])
    c, s = O.quantise_rows(x)
    assert s[0, 0] == 2.0 ** -7 and list(c[0, :3] & 127) == [127] * 3 and O.rows_values(c, s)[0, 3] == 3.0


def test_gated_at_the_ends():
    g = np.array([-800.0, -1.0, 0.0, 1.0, 800.0])
    h = O.gated(g, np.full(5, 2.0))
    assert h[0] == 0 and h[2] == 0 and h[4] == 1600 and abs(h[3] - 2 / (1 + np.exp(-1.0))) < 1e-15
