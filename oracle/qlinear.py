"""8-bit layers with a scale for each block of 128, in numpy and 64 bits: quantisers, product, gated product."""
from __future__ import annotations

import numpy as np

BLOCK, EMIN = 128, -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where(c >= 128, -v, v)
    v[(c & 127) == 127] = np.nan
    return v


_VALUES = e4m3_values()


def scale_of(x: np.ndarray) -> float:
    """The least power of two 2^e, e >= EMIN, with the largest finite magnitude <= 448 * 2^e."""
    x = np.abs(x[np.isfinite(x)])
    top = float(x.max()) if x.size else 0.0
    s = 2.0 ** EMIN
    while top > 448 * s:
        s *= 2
    return s


def codes_of(x: np.ndarray) -> np.ndarray:
    """E4M3 codes of numbers of at most 448: to the nearest value, halves to the even code; not finite: the NaN code."""
    a = np.abs(x)
    ok = np.isfinite(x)
    a = np.where(ok, a, 0.0)
    _, e = np.frexp(a)
    step = 2.0 ** (np.clip(e - 1, -6, 8) - 3.0)
    r = np.rint(a / step) * step  # numpy rounds halves to even
    c = np.searchsorted(_VALUES[:127], r)
    assert np.array_equal(_VALUES[c], r)
    return np.where(ok, c + np.where(np.signbit(x), 128, 0), np.where(np.signbit(x), 255, 127)).astype(np.uint8)


def quantise_rows(x: np.ndarray):
    """(codes [rows, k], scales [ceil(k / 128), rows])."""
    m, k = x.shape
    nb = -(-k // BLOCK)
    codes, scales = np.zeros((m, k), np.uint8), np.zeros((nb, m))
    for b in range(nb):
        for r in range(m):
            part = x[r, b * BLOCK:(b + 1) * BLOCK]
            scales[b, r] = scale_of(part)
            codes[r, b * BLOCK:(b + 1) * BLOCK] = codes_of(part / scales[b, r])
    return codes, scales


def quantise_weight(w: np.ndarray):
    """(codes [n, k], scales [ceil(n / 128), ceil(k / 128)])."""
    n, k = w.shape
    codes, scales = np.zeros((n, k), np.uint8), np.zeros((-(-n // BLOCK), -(-k // BLOCK)))
    for a in range(scales.shape[0]):
        for b in range(scales.shape[1]):
            at = np.s_[a * BLOCK:(a + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            scales[a, b] = scale_of(w[at])
            codes[at] = codes_of(w[at] / scales[a, b])
    return codes, scales


def rows_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return _VALUES[codes] * np.repeat(scales.T.astype(np.float64), BLOCK, 1)[:, :codes.shape[1]]


def weight_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    n, k = codes.shape
    return _VALUES[codes] * np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]


def matmul(x: np.ndarray, w: np.ndarray):
    """(x w^T, the sum of the terms' magnitudes) of values."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def gated(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u
