"""ORACLE (test infrastructure only): the 8-bit latent cache as its plain definition, numpy float64.

A page holds 64 tokens of E4M3 codes and one scale 2^e, -60 <= e <= 60; element = code * scale. Every head shares the
one latent, so a page has one scale.
"""
from __future__ import annotations

import math
from typing import List, Sequence, Tuple

import numpy as np

from .formats import E4M3_TABLE

PAGE = 64
EMAX = 60
# finite E4M3 magnitudes in order: codes 0..126
_GRID = E4M3_TABLE[:127]


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code (ties to the even code), saturating at 448; NaN becomes 0."""
    x = np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=1e300, neginf=-1e300)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 126)
    lo = hi - 1
    below, above = a - _GRID[lo], _GRID[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8) | np.where(np.signbit(x), 0x80, 0).astype(np.uint8)


def page_exponent(amax: float) -> int:
    """The least e with amax <= 448 * 2^e, clamped."""
    e = -EMAX
    while e < EMAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def _pages(n: int) -> int:
    return -(-n // PAGE)


def plan(length: Sequence[int], want: Sequence[int], table: np.ndarray, ring: np.ndarray, state: Tuple[int, int],
         max_new: int, max_seg: int):
    """Page plan in request order. table and ring are changed in place.

    Returns (length_out, state_out, cu_new, slots, positions, seg_row)."""
    n_pages, cap = len(ring), table.shape[1] * PAGE
    head, count = state
    out, cu, slots, pos, seg = [], [0], [], [], []
    taken, returned, room, spans, full = 0, 0, max_new, max_seg, False
    free = [int(ring[(head + i) % n_pages]) for i in range(count)]
    given: List[int] = []
    for b, (n, w) in enumerate(zip(length, want)):
        new = 0
        if not 0 <= n <= cap or not 0 <= w <= cap:
            out.append(n)
        elif w > n:
            need, touched = _pages(w) - _pages(n), _pages(w) - n // PAGE
            if full or need > len(free) - taken or w - n > room or touched > spans:
                full = True                        # and so are all growing requests after it
                out.append(n)
            else:
                for k in range(need):
                    table[b, _pages(n) + k] = free[taken + k]
                taken, room, spans, new = taken + need, room - (w - n), spans - touched, w - n
                for p in range(n, w):
                    if p == n or p % PAGE == 0:
                        seg.append(len(slots))
                    slots.append(int(table[b, p // PAGE]) * PAGE + p % PAGE)
                    pos.append(p)
                out.append(w)
        else:
            given += [int(table[b, k]) for k in range(_pages(w), _pages(n))]
            out.append(w)
        cu.append(cu[-1] + new)
    for k, pg in enumerate(given):
        ring[(head + count + k) % n_pages] = pg
    pad = lambda v, n, x: np.array(list(v) + [x] * (n - len(v)), dtype=np.int32)  # noqa: E731
    return (np.array(out, dtype=np.int32), ((head + taken) % n_pages, count - taken + len(given)),
            np.array(cu, dtype=np.int32), pad(slots, max_new, -1), pad(pos, max_new, -1),
            pad(seg, max_seg + 1, len(slots)))


def append(codes: np.ndarray, scales: np.ndarray, entries: np.ndarray, slots: np.ndarray, seg_row: np.ndarray):
    """Quantise a layer's entries [rows, D] into codes [n_pages, 64, D] and scales [n_pages], in place."""
    for a, z in zip(seg_row[:-1], seg_row[1:]):
        if z <= a or slots[a] < 0:
            continue
        page, off = divmod(int(slots[a]), PAGE)
        x = np.asarray(entries[a:z], dtype=np.float64)
        finite = np.abs(x[np.isfinite(x)])
        e = page_exponent(float(finite.max()) if finite.size else 0.0)
        if off:
            old = int(round(math.log2(float(scales[page]))))
            if old < e:
                codes[page, :off] = e4m3_encode(E4M3_TABLE[codes[page, :off]] * 2.0 ** (old - e))
            e = max(e, old)
        codes[page, off:off + z - a] = e4m3_encode(x * 2.0 ** -e)
        scales[page] = 2.0 ** e


def attend(codes: np.ndarray, scales: np.ndarray, table_row: np.ndarray, length: int, q: np.ndarray, kv: int,
           causal: bool, scale: float):
    """One request: q [n, H, D] float64 -> (o [n, H, kv], lse [n, H], sum of weight * |v| [n, H, kv],
    largest scale * sum |q||k| [n, H])."""
    n, H, _ = q.shape
    pages = [E4M3_TABLE[codes[p]] * float(scales[p]) for p in table_row[:_pages(length)]]
    k = np.concatenate(pages)[:length] if pages else np.zeros((0, q.shape[2]))
    o, lse = np.zeros((n, H, kv)), np.full((n, H), -np.inf)
    absolute, top = np.zeros((n, H, kv)), np.zeros((n, H))
    for i in range(n):
        seen = max(0, length - n + i + 1) if causal else length
        if seen == 0:
            continue
        s = scale * q[i] @ k[:seen].T
        m = s.max(axis=1, keepdims=True)
        w = np.exp(s - m)
        total = w.sum(axis=1)
        o[i] = (w @ k[:seen, :kv]) / total[:, None]
        absolute[i] = (w @ np.abs(k[:seen, :kv])) / total[:, None]
        lse[i] = m[:, 0] + np.log(total)
        top[i] = scale * (np.abs(q[i]) @ np.abs(k[:seen]).T).max(axis=1)
    return o, lse, absolute, top
