"""References of the rotating cache operators on the CPU, from the formulas alone (no product code):
in 64 bits, and in 32 bits with every product and sum rounded by itself, as the interface states
them (there every result is one number)."""
from __future__ import annotations

import numpy as np

from tests.cache_oracle import E4M3


def table(positions, dim, base=10000.0, seed=None):
    """f32 [positions, dim]: cosines, then sines."""
    f = base ** (-np.arange(0, dim, 2) / dim)
    a = np.arange(positions)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def pairs(dim, offset, interleaved):
    """The two dimensions of each pair."""
    i = np.arange(dim // 2)
    return (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + dim // 2)


def rotate(x, tab, positions, head_dim, offset, interleaved, inverse=False, dtype=np.float64):
    """x [rows, heads * head_dim] rotated, in ``dtype``; rows with positions < 0 as they are."""
    rows = x.shape[0]
    y = np.array(x, dtype=dtype).reshape(rows, -1, head_dim)
    one, two = pairs(tab.shape[1], offset, interleaved)
    for r in range(rows):
        t = positions[r]
        if t < 0:
            continue
        c, s = np.split(tab[t].astype(dtype), 2)
        s = -s if inverse else s
        a, b = y[r][:, one].copy(), y[r][:, two].copy()
        y[r][:, one] = a * c - b * s
        y[r][:, two] = b * c + a * s
    return y.reshape(rows, -1)


FINITE = np.unique(E4M3[np.isfinite(E4M3)])  # -448 .. 448, one zero


def nearest_codes(v):
    """e4m3 values (f32 in) nearest to v, ties to the even code, saturating; NaN stays."""
    v = np.asarray(v, np.float64)
    i = np.clip(np.searchsorted(FINITE, v), 1, len(FINITE) - 1)
    lo, hi = FINITE[i - 1], FINITE[i]
    mid = (lo + hi) / 2  # exact
    # codes count magnitudes up: of two neighbours the even one
    even = {x: b % 2 == 0 for b, x in enumerate(E4M3[:127])}
    lo_even = np.array([even[abs(x)] for x in lo.ravel()]).reshape(lo.shape)
    out = np.where(v < mid, lo, np.where(v > mid, hi, np.where(lo_even, lo, hi)))
    return np.where(np.isnan(v), np.nan, np.copysign(out, v))  # (what rounds to zero keeps its sign)


def record(y):
    """(code values, scale) of a latent y (f32)."""
    with np.errstate(all="ignore"):
        mag = np.abs(y[~np.isnan(y)])
        s = np.float32(mag.max() if mag.size else 0) / np.float32(448.0)
        if s == 0:
            s = np.float32(1.0)
        return nearest_codes(y / s), s
