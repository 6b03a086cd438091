"""Plain f64 CPU oracle of the attention over a paged key/value cache
(moe_attn_* in include/fp8moe.h): head norm and rotation, e4m3 rows, and the
attention of one new token per sequence.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.  Everything is written
from the formulas; e4m3 rounding is a search over the format's values.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import E4M3_TABLE

# the 127 finite non-negative codes in ascending order of value
_CODES = np.arange(127)
_VALUES = np.asarray(E4M3_TABLE, dtype=np.float64)[:127]
_MIDS = (_VALUES[1:] + _VALUES[:-1]) / 2


def norm_rope(x, weight, positions, freqs, interleaved: bool, eps: float) -> np.ndarray:
    """x f64 [T, heads, d]; weight [d] or None; freqs f64 [R/2] (may be empty)."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    half = len(freqs)
    if half == 0:
        return y
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(freqs, np.float64)
    c, s = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def e4m3_round(y) -> np.ndarray:
    """Codes of y (f64, |y| <= 448 or NaN), nearest value, ties to the even code."""
    y = np.asarray(y, np.float64)
    a = np.abs(y)
    nan = np.isnan(a)
    hi = np.searchsorted(_MIDS, np.where(nan, 0.0, a), side="right")   # a tie goes up ..
    lo = np.searchsorted(_MIDS, np.where(nan, 0.0, a), side="left")    # .. or down
    code = np.where(hi == lo, hi, np.where(_CODES[lo] % 2 == 0, lo, hi))
    return np.where(nan, 0x7F, code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def e4m3_row(v) -> tuple[np.ndarray, np.ndarray]:
    """Codes and scales of rows v f64 [..., d]; a value that is not finite
    becomes the NaN code (0x7F, sign ignored by the caller)."""
    v = np.asarray(v, np.float64)
    fin = np.isfinite(v)
    amax = np.where(fin, np.abs(v), 0.0).max(axis=-1)
    e = np.full(amax.shape, -126)
    for k in range(-126, 128):  # smallest exponent that fits
        e = np.where((e == k) & (amax > 448.0 * 2.0 ** k), k + 1, e)
    e = np.where(amax == 0, 0, e)
    scale = 2.0 ** e.astype(np.float64)
    return e4m3_round(np.where(fin, v / scale[..., None], np.nan)), scale


def decode(q, K, V, lens, starts=None, scale=None, softcap=0.0, slopes=None, window=0):
    """q f64 [B, nh, d]; K, V: lists of f64 [len_b or more, n_kv, d] in position
    order.  Returns out, lse, and two magnitudes that rounding errors scale
    with: sum_j p_j |v_j| like out, and max_j scale * sum_i |q_i k_ji| like lse."""
    B, nh, d = q.shape
    out, mag = np.zeros((B, nh, d)), np.zeros((B, nh, d))
    lse, reach = np.full((B, nh), -np.inf), np.zeros((B, nh))
    scale = d ** -0.5 if scale is None else scale
    for b in range(B):
        n = int(lens[b])
        lo = max(0, int(starts[b]) if starts is not None else 0, n - window if window else 0)
        if lo >= n:
            continue
        g = nh // K[b].shape[1]
        for h in range(nh):
            k, v = K[b][lo:n, h // g], V[b][lo:n, h // g]
            s = scale * (k @ q[b, h])
            reach[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + slopes[h] * (np.arange(lo, n) - (n - 1.0))
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + np.log(p.sum())
            p = p / p.sum()
            out[b, h], mag[b, h] = p @ v, p @ np.abs(v)
    return out, lse, mag, reach
