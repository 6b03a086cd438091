"""Plain f64 CPU oracle of the projections (moe_proj_* in include/fp8moe.h), written
from the formulas.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import E4M3_TABLE

BLOCK = 128


def norm(x, weight, eps) -> np.ndarray:
    """x f64 [T, H]."""
    if weight is None:
        return np.array(x, np.float64)
    return x / np.sqrt((x ** 2).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def block_scales(y) -> np.ndarray:
    """f64 [T, ceil(H / 128)]: max|y| / 448 over the finite values of a block, at least
    2^-126, 1 where they are all zero."""
    T, H = y.shape
    a = np.where(np.isfinite(y), np.abs(y), 0.0)
    top = np.stack([a[:, c:c + BLOCK].max(1) for c in range(0, H, BLOCK)], 1)
    return np.where(top == 0, 1.0, np.maximum(top / 448.0, 2.0 ** -126))


def spread(scales, H) -> np.ndarray:
    """A scale per column."""
    return np.repeat(scales, BLOCK, axis=1)[:, :H]


def matmul(a, a_scale, w, w_scale) -> tuple[np.ndarray, np.ndarray]:
    """Codes uint8 [M, K], [N, K] and their scales: (out f64 [M, N], the same of the
    magnitudes)."""
    table = np.asarray(E4M3_TABLE, np.float64)
    M, K = a.shape
    N = w.shape[0]
    A = table[a] * spread(np.asarray(a_scale, np.float64), K)
    W = table[w] * np.repeat(spread(np.asarray(w_scale, np.float64), K), BLOCK, axis=0)[:N]
    return A @ W.T, np.abs(A) @ np.abs(W).T
