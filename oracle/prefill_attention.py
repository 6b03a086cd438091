"""Plain f64 CPU oracle of the attention of packed prompts (moe_attn_prefill in
include/fp8moe.h), written from the formulas.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.
"""
from __future__ import annotations

import numpy as np


def visible(n: int, m: int, causal: bool, window: int) -> np.ndarray:
    """bool [n, m]: key j is visible to query i, whose position is i + m - n."""
    p = np.arange(n)[:, None] + (m - n)
    j = np.arange(m)[None, :]
    seen = np.ones((n, m), bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    return seen


def scores(q, k, scale, softcap=0.0, slope=0.0) -> np.ndarray:
    """f64 [n, m] of one head, hidden ones included."""
    n, m = len(q), len(k)
    s = (q @ k.T) * scale
    if softcap:
        s = softcap * np.tanh(s / softcap)
    return s + slope * (np.arange(m)[None, :] - (np.arange(n)[:, None] + (m - n)))


def prefill(q, k, v, q_starts, k_starts, scale, causal=True, softcap=0.0, slopes=None, window=0):
    """q f64 [Tq, heads, d], k and v f64 [Tk, kv heads, d].  Returns (out f64, lse f64,
    weighted sizes sum_j p_j |v_j|); rows of no sequence are NaN."""
    Tq, nh, d = q.shape
    g = nh // k.shape[1]
    out, lse = np.full((Tq, nh, d), np.nan), np.full((Tq, nh), np.nan)
    size = np.full((Tq, nh, d), np.nan)
    for b in range(len(q_starts) - 1):
        q0, q1, k0, k1 = q_starts[b], q_starts[b + 1], k_starts[b], k_starts[b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0:
            continue
        seen = visible(n, m, causal, window)
        for h in range(nh):
            K, V = k[k0:k1, h // g], v[k0:k1, h // g]
            Q = q[q0:q1, h]
            out[q0:q1, h], lse[q0:q1, h], size[q0:q1, h] = _rows(Q, K, V, seen, scale, softcap, 0.0 if slopes is None else slopes[h])
    return out, lse, size


def _rows(Q, K, V, seen, scale, softcap, slope):
    n, m = seen.shape
    if m == 0 or not seen.any():
        return np.zeros((n, V.shape[1])), np.full(n, -np.inf), np.zeros((n, V.shape[1]))
    # hidden keys and values take no part, whatever they hold
    used = seen.any(0)
    K, V = np.where(used[:, None], K, 0.0), np.where(used[:, None], V, 0.0)
    s = np.where(seen, scores(Q, K, scale, softcap, slope), -np.inf)
    top = s.max(1, keepdims=True)
    top = np.where(np.isneginf(top), 0.0, top)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    safe = np.where(total == 0, 1.0, total)
    finite = np.isfinite(V).all()
    if finite:
        o, a = p @ V / safe, p @ np.abs(V) / safe
    else:  # a row's own visible values only
        o, a = np.zeros((n, V.shape[1])), np.zeros((n, V.shape[1]))
        for i in range(n):
            j = seen[i]
            o[i] = (p[i, j, None] / safe[i] * V[j]).sum(0)
            a[i] = (p[i, j, None] / safe[i] * np.abs(V[j])).sum(0)
    with np.errstate(divide="ignore"):
        return o, (np.log(total) + top)[:, 0], a
