"""Pins of the oracles of the projections and of the prompts' attention."""
import math

import numpy as np
import pytest
import torch

from oracle import E4M3_TABLE
from oracle import paged_attention as D
from oracle import prefill_attention as A
from oracle import projection as P


@pytest.mark.parametrize("causal,window,softcap,slopes", [(True, 0, 0.0, False), (False, 0, 0.0, False), (True, 3, 0.0, True),
                                                         (False, 2, 5.0, False), (True, 0, 2.0, True)])
def test_prefill_against_loops(causal, window, softcap, slopes):
    rng = np.random.default_rng(3)
    q_starts, k_starts = [1, 4, 4, 9], [0, 5, 6, 9]  # a chunk, no queries, fewer keys than queries
    q, k, v = rng.normal(size=(10, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    sl = [0.5, 0.25, 1.0, 0.0] if slopes else None
    out, lse, size = A.prefill(q, k, v, q_starts, k_starts, 0.3, causal, softcap, sl, window)
    assert np.isnan(out[0]).all() and np.isnan(lse[9]).all()
    for b in range(3):
        n, m = q_starts[b + 1] - q_starts[b], k_starts[b + 1] - k_starts[b]
        for i in range(n):
            for h in range(4):
                p, terms = i + m - n, []
                for j in range(m):
                    if (causal and j > p) or (window and j <= p - window):
                        continue
                    s = 0.3 * math.fsum(q[q_starts[b] + i, h] * k[k_starts[b] + j, h // 2])
                    if softcap:
                        s = softcap * math.tanh(s / softcap)
                    if slopes:
                        s += sl[h] * (j - p)
                    terms.append((math.exp(s), v[k_starts[b] + j, h // 2]))
                total = math.fsum(w for w, _ in terms)
                r = q_starts[b] + i
                if not terms:
                    assert (out[r, h] == 0).all() and lse[r, h] == -math.inf
                    continue
                assert abs(lse[r, h] - math.log(total)) < 1e-13
                for e in range(8):
                    assert abs(out[r, h, e] - math.fsum(w * x[e] for w, x in terms) / total) < 1e-13
                    assert abs(size[r, h, e] - math.fsum(w * abs(x[e]) for w, x in terms) / total) < 1e-13


def test_prefill_last_token_is_a_decode_step():
    """The last query of a causal prompt sees what a decode step sees."""
    rng = np.random.default_rng(4)
    q, k, v = rng.normal(size=(7, 4, 16)), rng.normal(size=(7, 2, 16)), rng.normal(size=(7, 2, 16))
    out, lse, _ = A.prefill(q, k, v, [0, 7], [0, 7], 0.25, window=5)
    for h in range(4):
        s = k[2:, h // 2] @ q[6, h] * 0.25
        w = np.exp(s - s.max())
        assert np.allclose(out[6, h], w @ v[2:, h // 2] / w.sum(), atol=1e-14)
        assert abs(lse[6, h] - (math.log(w.sum()) + s.max())) < 1e-13


def test_prefill_hidden_values_take_no_part():
    rng = np.random.default_rng(5)
    q, k, v = (rng.normal(size=(4, 1, 8)) for _ in range(3))
    want, _, _ = A.prefill(q, k, v, [0, 4], [0, 4], 1.0)
    k[3], v[3, 0, 2] = np.nan, np.inf
    got, _, _ = A.prefill(q, k, v, [0, 4], [0, 4], 1.0)
    assert np.allclose(got[:3], want[:3], atol=1e-14) and np.isnan(got[3]).any()


def test_norm_and_scales_against_loops():
    rng = np.random.default_rng(6)
    x, w = rng.normal(size=(3, 200)), rng.normal(size=200)
    y = P.norm(x, w, 1e-3)
    for t in range(3):
        r = math.sqrt(math.fsum(x[t] ** 2) / 200 + 1e-3)
        assert np.allclose(y[t], x[t] / r * w, rtol=1e-14)
    y[1] = 0.0
    y[2, 150] = np.inf
    y[2, 151:] = 1e-45
    y[2, 128:150] = 0.0
    s = P.block_scales(y)
    assert s.shape == (3, 2) and (s[1] == 1).all() and s[2, 1] == 2.0 ** -126
    assert s[0, 1] == max(abs(a) for a in y[0, 128:]) / 448 and P.spread(s, 200).shape == (3, 200)
    assert P.spread(s, 200)[0, 127] == s[0, 0] and P.spread(s, 200)[0, 128] == s[0, 1]
    assert (P.norm(x, None, 0.0) == x).all()


def test_matmul_against_loops():
    rng = np.random.default_rng(7)
    M, N, K = 3, 130, 140
    a, w = (rng.integers(0, 127, size=s).astype(np.uint8) for s in ((M, K), (N, K)))
    sa, sw = rng.uniform(0.5, 2, size=(M, 2)), rng.uniform(0.5, 2, size=(2, 2))
    out, size = P.matmul(a, sa, w, sw)
    for m, n in ((0, 0), (2, 129), (1, 127), (0, 128)):
        terms = [E4M3_TABLE[a[m, k]] * sa[m, k // 128] * E4M3_TABLE[w[n, k]] * sw[n // 128, k // 128] for k in range(K)]
        assert abs(out[m, n] - math.fsum(terms)) <= 1e-12 * size[m, n]
    assert (size >= np.abs(out)).all()


def test_prefill_last_token_against_the_paged_decode_oracle():
    rng = np.random.default_rng(8)
    q, k, v = rng.normal(size=(9, 6, 16)), rng.normal(size=(30, 2, 16)), rng.normal(size=(30, 2, 16))
    for window, softcap, slopes in ((0, 0.0, None), (7, 0.0, None), (0, 3.0, None), (11, 2.0, [0.5, -0.25, 0.0, 1.0, 0.125, 2.0])):
        out, lse, size = A.prefill(q, k, v, [0, 9], [0, 30], 0.25, True, softcap, slopes, window)
        want, wlse, mag, _ = D.decode(q[8:], [k], [v], [30], None, 0.25, softcap, slopes, window)
        assert np.allclose(out[8:], want, atol=1e-14) and np.allclose(lse[8:], wlse, atol=1e-13) and np.allclose(size[8:], mag, atol=1e-14)


def test_codes_of_the_quotient_against_torch():
    """The codes of a row are torch's conversion of the f32 quotient, for every scale a row of bf16 can have."""
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(size=(200, 256)) * np.exp(rng.normal(size=(200, 1)) * 20)).to(torch.bfloat16)
    y = x.double().numpy()
    s = P.block_scales(y)
    assert (P.spread(s, 256)[:, ::128] == s).all()
    s32 = (np.abs(y.astype(np.float32)).reshape(200, 2, 128).max(2) / np.float32(448)).astype(np.float32)
    assert (np.abs(s32 - s) <= 2.0 ** -24 * s).all()
    q = (y.astype(np.float32) / np.repeat(s32, 128, 1)).astype(np.float32)
    codes = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (D.e4m3_round(q.astype(np.float64)) == codes).all()
    table = np.asarray(E4M3_TABLE, np.float64)
    top = np.abs(table[codes]).reshape(200, 2, 128).max(2)
    assert (top == 448).all()
