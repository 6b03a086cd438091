"""Pins of the paged-attention oracle (no GPU): brute force with exactly
rounded sums, torch's e4m3 type, closed forms and planted mistakes; and the
64-bit fraction-of-a-turn arithmetic of the rotation's angles."""
import math
from fractions import Fraction

import numpy as np
import torch

from oracle import attention as A
from oracle import paged_attention as P
from oracle import round_to_bf16


def _rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape)


def test_norm_and_rotation_against_loops():
    x, w = _rand((3, 2, 32), 1), _rand(32, 2)
    pos, freqs = [0, 7, -3], [1.0, 0.3, 0.01, 2.5e-5] * 2
    for inter in (False, True):
        got = P.norm_rope(x, w, pos, freqs, inter, 1e-3)
        for t in range(3):
            for h in range(2):
                r = math.sqrt(math.fsum(v * v for v in x[t, h]) / 32 + 1e-3)
                y = [x[t, h, i] / r * w[i] for i in range(32)]
                want = list(y)
                for i, f in enumerate(freqs):
                    a, b = (2 * i, 2 * i + 1) if inter else (i, i + 8)
                    z = complex(y[a], y[b]) * complex(math.cos(pos[t] * f), math.sin(pos[t] * f))
                    want[a], want[b] = z.real, z.imag
                assert np.allclose(got[t, h], want, rtol=0, atol=1e-13)
    # rotation keeps the length of a pair, and the score of two rotated rows
    # depends on their distance alone
    q, k = _rand((2, 1, 32), 3), _rand((2, 1, 32), 4)
    q[1], k[1] = q[0], k[0]
    fr = [10000.0 ** (-2 * i / 32) for i in range(16)]
    a, b = P.norm_rope(q, None, [5, 105], fr, False, 0.0), P.norm_rope(k, None, [2, 102], fr, False, 0.0)
    assert abs((a[0] * b[0]).sum() - (a[1] * b[1]).sum()) < 1e-10
    # planted: the other pairing, the other direction
    assert np.abs(P.norm_rope(q, None, [5, 9], fr, True, 0.0) - P.norm_rope(q, None, [5, 9], fr, False, 0.0)).max() > 0.1
    assert np.abs(P.norm_rope(q, None, [5, 9], fr, True, 0.0) - P.norm_rope(q, None, [-5, -9], fr, True, 0.0)).max() > 0.1


def test_e4m3_rows():
    # every value, every midpoint and their neighbours against torch's cast
    v = np.concatenate([P._VALUES, P._MIDS, np.nextafter(P._MIDS, 0), np.nextafter(P._MIDS, 1e9)])
    v = np.concatenate([v, -v]).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(P.e4m3_round(v), want)
    rows = np.array([[448.0, -1.0], [448.0001, 2.0], [2.0 ** -130, 0.0], [0.0, 0.0], [3.0e38, -1e30],
                     [0.875 * 2.0 ** 9 * 2.0 ** -20, 0.0], [np.inf, 7.0], [np.nan, 0.0]])
    codes, scale = P.e4m3_row(rows)
    assert scale.tolist()[:4] == [1.0, 2.0, 2.0 ** -126, 1.0]
    assert scale[5] == 2.0 ** -20 and scale[6] == 2.0 ** -6 and scale[7] == 1.0
    assert 448 * scale[4] >= 3e38 > 224 * scale[4]
    assert codes[6, 0] == 0x7F and codes[7, 0] == 0x7F and codes[0, 0] == 0x7E


def test_decode_against_the_contiguous_oracle_and_closed_forms():
    B, S, nh, nkv, d = 2, 9, 6, 2, 16
    bits = [round_to_bf16(_rand(s, i)) for i, s in enumerate([(B, nh, d), (B, S, nkv, d), (B, S, nkv, d)])]
    from oracle import bf16_to_f64
    q, K, V = (bf16_to_f64(b) for b in bits)
    out, lse, mag, reach = P.decode(q, K, V, [S, S])
    assert np.allclose(out, A.decode_attention(*bits), rtol=1e-12, atol=1e-13)
    assert (np.abs(out) <= mag + 1e-15).all() and (reach > 0).all()
    # a shorter length is the same as cutting the cache; a start drops the first keys
    o2, l2, _, _ = P.decode(q, K, V, [5, 0], starts=[2, 0])
    assert np.allclose(o2[:1], A.decode_attention(bits[0][:1], bits[1][:1, 2:5], bits[2][:1, 2:5]))
    assert (o2[1] == 0).all() and np.isneginf(l2[1]).all()
    # a window of one shows the newest key alone: its value row, its score as lse
    o3, l3, _, _ = P.decode(q, K, V, [S, 4], window=1)
    assert np.allclose(o3[0, 0], V[0, S - 1, 0]) and np.allclose(l3[1, 5], q[1, 5] @ K[1, 3, 1] / 4.0)
    # a tight cap flattens the scores, a steep slope leaves the newest key
    o4, _, _, _ = P.decode(q, K, V, [S, S], softcap=1e-9)
    assert np.allclose(o4[0, 0], V[0, :, 0].mean(axis=0), atol=1e-7)
    o5, _, _, _ = P.decode(q, K, V, [S, S], slopes=np.full(nh, 1e4))
    assert np.allclose(o5[1, 5], V[1, S - 1, 1])
    # planted: the cap after the slope, slopes of the wrong sign, starts ignored
    sl = 0.5 ** np.arange(1, nh + 1)
    base = P.decode(q, K, V, [S, S], softcap=0.5, slopes=sl)[0]
    assert np.abs(base - P.decode(q, K, V, [S, S], softcap=0.5, slopes=-sl)[0]).max() > 1e-3
    assert np.abs(o2[0] - P.decode(q, K, V, [5, 0])[0][0]).max() > 1e-3


def test_angles_as_64_bit_fractions_of_a_turn():
    """position * round(2^64 freq / 2 pi) mod 2^64 is the angle to 2^-33 turns
    at every int32 position, where f32 products are off by whole turns."""
    two_pi = Fraction(2) * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    for f in (1.0, 0.1, 10000.0 ** (-62 / 64), 5e-7):
        unit = round(Fraction(f) / two_pi * 2 ** 64)
        for pos in (1, 12345, 2 ** 20 + 7, 2 ** 31 - 1, -2 ** 31):
            got = Fraction((pos * unit) % 2 ** 64, 2 ** 64)
            want = Fraction(f) * pos / two_pi
            off = (got - want) % 1
            assert min(off, 1 - off) <= Fraction(1, 2 ** 33)
    p = np.float32(2 ** 31 - 1) * np.float32(0.1)
    assert abs(float(p) - (2 ** 31 - 1) * 0.1) > 1.0
