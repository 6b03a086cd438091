"""Attention of packed prompts on the GPU against the f64 oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32):
  * scores: a d-term f32 sum through 16-wide matrix steps, each charged 8 units u
    of the running sum of magnitudes, and the products with the scale: eps_s =
    (d / 2 + 16) u reach, plus 16 u cap for the tanh, 4 u per unit of distance bias;
  * out: a weight is off by eps_s, 2^-20 for exp and half a step of bf16, 2^-8, and
    the sum over n keys by (n / 2 + 64) u: all times sum_j p_j |v_j|, and half a step
    of the output, 2^-8 |exact|;
  * lse: eps_s + 2^-20 + (n / 2 + 64) u + 2 u |lse|.
"""
import numpy as np
import pytest
import torch

from fp8_routed_expert_gb300 import C, DecodeAttention, PagedKVCache, lib
from oracle import prefill_attention as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def starts_of(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def inputs(nq, nk, nh, nkv, d, seed, before=0, behind=0, size=1.0):
    """Packed rows with `before` and `behind` rows of NaN that no sequence has."""
    g = gen(seed)
    q0, k0 = starts_of(nq, before), starts_of(nk, before)
    q = torch.randn(q0[-1] + behind, nh, d, generator=g, device=DEV) * size
    kv = torch.randn(k0[-1] + behind, 2 * nkv, d, generator=g, device=DEV)
    for t, end in ((q, q0[-1]), (kv, k0[-1])):
        t[:before], t[end:] = float("nan"), float("nan")
    kv = kv.to(torch.bfloat16)
    return q.to(torch.bfloat16), kv[:, :nkv], kv[:, nkv:], q0, k0


def dev(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(DEV)


def check(q, k, v, q0, k0, causal=True, softcap=0.0, slopes=None, window=0, scale=None, attn=None):
    Tq, nh, d = q.shape
    attn = attn or DecodeAttention(nh, k.shape[1], d)
    out = torch.full((Tq, nh, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Tq, nh), 7.0, device=DEV)
    attn.prefill(q, k, v, dev(q0), dev(k0), causal=causal, softcap=softcap, slopes=slopes, window=window, scale=scale, out=out, lse=lse)
    assert attn.status() == 0
    real = d ** -0.5 if scale is None else scale
    sl = None if slopes is None else f64(slopes)
    Q, K, V = f64(q), f64(k), f64(v)
    want, wlse, size = A.prefill(Q, K, V, q0, k0, real, causal, softcap, sl, window)
    rows = ~np.isnan(wlse[:, 0])
    o, z = f64(out), f64(lse)
    assert (o[~rows] == 7).all() and (z[~rows] == 7).all()  # rows of no sequence
    # reach: the largest sum of magnitudes of a product, over a sequence's heads
    tol_s = np.zeros(wlse.shape)
    n_keys = np.zeros(Tq)
    g = nh // k.shape[1]
    for b in range(len(q0) - 1):
        a, e, c, f = q0[b], q0[b + 1], k0[b], k0[b + 1]
        if e == a or f == c:
            continue
        n_keys[a:e] = f - c
        for h in range(nh):
            reach = (np.abs(Q[a:e, h]) @ np.abs(K[c:f, h // g]).T).max() * abs(real)
            far = 0.0 if sl is None else abs(sl[h]) * max(f - c, e - a)
            tol_s[a:e, h] = (d / 2 + 16) * U * reach + 16 * U * softcap + 4 * U * far
    tol_w = tol_s + 2.0 ** -20 + ((n_keys / 2 + 64) * U)[:, None]
    empty = rows[:, None] & np.isneginf(wlse)
    assert (np.isneginf(z) == empty).all() and (o[empty] == 0).all()
    ok = rows[:, None] & ~empty
    tol_l = tol_w + 2 * U * np.abs(np.where(ok, wlse, 0))
    bad = ok & ~(np.abs(z - np.where(ok, wlse, 0)) <= tol_l)
    assert not bad.any(), (np.argwhere(bad)[:4], z[bad][:4], wlse[bad][:4])
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + tol_w)[:, :, None] * size
    bad = ok[:, :, None] & ~(np.abs(o - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), o[bad][:4], want[bad][:4], tol[bad][:4])
    return out, lse


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_one_prompt(d, n):
    check(*inputs([n], [n], 2, 2, d, n + d))


@pytest.mark.parametrize("nq,nk,nh,nkv,d", [
    ([5, 0, 300, 1, 64], [5, 0, 300, 1, 64], 4, 2, 128), ([3, 130, 17], [40, 130, 500], 8, 1, 128),
    ([70, 9, 200], [0, 5, 100], 6, 2, 64), ([1] * 20, list(range(1, 21)), 16, 2, 128), ([33, 500], [600, 513], 5, 5, 256),
    ([128, 128, 128], [128, 256, 64], 21, 7, 64), ([40, 41], [90, 41], 17, 1, 128), ([19, 200], [19, 333], 33, 1, 64),
    ([77], [200], 128, 2, 64), ([300, 2], [300, 900], 24, 2, 256), ([2000, 1, 0, 555], [2000, 1000, 3, 555], 12, 1, 128)])
def test_packed(nq, nk, nh, nkv, d):
    """Groups that do and do not divide a tile, chunks of prompts, empty sequences,
    fewer keys than queries (rows without a visible key), rows around the sequences."""
    q, k, v, q0, k0 = inputs(nq, nk, nh, nkv, d, sum(nk) + nh, before=3, behind=5)
    check(q, k, v, q0, k0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window,softcap,slopes,scale", [
    (False, 0, 0.0, False, None), (True, 1, 0.0, False, None), (True, 100, 0.0, False, None), (False, 37, 0.0, False, None),
    (True, 0, 20.0, False, None), (True, 0, 0.0, True, None), (True, 300, 5.0, True, 0.3), (False, 0, 0.0, True, None),
    (True, 0, 0.0, False, -0.1), (True, 0, 0.0, False, 0.0), (True, 2 ** 31 - 1, 0.0, False, None)])
def test_options(d, causal, window, softcap, slopes, scale):
    q, k, v, q0, k0 = inputs([150, 1, 0, 260, 40], [420, 1, 9, 260, 10], 6, 2, d, window % 1000 + d, behind=2, size=2.0)
    sl = torch.tensor([0.5, 0.25, 0.125, -0.3, 0.0, 2.0], device=DEV) if slopes else None
    check(q, k, v, q0, k0, causal, softcap, sl, window, scale)


@pytest.mark.parametrize("B", [127, 128, 129, 400])
def test_many_sequences(B):
    """Short sequences of 0..9 tokens, as many as a warp holds the lengths of, and more."""
    rng = np.random.default_rng(B)
    nq = rng.integers(0, 10, B)
    nk = nq + rng.integers(0, 30, B) * (rng.random(B) < 0.3)
    nq[B // 2] = 200
    nk[B // 2] = 333
    check(*inputs(nq.tolist(), nk.tolist(), 4, 2, 64, B, before=1, behind=1))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_steep_slopes(d, causal):
    """Distance biases that rise or fall by hundreds within a block of keys."""
    q, k, v, q0, k0 = inputs([500, 3, 130], [600, 700, 130], 6, 1, d, d + causal)
    sl = torch.tensor([5.0, -5.0, 1.2, -1.2, 0.9, -30.0], device=DEV)
    check(q, k, v, q0, k0, causal, 0.0, sl)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.1, 0.25, -0.2, 1.0])
def test_references_that_move_often(d, scale):
    """Large scores in random order: what the softmax is relative to moves in many blocks,
    while the products with the values are on their way.  The same bits each time."""
    q, k, v, q0, k0 = inputs([400, 90], [900, 90], 6, 2, d, int(scale * 100) + d, size=3.0)
    attn = DecodeAttention(6, 2, d)
    out, _ = check(q, k, v, q0, k0, scale=scale, attn=attn)
    for _ in range(10):
        assert torch.equal(attn.prefill(q, k, v, dev(q0), dev(k0), scale=scale), out)


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    rng = np.random.default_rng(seed)
    d, nkv = int(rng.choice([64, 128, 256])), int(rng.choice([1, 2, 3]))
    nh = nkv * int(rng.choice([1, 2, 3, 5, 8, 16, 17, 20]))
    B = int(rng.integers(1, 6))
    nq = rng.integers(0, 300, B)
    nk = np.maximum(0, nq + rng.integers(-50, 400, B) * (rng.random(B) < 0.5))
    window = int(rng.choice([0, 0, 1, 17, 128, 129, 500]))
    sl = torch.from_numpy(rng.normal(size=nh).astype(np.float32)).to(DEV) if rng.random() < 0.3 else None
    check(*inputs(nq.tolist(), nk.tolist(), nh, nkv, d, seed, before=int(rng.integers(0, 3)), behind=int(rng.integers(0, 3)), size=1.5),
          causal=bool(rng.random() < 0.8), softcap=float(rng.choice([0.0, 0.0, 3.0, 40.0])), slopes=sl, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_nan_that_every_row_sees(d):
    q, k, v, q0, k0 = inputs([260], [260], 4, 2, d, 8)
    v = v.clone()
    v[0, 1, 5] = float("nan")
    attn = DecodeAttention(4, 2, d)
    out = f64(attn.prefill(q, k, v, dev(q0), dev(k0)))
    v[0, 1, 5] = 0
    clean = f64(attn.prefill(q, k, v, dev(q0), dev(k0)))
    assert np.isnan(out[:, 2:, 5]).all() and np.isfinite(out[:, :2]).all()
    keep = np.delete(out[:, 2:], 5, 2)
    assert (np.abs(keep - np.delete(clean[:, 2:], 5, 2)) <= 2.0 ** -6 * np.abs(clean).max()).all()


def test_two_calls_at_once_on_one_context():
    q, k, v, q0, k0 = inputs([1500, 700], [1500, 700], 8, 2, 128, 77)
    qs, ks = dev(q0), dev(k0)
    attn = DecodeAttention(8, 2, 128)
    want = attn.prefill(q, k, v, qs, ks)
    outs = [torch.empty_like(want) for _ in range(6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, o in enumerate(outs):
        attn.prefill(q, k, v, qs, ks, out=o, stream=side if i % 2 else None)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and attn.status() == 0


def test_strided_rows_and_heads():
    """Slices of a fused projection's rows, and outputs within wider rows."""
    g = gen(11)
    T, nh, nkv, d = 333, 8, 2, 128
    fused = torch.randn(T, nh + 2 * nkv + 1, d, generator=g, device=DEV).to(torch.bfloat16)
    q, k, v = fused[:, 1:nh + 1], fused[:, nh + 1:nh + nkv + 1], fused[:, nh + nkv + 1:]
    s = dev([0, 100, 333])
    attn = DecodeAttention(nh, nkv, d)
    want = attn.prefill(q.contiguous(), k.contiguous(), v.contiguous(), s)
    wide = torch.zeros(T, nh + 2, d, dtype=torch.bfloat16, device=DEV)
    out = attn.prefill(q, k, v, s, out=wide[:, 1:-1])
    assert torch.equal(out, want) and (wide[:, 0] == 0).all() and (wide[:, -1] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sharp_and_shifting_scores(d):
    """Scores that rise by hundreds along the keys (the reference moves in every
    block), and one key that has nearly all of the weight."""
    q, k, v, q0, k0 = inputs([400], [400], 2, 1, d, 5)
    k = k.clone()
    k[..., 0] = torch.arange(400, device=DEV).view(-1, 1) * 0.5
    q[:, 0, 0], q[:, 1, 0] = 8.0, -8.0
    check(q, k, v, q0, k0, scale=0.5)
    k[..., 0] = 0
    k[200] = q[300, 0].float().mul(3).to(torch.bfloat16)
    check(q, k, v, q0, k0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("what", ["value", "key", "inf", "query"])
def test_nan_and_infinity(d, what):
    """A NaN or an infinity reaches the rows that see it and no other: earlier rows of
    the same tile, later rows beyond the window, other heads, other sequences."""
    q, k, v, q0, k0 = inputs([300, 50], [300, 50], 4, 2, d, 3)
    attn = DecodeAttention(4, 2, d)
    clean = attn.prefill(q, k, v, dev(q0), dev(k0), window=150).clone()
    q, k, v = q.clone(), k.clone(), v.clone()
    if what == "query":
        q[100, 1, 3] = float("nan")
        hit = np.zeros((350, 4), bool)
        hit[100, 1] = True
    else:
        t = k if what == "key" else v
        t[100, 0, 3] = float("inf") if what == "inf" else float("nan")
        hit = np.zeros((350, 4), bool)
        hit[100:250, :2] = True
    lse = torch.empty(350, 4, device=DEV)
    out = attn.prefill(q, k, v, dev(q0), dev(k0), window=150, lse=lse)[0]
    assert attn.status() == 0
    o, c = f64(out), f64(clean)
    assert (np.abs(o[~hit] - c[~hit]) <= 2.0 ** -6 * np.abs(c).max()).all()  # same rows, at most summed in another order
    if what in ("value", "inf"):
        lane = o[hit][:, 3]
        assert np.isnan(lane).all() if what == "value" else (lane == np.inf).all()
        rest = np.delete(o[hit], 3, 1)
        assert (np.abs(rest - np.delete(c[hit], 3, 1)) <= 2.0 ** -6 * np.abs(c).max()).all()
        assert torch.isfinite(lse).all()
    else:
        assert np.isnan(o[hit]).all() and np.isnan(f64(lse)[hit]).all() and np.isfinite(f64(lse)[~hit]).all()


def test_masked_values_of_the_lowest_and_highest():
    """Hidden keys that would win by far, hidden values at the end of bf16's range."""
    q, k, v, q0, k0 = inputs([200], [200], 2, 2, 128, 9)
    k, v = k.clone(), v.clone()
    k[150:] = 3e38
    v[150:] = -3.38e38
    out = DecodeAttention(2, 2, 128).prefill(q, k, v, dev(q0), dev(k0))
    want, _, _ = A.prefill(f64(q)[:150], f64(k)[:150], f64(v)[:150], [0, 150], [0, 150], 128 ** -0.5)
    assert np.abs(f64(out)[:150] - want).max() < 2.0 ** -6


def test_bad_starts_are_reported_and_never_followed():
    attn = DecodeAttention(2, 2, 64)
    q, k, v, q0, k0 = inputs([30, 30], [30, 30], 2, 2, 64, 1)
    good = attn.prefill(q, k, v, dev([0, 30, 60]), dev([0, 30, 60]))
    assert attn.status() == 0
    for qs, ks in (([0, 30, 61], [0, 30, 60]), ([-5, 30, 60], [0, 30, 60]), ([0, 40, 30], [0, 30, 60]),
                   ([0, 30, 60], [0, 2 ** 31 - 1, 60]), ([0, 30, 60], [0, 30, -2 ** 31]), ([2 ** 31 - 1, 0, 1], [0, 0, 0])):
        attn.prefill(q, k, v, dev(qs), dev(ks))
        assert attn.status() == C["MOE_ERR_DEVICE"]
    assert torch.equal(attn.prefill(q, k, v, dev([0, 30, 60])), good) and attn.status() == 0


def test_no_keys_no_queries_no_sequences():
    attn = DecodeAttention(4, 2, 128)
    e = lambda t, h: torch.empty(t, h, 128, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    out, lse = attn.prefill(e(5, 4), e(0, 2), e(0, 2), dev([0, 2, 5]), dev([0, 0, 0]), lse=torch.empty(5, 4, device=DEV))
    assert (out == 0).all() and torch.isneginf(lse).all()
    assert attn.prefill(e(0, 4), e(3, 2), e(3, 2), dev([0, 0]), dev([0, 3])).shape == (0, 4, 128)
    o = torch.full((5, 4, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    attn.prefill(e(5, 4), e(3, 2), e(3, 2), dev([0]), dev([0]), out=o)
    assert (o == 3).all() and attn.status() == 0


def test_same_bits_twice_in_a_graph_and_on_streams():
    q, k, v, q0, k0 = inputs([900, 77, 300], [1200, 77, 300], 8, 2, 128, 21)
    qs, ks = dev(q0), dev(k0)
    attn = DecodeAttention(8, 2, 128)
    want = attn.prefill(q, k, v, qs, ks).clone()
    assert torch.equal(attn.prefill(q, k, v, qs, ks), want)
    out = torch.empty_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    attn.prefill(q, k, v, qs, ks, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.prefill(q, k, v, qs, ks, out=out)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
    # other lengths in the same graph: they are read on the device
    qs.copy_(dev([0, 10, 500, 1277]))
    ks.copy_(dev([0, 10, 600, 1577]))
    g.replay()
    assert torch.equal(out, attn.prefill(q, k, v, qs, ks)) and attn.status() == 0


def test_few_sms_give_the_same_bits():
    q, k, v, q0, k0 = inputs([500, 300], [500, 800], 4, 4, 128, 22)
    want = DecodeAttention(4, 4, 128).prefill(q, k, v, dev(q0), dev(k0))
    assert torch.equal(DecodeAttention(4, 4, 128, max_sms=3).prefill(q, k, v, dev(q0), dev(k0)), want)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap", [4096.0, 4097.0, 1e6, 1e30])
def test_caps_far_above_the_scores(d, cap):
    """|s| < 40 makes s - cap tanh(s / cap) at most 40^3 / (3 cap^2) < 2e-3: the same outputs as without a
    cap, weights off by that and by the cap's own error, 2^-21 cap where the cap is at most 4096."""
    q, k, v, q0, k0 = inputs([150, 9], [200, 700], 4, 2, d, 77)
    attn = DecodeAttention(4, 2, d)
    want, wlse = attn.prefill(q, k, v, dev(q0), dev(k0), lse=torch.empty(159, 4, device=DEV))
    out, lse = attn.prefill(q, k, v, dev(q0), dev(k0), softcap=cap, lse=torch.empty(159, 4, device=DEV))
    off = 40 ** 3 / (3 * cap * cap) + (2.0 ** -21 * cap if cap <= 4096 else 0) + 2.0 ** -18
    size = torch.from_numpy(A.prefill(f64(q), f64(k), f64(v), q0, k0, d ** -0.5)[2]).to(DEV)  # sum p |v|
    assert ((lse - wlse).abs() <= off + 2 * U * wlse.abs()).all()
    assert ((out.double() - want.double()).abs() <= 2 * 2.0 ** -8 * want.double().abs() + (2 * 2.0 ** -8 + 2 * off) * size).all()


# Few queries and many keys: a cluster's CTAs share an item's keys.
SPLIT = [
    ([1], [3000], 8, 8, 128), ([1], [20001], 16, 1, 128), ([37], [2500], 8, 2, 128), ([64], [2064], 16, 4, 64),
    ([20, 90], [3000, 1000], 8, 2, 256), ([1, 0, 64, 3], [3000, 0, 64, 2000], 8, 2, 128), ([5, 18, 19], [900, 5000, 901], 21, 3, 64),
    ([9], [4000], 33, 1, 128), ([2] * 9, [1000 + 333 * i for i in range(9)], 2, 2, 256), ([300], [5000], 4, 1, 64), ([65], [129 * 64], 4, 4, 128),
]


@pytest.mark.parametrize("nq,nk,nh,nkv,d", SPLIT)
def test_few_queries_and_many_keys(nq, nk, nh, nkv, d):
    check(*inputs(nq, nk, nh, nkv, d, sum(nk) + nh, before=3, behind=5))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window,softcap,slopes", [
    (False, 0, 0.0, None), (True, 1, 0.0, None), (True, 1500, 0.0, None), (False, 700, 3.0, None), (True, 0, 20.0, None),
    (True, 0, 0.0, [0.5, 0.25, 0.001, -0.3, 0.0, 2.0]), (False, 0, 2.0, [0.01, -0.01, 0.001, -0.001, 0.0, 1e-4])])
def test_few_queries_and_many_keys_with_options(d, causal, window, softcap, slopes):
    q, k, v, q0, k0 = inputs([20, 1, 0, 40], [4000, 3333, 9, 2000], 6, 2, d, window + d, behind=2, size=2.0)
    check(q, k, v, q0, k0, causal, softcap, None if slopes is None else torch.tensor(slopes, device=DEV), window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 1500, 2990])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_hidden_values_of_shared_keys(d, at, what):
    """The last query sees a value that is not finite, the others' outputs are as without it."""
    q, k, v, q0, k0 = inputs([10], [2991], 4, 2, d, at + d)
    attn = DecodeAttention(4, 2, d)
    clean, lse = attn.prefill(q, k, v, dev(q0), dev(k0), window=2982 if at == 0 else 0, lse=torch.empty(10, 4, device=DEV))
    v = v.clone()
    v[at] = what
    out, lse2 = attn.prefill(q, k, v, dev(q0), dev(k0), window=2982 if at == 0 else 0, lse=torch.empty(10, 4, device=DEV))
    seen = torch.tensor([(at == 0 and i == 0) or (at == 1500) or (at == 2990 and i == 9) for i in range(10)], device=DEV)
    assert torch.isfinite(out[~seen]).all() and not torch.isfinite(out[seen]).any() and torch.isfinite(lse2).all()
    # a row that met a value that is not finite is computed again, with f32 weights: both outputs are
    # within 2^-8 (|out| + sum p |v|) of the exact one, and sum p |v| is about 0.8
    assert (out[~seen].float() - clean[~seen].float()).abs().max() < 0.02 if (~seen).any() else True
    assert (lse2 - lse).abs().max() < 1e-4 and attn.status() == 0


def test_shared_keys_on_streams_and_in_graphs():
    q, k, v, q0, k0 = inputs([64, 1], [2064, 4000], 16, 4, 128, 5)
    qs, ks = dev(q0), dev(k0)
    attn = DecodeAttention(16, 4, 128)
    want = attn.prefill(q, k, v, qs, ks).clone()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in range(24)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        attn.prefill(q, k, v, qs, ks, out=o, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(g):
        for _ in range(3):
            attn.prefill(q, k, v, qs, ks, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    qs.copy_(dev([0, 3, 65]))  # read on the device
    ks.copy_(dev([0, 0, 6064]))
    g.replay()
    assert torch.equal(out, attn.prefill(q, k, v, qs, ks)) and (out[:3] == 0).all() and attn.status() == 0


def test_chunks_of_a_prompt_through_the_cache():
    """A prompt in chunks, each with the keys and values read back from the pages, is
    the prompt at once; its last token is the decode step's."""
    nh, nkv, d, n = 8, 2, 128, 333
    q, k, v, _, _ = inputs([n], [n], nh, nkv, d, 31)
    attn = DecodeAttention(nh, nkv, d)
    cache = PagedKVCache.empty(16, 32, nkv, d)
    order = torch.randperm(16, generator=gen(1), device=DEV)
    j = torch.arange(n, device=DEV)
    slots = order[j // 32] * 32 + j % 32
    attn.write(cache, k, v, slots)
    whole = attn.prefill(q, k, v, dev([0, n]))
    for a, e in ((0, 100), (100, 101), (101, 333)):
        kc, vc = attn.read(cache, slots[:e].contiguous())
        part = attn.prefill(q[a:e], kc, vc, dev([0, e - a]), dev([0, e]))
        assert (part.float() - whole[a:e].float()).abs().max() <= 2.0 ** -6 * whole.float().abs().max()
    one = attn.decode(q[n - 1:], cache, order.to(torch.int32).view(1, -1), dev([n]))
    assert (one.float() - whole[n - 1:].float()).abs().max() <= 2.0 ** -6 * whole.float().abs().max()
    assert attn.status() == 0


def test_refusals():
    attn = DecodeAttention(4, 2, 128)
    q, k, v, q0, k0 = inputs([9], [9], 4, 2, 128, 1)
    qs, ks = dev(q0), dev(k0)
    for bad in (dict(q=q[:, :3]), dict(k=q), dict(v=v[:5]), dict(q=q.float()), dict(q=q.cpu()), dict(q_starts=qs.long()),
                dict(k_starts=ks[:1]), dict(q_starts=qs[:0]), dict(window=-1), dict(window=2 ** 31), dict(out=q[:4]),
                dict(lse=torch.empty(9, 3, device=DEV)), dict(slopes=torch.zeros(3, device=DEV)), dict(q=q.transpose(0, 1))):
        with pytest.raises(ValueError):
            attn.prefill(**{**dict(q=q, k=k, v=v, q_starts=qs, k_starts=ks), **bad})
    for bad in (dict(softcap=-1.0), dict(scale=float("nan"))):
        with pytest.raises(RuntimeError):
            attn.prefill(q, k, v, qs, ks, **bad)
    attn.close()
    with pytest.raises(ValueError):
        attn.prefill(q, k, v, qs, ks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,softcap,slope", [(True, 0.0, 0.0), (False, 0.0, 0.0), (True, 0.0, 2.0 ** -20), (True, 64.0, 0.0), (True, 300.0, 0.0)])
@pytest.mark.parametrize("at", [[300], [0, 300], [5, 140, 141, 700]])
def test_a_key_that_has_all_of_the_weight(d, causal, softcap, slope, at):
    """One key's score is 25 to 45 above all others', whose weights together stay below 1000 e^-25 < 2^-26: the
    output is its value to the bit, however the weights were rounded.  Several such keys share one value."""
    q, k, v, q0, k0 = inputs([300, 40], [900, 800], 4, 2, d, d + len(at))
    g = gen(5)
    k, v = torch.zeros_like(k), (torch.rand(v.shape, generator=g, device=DEV) + 1).to(torch.bfloat16)
    q = torch.zeros_like(q)
    q[..., 0] = 25 + 20 * torch.rand(q.shape[:2], generator=g, device=DEV)
    q[..., 1] = torch.rand(q.shape[:2], generator=g, device=DEV)
    for start in (0, 900):
        for j in at:
            k[start + j, :, :2] = 1.0
            v[start + j] = v[start + at[0]]
    attn = DecodeAttention(4, 2, d)
    sl = torch.full((4,), slope, device=DEV) if slope else None
    out = attn.prefill(q, k, v, dev(q0), dev(k0), causal=causal, scale=1.0, softcap=softcap, slopes=sl)
    for start, a, e, n in ((0, 0, 300, 900), (900, 300, 340, 800)):
        first = a if not causal else max(a, a + at[0] - (n - (e - a)))
        want = v[start + at[0]].repeat_interleave(2, 0)
        assert (out[first:e] == want).all(), int((out[first:e] != want).sum())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nk", [700, 5])
@pytest.mark.parametrize("cap", [2.0, 30.0, 50.0, 100.0, 127.9, 129.0, 400.0, 1000.0, 4096.0, 5000.0, 1e5])
def test_caps_at_the_stated_bound(d, nk, cap):
    """A score is off by 2^-19 of a cap up to 128 and by 2^-20 of itself above, with the sums' and the exponentials'
    own errors; lse is off by as much, an output by the weights' 2^-8 and twice the scores'."""
    q, k, v, q0, k0 = inputs([150, 9], [nk + 150, nk], 4, 2, d, int(cap) + nk, size=2.0)
    q[::7] *= 3
    attn = DecodeAttention(4, 2, d)
    out, lse = attn.prefill(q, k, v, dev(q0), dev(k0), softcap=cap, lse=torch.empty(159, 4, device=DEV))
    Q, K, V = f64(q), f64(k), f64(v)
    want, wlse, size = A.prefill(Q, K, V, q0, k0, d ** -0.5, softcap=cap)
    n = 0
    for b in range(2):
        for h in range(4):
            a, e, c, f = q0[b], q0[b + 1], k0[b], k0[b + 1]
            reach = (np.abs(Q[a:e, h]) @ np.abs(K[c:f, h // 2]).T).max(1) * d ** -0.5
            s = np.abs(Q[a:e, h] @ K[c:f, h // 2].T).max(1) * d ** -0.5
            off = (d / 2 + 16) * U * reach + (2.0 ** -19 * cap if cap <= 128 else 2.0 ** -20 * np.minimum(s, cap))
            off = off + 2.0 ** -20 + ((f - c) / 2 + 64) * U
            z, o, wz = f64(lse)[a:e, h], f64(out)[a:e, h], wlse[a:e, h]
            assert (np.isneginf(z) == np.isneginf(wz)).all()  # no visible key
            z, wz = (np.where(np.isneginf(x), 0.0, x) for x in (z, wz))
            assert (np.abs(z - wz) <= off + 2 * U * np.abs(wz)).all(), (np.abs(z - wz) / off).max()
            tol = 2.0 ** -8 * np.abs(want[a:e, h]) + (2.0 ** -8 + 2 * off[:, None]) * size[a:e, h]
            assert (np.abs(o - want[a:e, h]) <= tol).all()
            n += 1
    assert n == 8 and attn.status() == 0


def test_rows_computed_again_for_seconds_are_not_a_hang():
    """One SM, three items: 32 rows over 1.4 million keys whose first value is a NaN take about 3 s to compute
    again, while the other roles wait for the next item's first block; nothing gives up (a wait's limit grows
    with the keys) and the other sequence's outputs are as without the first."""
    n, d = 1_400_000, 64
    q, k, v, q0, k0 = inputs([32, 300], [n, 300], 1, 1, d, 4)
    attn = DecodeAttention(1, 1, d, max_sms=1)
    want, wlse = attn.prefill(q, k, v, dev([32, 332]), dev([n, n + 300]), lse=torch.zeros(332, 1, device=DEV))
    v = v.clone()
    v[0, 0, 3] = float("nan")
    out, lse = attn.prefill(q, k, v, dev(q0), dev(k0), lse=torch.zeros(332, 1, device=DEV))
    assert attn.status() == 0
    assert torch.equal(out[32:], want[32:]) and torch.equal(lse[32:], wlse[32:])
    assert torch.isnan(out[:32, 0, 3]).all()
    # the others' exact values, with f32 weights and sums of 1.4 million
    s = q[:32, 0].double() @ k[:n, 0].double().t() * d ** -0.5
    p = torch.arange(32, device=DEV)[:, None] + n - 32
    s.masked_fill_(torch.arange(n, device=DEV)[None] > p, -float("inf"))
    z = torch.logsumexp(s, 1, keepdim=True)
    w = torch.exp(s - z)
    v[0, 0, 3] = 0
    o, size = w @ v[:n, 0].double(), w @ v[:n, 0].double().abs()
    off = 2.0 ** -16 + (n / 32 + 64) * U  # exponentials, then a sum of n / 32 groups of 32
    keep = [e for e in range(d) if e != 3]
    assert ((out[:32, 0].double() - o).abs() <= 2.0 ** -8 * o.abs() + off * size)[:, keep].all()
    assert ((lse[:32] - z).abs() <= off + 2 * U * z.abs()).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_first_prompt_of_a_context_may_be_captured(d):
    """A context readies the prompts' kernels at its first prompt, which may be a captured one."""
    q, k, v, q0, k0 = inputs([70, 1], [300, 2000], 4, 2, d, 6)
    qs, ks, out = dev(q0), dev(k0), torch.zeros_like(q)
    attn, g = DecodeAttention(4, 2, d), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.prefill(q, k, v, qs, ks, out=out)
    g.replay()
    assert torch.equal(out, DecodeAttention(4, 2, d).prefill(q, k, v, qs, ks)) and attn.status() == 0


def check16(q, k, v, q0, k0, causal=True, softcap=0.0, slopes=None, window=0, scale=None):
    """Weights of 16 bits: each is off by 2^-15 at most besides the scores' errors, so that outputs that are small
    beside their terms keep far more than 8 bits of these."""
    nh, d = q.shape[1:]
    attn = DecodeAttention(nh, k.shape[1], d, prefill_bits=16)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out, _ = attn.prefill(q, k, v, dev(q0), dev(k0), causal=causal, softcap=softcap, slopes=slopes, window=window, scale=scale, lse=lse)
    assert attn.status() == 0
    real, sl = d ** -0.5 if scale is None else scale, None if slopes is None else f64(slopes)
    Q, K, V = f64(q), f64(k), f64(v)
    want, wlse, size = A.prefill(Q, K, V, q0, k0, real, causal, softcap, sl, window)
    o, z = f64(out), f64(lse)
    for b in range(len(q0) - 1):
        a, e, c, f = q0[b], q0[b + 1], k0[b], k0[b + 1]
        for h in range(nh if e > a else 0):
            reach = (np.abs(Q[a:e, h]) @ np.abs(K[c:f, h // (nh // k.shape[1])]).T).max() * abs(real) if f > c else 0.0
            far = 0.0 if sl is None else abs(sl[h]) * max(f - c, e - a)
            off = (d / 2 + 16) * U * reach + (2.0 ** -19 * softcap if softcap <= 128 else 2.0 ** -20 * reach) + 4 * U * far
            off += 2.0 ** -20 + ((f - c) / 2 + 64) * U
            none = np.isneginf(wlse[a:e, h])
            assert (np.isneginf(z[a:e, h]) == none).all()
            w, wz = want[a:e, h], np.where(none, 0, wlse[a:e, h])
            assert (np.abs(np.where(none, 0, z[a:e, h]) - wz) <= off + 2 * U * np.abs(wz)).all()
            bad = np.abs(o[a:e, h] - w) > 2.0 ** -8 * np.abs(w) + (2.0 ** -15 + 2 * off) * size[a:e, h]
            assert not bad.any(), (b, h, int(bad.sum()))
    return attn, out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("nq,nk,nh,nkv", [([1], [1], 2, 2), ([64, 65, 0, 1], [64, 65, 0, 129], 4, 1), ([150, 1, 0, 260, 40], [420, 1, 9, 260, 10], 6, 2),
                                          ([20, 90], [3000, 1000], 8, 2), ([700], [700], 2, 2), ([40, 41], [90, 41], 17, 1)])
def test_weights_of_sixteen_bits(d, nq, nk, nh, nkv):
    check16(*inputs(nq, nk, nh, nkv, d, sum(nk) + d, before=2, behind=3))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window,softcap,slopes,scale,size", [
    (False, 0, 0.0, False, None, 1.0), (True, 100, 0.0, False, None, 2.0), (True, 0, 20.0, False, None, 2.0), (True, 0, 200.0, True, None, 2.0),
    (True, 0, 0.0, True, None, 1.0), (True, 0, 0.0, False, 0.25, 3.0), (False, 37, 5.0, True, -0.2, 1.0)])
@pytest.mark.parametrize("shared", [False, True])
def test_weights_of_sixteen_bits_with_options(d, causal, window, softcap, slopes, scale, size, shared):
    q, k, v, q0, k0 = inputs([20] if shared else [150, 260], [4000] if shared else [420, 260], 6, 2, d, window + d, behind=2, size=size)
    sl = torch.tensor([0.5, 0.25, 0.125, -0.01, 0.0, 2.0], device=DEV) if slopes else None
    check16(q, k, v, q0, k0, causal, softcap, sl, window, scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sixteen_bits_special_values_and_bits_on_demand(d):
    """A NaN that some rows see, infinities in hidden places; the same bits in a graph and after a turn of 8 bits."""
    q, k, v, q0, k0 = inputs([300, 50, 9], [300, 50, 2000], 4, 2, d, 3)
    attn, want = check16(q, k, v, q0, k0)
    qs, ks = dev(q0), dev(k0)
    with pytest.raises(RuntimeError):
        DecodeAttention(4, 2, d, prefill_bits=12)
    eight = DecodeAttention(4, 2, d).prefill(q, k, v, qs, ks)
    assert not torch.equal(eight, want) and (eight.float() - want.float()).abs().max() < 2.0 ** -6 * 5
    assert lib().moe_attn_prefill_bits(attn.handle, 8) == 0
    assert torch.equal(attn.prefill(q, k, v, qs, ks), eight)
    assert lib().moe_attn_prefill_bits(attn.handle, 16) == 0
    out, g = torch.zeros_like(q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn.prefill(q, k, v, qs, ks, out=out)
    g.replay()
    assert torch.equal(out, want)
    v = v.clone()
    v[100, 0, 3], v[349, 1, 0] = float("nan"), float("inf")  # seen by rows 100.. of two heads, by the last row of the second sequence
    got = attn.prefill(q, k, v, qs, ks)
    assert torch.isnan(got[100:300, :2, 3]).all() and torch.isfinite(got[:100]).all() and torch.isfinite(got[300:349]).all()
    assert (got[349, 2:, 0] == float("inf")).all() and torch.isfinite(got[:, 2:, 1:]).all() and attn.status() == 0


def test_a_nan_in_an_early_key_of_a_long_prompt():
    """Nearly every row of two of four heads is computed again: 16 thousand tokens take a fraction of a second, and
    the first row and the other heads are as without it."""
    n = 16384
    q, k, v, q0, k0 = inputs([n], [n], 4, 2, 128, 9)
    attn, s = DecodeAttention(4, 2, 128), dev(q0)
    clean, lse = attn.prefill(q, k, v, s, lse=torch.zeros(n, 4, device=DEV))
    k = k.clone()
    k[1, 0, 5] = float("nan")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out, lse2 = attn.prefill(q, k, v, s, lse=torch.zeros(n, 4, device=DEV))
    end.record()
    assert attn.status() == 0 and start.elapsed_time(end) < 5000
    assert torch.isnan(out[1:, :2]).all() and torch.isnan(lse2[1:, :2]).all()
    assert torch.equal(out[:, 2:], clean[:, 2:]) and torch.equal(lse2[:, 2:], lse[:, 2:])
    assert (out[0].float() - clean[0].float()).abs().max() <= 2.0 ** -8 * 8 and torch.isfinite(lse2[0]).all()
