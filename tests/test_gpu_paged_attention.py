"""Paged-cache attention on the GPU against the f64 oracle: norm and rotation,
cache write and read-back, decode attention.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32):
  * bf16 outputs: half a bf16 step, 2^-8 |exact| (subnormals aside, which the
    data avoids), plus the f32 error of the value itself;
  * norm and rotation: y = x * r * w carries the mean's error (at most 12
    additions deep, halved by the root) and about six more roundings, cos and
    sin 2 u each: 24 u of |a| + |b|, the pair's sizes;
  * e4m3 rows of bf16 input: exact (a power-of-two scale, one rounding), so
    codes and scales are equal.  For normed keys the f32 error may move a value
    over a rounding border, so the read-back is held to half a step, 2^-4
    relative or 2^-10 of the scale below the normal range, plus that error;
  * scores: a d-term f32 sum through 16-wide matrix steps, each charged 8
    units u of the running sum of magnitudes: eps_s = (d / 2 + 16) u reach,
    plus 16 u cap for the tanh and 2 u per unit of distance bias;
  * out: exp and the weights' own rounding are relative errors of p (2^-20
    and, where weights are kept in f16, half a step 2^-11), the sum over n
    keys another (n / 2 + 64) u: all times sum_j p_j |v_j|; lse: eps_s +
    2^-20 + 64 u + 2 u |lse|.
"""
import ctypes

import numpy as np
import pytest
import torch

from fp8_routed_expert_gb300 import C, DecodeAttention, PagedKVCache, lib, rope_frequencies
from oracle import E4M3_TABLE, bf16_to_f64
from oracle import paged_attention as P

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16, spread=0.0):
    x = torch.randn(*shape, generator=g, device=DEV)
    if spread:
        x = x * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g, device=DEV))
    return x.to(dtype)


def close(got, want, tol):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])


# ---------------------------------------------------------- norm, rotation

def _pairs(y, half, inter):
    """Size of each element's pair: |a| + |b| (|a| alone where not rotated)."""
    m = np.abs(y)
    if half:
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        s = m[..., a] + m[..., b]
        m[..., a] = s
        m[..., b] = s
    return m


def _want_rows(x, w, pos, freqs, inter, eps):
    want = P.norm_rope(f64(x), None if w is None else f64(w), None if pos is None else pos.cpu().numpy(), freqs, inter, eps)
    size = P.norm_rope(f64(x), None if w is None else f64(w), None, [], inter, eps)
    return want, 24 * U * _pairs(size, len(freqs), inter)


@pytest.mark.parametrize("T,nh,nkv,d,R,inter,norm", [
    (1, 16, 16, 128, 128, False, True), (3, 1, 1, 64, 64, True, True), (33, 5, 5, 64, 16, False, True),
    (7, 24, 2, 256, 256, True, True), (130, 9, 3, 256, 64, False, True), (257, 32, 8, 128, 96, False, True),
    (5, 48, 8, 128, 0, False, True), (9, 40, 1, 128, 32, True, False), (2, 256, 16, 64, 48, False, True),
    (1031, 6, 2, 128, 128, False, True)])
def test_norm_rope(T, nh, nkv, d, R, inter, norm):
    g = gen(T + nh)
    fused = randn(g, T, nh + 2 * nkv + 1, d, spread=1.0)  # heads of one projection's rows: strided views
    q, k = fused[:, 1:nh + 1], fused[:, nh + 1:nh + nkv + 1]
    wq, wk = (randn(g, d, dtype=torch.float32) for _ in range(2)) if norm else (None, None)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=g, device=DEV).to(torch.int32) if R else None
    freqs = rope_frequencies(R) if R else []
    attn = DecodeAttention(nh, nkv, d, rope_freqs=freqs or None, interleaved=inter)
    want_q, tq = _want_rows(q, wq, pos, freqs, inter, 1e-5)
    want_k, tk = _want_rows(k, wk, pos, freqs, inter, 1e-5)
    # an f64 angle at 2^31 is itself off by up to 2^31 * 2^-53 radians
    tq, tk = (t + 2.0 ** -21 * t / (24 * U) for t in (tq, tk)) if R else (tq, tk)
    qo, ko = attn.norm_rope(q, k, pos, wq, wk, eps=1e-5)
    close(qo, want_q, 2.0 ** -8 * np.abs(want_q) + tq)
    close(ko, want_k, 2.0 ** -8 * np.abs(want_k) + tk)
    assert attn.status() == 0
    # in place, and into strided rows whose neighbours stay as they are
    keep = fused.clone()
    attn.norm_rope(q, k, pos, wq, wk, eps=1e-5, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(fused[:, 0], keep[:, 0]) and torch.equal(fused[:, nh + nkv + 1:], keep[:, nh + nkv + 1:])


def test_rotation_close_to_quarter_turns():
    """Positions whose angles lie next to quarter turns, where a sine or cosine
    is small: right to its own bf16 digits.  Besides their rounding, the angle
    is off by two units of 2^-64 turns per position and by f32 roundings of the
    rest of a quarter turn, of which it and its sine are some 2^-22."""
    pos = [11, 22, 333, 355, 710, 51819, 52174, 103993, 104348, 208341, 260515, 312689, 573204, 833719, 1146408, 4272943, 5419351]
    pos = np.array(pos + [-p for p in pos], np.int32)
    attn = {i: DecodeAttention(1, 1, 64, rope_freqs=[1.0] + [0.0] * 7, interleaved=i) for i in (False, True)}
    x = torch.zeros(len(pos), 1, 64, dtype=torch.bfloat16, device=DEV)
    x[..., 0] = 1.0
    far = np.abs(pos.astype(np.float64)) * (2 * np.pi * 2.0 ** -63)
    for inter, second in ((False, 8), (True, 1)):
        for y in attn[inter].norm_rope(x, x, torch.from_numpy(pos).to(DEV)):
            for at, want in ((0, np.cos(pos.astype(np.float64))), (second, np.sin(pos.astype(np.float64)))):
                close(y[:, 0, at], want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + far)


def test_norm_rope_special_rows():
    """Zeros stay zeros, large and tiny rows are normed within f32, NaN stays
    within its row."""
    attn = DecodeAttention(4, 2, 64)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 1] = 1e18
    q[0, 2] = 1e-15
    q[1, 0, 5] = float("nan")
    k = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, device=DEV)
    qo, ko = attn.norm_rope(q, k, None, w, w, eps=0.0)
    assert torch.isnan(qo[0, 0]).all() and torch.isnan(qo[1, 0]).all()  # 0 / 0 without an eps
    assert (qo[0, 1] == 1).all() and (qo[0, 2] == 1).all() and (ko == 1).all()
    qo, _ = attn.norm_rope(q, k, None, w, w, eps=1e-6)
    assert (qo[0, 0] == 0).all() and (qo[1, 1:] == 0).all()


# ------------------------------------------------------------------- cache

def make_cache(n_pages, page, nkv, d, fmt, layout="head", fill=None):
    """A cache whose tensors are views of a larger block: pages outermost and
    heads or slots next, or one layer of two interleaved per slot."""
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8

    def block(last, dtype):
        if layout == "head":
            t = torch.empty(n_pages, nkv, page, *last, dtype=dtype, device=DEV)
        elif layout == "slot":
            t = torch.empty(n_pages, page, nkv, *last, dtype=dtype, device=DEV).transpose(1, 2)
        else:
            t = torch.empty(n_pages, page, 2, nkv, *last, dtype=dtype, device=DEV)[:, :, 1].transpose(1, 2)
        return t

    kv = [block((d,), dt) for _ in range(2)]
    sc = [block((), torch.float32) for _ in range(2)] if fmt == "e4m3" else []
    if fill is not None:
        for t in kv:
            t.fill_(fill if fmt == "bf16" else 0x7F)
        for t in sc:
            t.fill_(fill)
    return PagedKVCache(*kv, *sc)


def cache_values(cache, which):
    """f64 [n_pages, n_kv, page, d] that the cache stands for."""
    t, s = (cache.k, cache.k_scale) if which == 0 else (cache.v, cache.v_scale)
    if cache.format == "bf16":
        return f64(t)
    table = np.asarray(E4M3_TABLE, dtype=np.float64)
    return table[t.cpu().numpy()] * f64(s)[..., None]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,nkv,d,page,layout", [(1, 16, 128, 16, "head"), (37, 3, 64, 24, "slot"), (65, 1, 256, 1, "head"),
                                                 (513, 8, 128, 100, "layer"), (2, 32, 64, 7, "slot"), (1500, 2, 128, 64, "head")])
def test_write_and_read(T, nkv, d, page, layout, fmt):
    g = gen(T)
    kv = randn(g, T, 2 * nkv, d, spread=2.0)
    k, v = kv[:, :nkv], kv[:, nkv:]
    v[0, 0] = 0.0
    n_pages = -(-2 * T // page) + 1
    slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T].contiguous()
    slots[T // 2] = -1 - T if T > 1 else slots[0]
    cache = make_cache(n_pages, page, nkv, d, fmt, layout, fill=3.0)
    before = cache.k.clone()
    attn = DecodeAttention(nkv, nkv, d)
    attn.write(cache, k, v, slots)
    assert attn.status() == 0
    sl = slots.cpu().numpy()
    on = sl >= 0
    p, r = sl[on] // page, sl[on] % page
    for x, t, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        if fmt == "bf16":
            assert torch.equal(t[p, :, r], x[torch.from_numpy(on).to(DEV)])
        else:
            codes, scale = P.e4m3_row(f64(x)[on])
            assert np.array_equal(t[p, :, r].cpu().numpy(), codes)
            assert np.array_equal(f64(s[p, :, r]), scale)
    # nothing else was touched
    rest = np.ones((n_pages, page), bool)
    rest[p, r] = False
    rp, rr = np.nonzero(rest)
    assert torch.equal(cache.k[rp, :, rr].view(torch.uint8), before[rp, :, rr].view(torch.uint8))
    # reading back: the values, rounded once
    for x, o in zip((k, v), attn.read(cache, slots)):
        if fmt == "bf16":
            want = torch.where((slots >= 0)[:, None, None], x, torch.zeros_like(x))
        else:
            codes, scale = P.e4m3_row(f64(x))
            val = np.asarray(E4M3_TABLE)[codes] * scale[..., None] * on[:, None, None]
            want = torch.from_numpy(val).to(torch.bfloat16).to(DEV)
        assert torch.equal(o, want)


def test_write_rows_that_are_not_finite():
    attn = DecodeAttention(1, 1, 64)
    cache = make_cache(2, 4, 1, 64, "e4m3", fill=1.0)
    k = torch.full((3, 1, 64), 2.0, dtype=torch.bfloat16, device=DEV)
    k[0, 0, 3] = float("inf")
    k[1, 0, 60] = float("nan")
    k[2] = float("-inf")
    attn.write(cache, k, k, torch.tensor([1, 2, 3], device=DEV))
    ko, vo = attn.read(cache, torch.tensor([1, 2, 3], device=DEV))
    assert torch.equal(torch.isnan(ko), ~torch.isfinite(k)) and torch.equal(torch.isnan(vo), ~torch.isfinite(k))
    assert (ko[torch.isfinite(k)] == 2.0).all() and (cache.k_scale[0, 0, 3] == 1.0)


def test_slots_outside_the_cache_are_left_out_and_reported():
    attn = DecodeAttention(2, 1, 64)
    for fmt in ("bf16", "e4m3"):
        cache = make_cache(2, 8, 1, 64, fmt, fill=1.0)
        before = cache.k.clone()
        x = randn(gen(1), 4, 1, 64)
        bad = torch.tensor([16, 2 ** 31, 2 ** 62, -5], device=DEV)
        attn.write(cache, x, x, bad)
        assert attn.status() == C["MOE_ERR_DEVICE"] and attn.status() == 0
        assert torch.equal(cache.k.view(torch.uint8), before.view(torch.uint8))
        ko, vo = attn.read(cache, bad)
        assert (ko == 0).all() and (vo == 0).all() and attn.status() == C["MOE_ERR_DEVICE"]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,nh,nkv,d,R,inter", [(1, 16, 16, 128, 128, False), (40, 12, 4, 64, 32, True), (257, 7, 1, 256, 128, False)])
def test_append(T, nh, nkv, d, R, inter, fmt):
    g = gen(T + d)
    fused = randn(g, T, nh + 2 * nkv, d, spread=1.0)
    q, k, v = fused[:, :nh], fused[:, nh:nh + nkv], fused[:, nh + nkv:]
    wq, wk = 1 + 0.3 * randn(g, d, dtype=torch.float32), 1 + 0.3 * randn(g, d, dtype=torch.float32)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV).to(torch.int32)
    freqs = rope_frequencies(R)
    cache = make_cache(T + 2, 3, nkv, d, fmt, "slot", fill=7.0)
    slots = torch.randperm(3 * (T + 2), generator=g, device=DEV)[:T].contiguous()
    if T > 1:
        slots[1] = -1
    attn = DecodeAttention(nh, nkv, d, rope_freqs=freqs, interleaved=inter)
    qo = attn.append(q, k, v, pos, slots, cache, wq, wk)
    assert attn.status() == 0
    qn, kn = attn.norm_rope(q, k, pos, wq, wk)
    assert torch.equal(qo, qn)
    on = (slots >= 0).cpu().numpy()
    sl = slots.cpu().numpy()[on]
    at = (sl // 3, slice(None), sl % 3)
    want, tol = _want_rows(k, wk, pos, freqs, inter, 1e-6)
    if fmt == "bf16":
        assert torch.equal(cache.k[at], kn[torch.from_numpy(on).to(DEV)])
        assert torch.equal(cache.v[at], v[torch.from_numpy(on).to(DEV)])
        return
    codes, scale = P.e4m3_row(f64(v)[on])
    assert np.array_equal(cache.v[at].cpu().numpy(), codes) and np.array_equal(f64(cache.v_scale[at]), scale)
    got, sc = cache_values(cache, 0)[at], f64(cache.k_scale[at])
    want, tol = want[on], tol[on]
    # the row's scale: the smallest power of two that holds the largest value, to its error
    amax, slack = np.abs(want).max(-1), tol.max(-1)
    assert (amax - slack <= 448 * sc).all() and (amax + slack > 224 * sc).all() and (np.log2(sc) % 1 == 0).all()
    half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * sc[..., None])
    bad = np.abs(got - want) > half + tol * (1 + 2.0 ** -4)
    assert not bad.any(), np.argwhere(bad)[:4]


# ------------------------------------------------------------------ decode

class Batch:
    """Sequences over a shared cache, everything that no sequence sees set to NaN."""

    def __init__(self, lens, nh, nkv, d, fmt, page, layout="head", seed=0, width=None, hidden=None):
        self.lens, self.nh, self.nkv, self.d, self.fmt, self.page = list(lens), nh, nkv, d, fmt, page
        g = gen(seed)
        B = len(self.lens)
        used = [-(-max(n, 0) // page) for n in self.lens]
        n_pages = sum(used) + 2
        self.width = width or max(1, max(used))
        self.cache = make_cache(n_pages, page, nkv, d, fmt, layout, fill=float("nan"))
        order = torch.randperm(n_pages, generator=g, device=DEV).cpu().numpy()
        table = np.full((B, self.width + 3), 2 ** 30, np.int32)  # never read: past each length
        self.q = randn(g, B, nh + 1, d, spread=0.5)[:, :nh]
        self.K, self.V = [], []
        attn = DecodeAttention(nkv, nkv, d)
        at = 0
        for b, n in enumerate(self.lens):
            mine = order[at:at + used[b]]
            at += used[b]
            table[b, :used[b]] = mine
            j = np.arange(n)
            slots = mine[j // page].astype(np.int64) * page + j % page if n else np.zeros(0, np.int64)
            k, v = (randn(g, n, nkv, d, spread=0.7) for _ in range(2))
            if n:
                attn.write(self.cache, k, v, torch.from_numpy(slots).to(DEV))
            if fmt == "e4m3" and n:
                (kc, ks), (vc, vs) = P.e4m3_row(f64(k)), P.e4m3_row(f64(v))
                tab = np.asarray(E4M3_TABLE, np.float64)
                self.K.append(tab[kc] * ks[..., None])
                self.V.append(tab[vc] * vs[..., None])
            else:
                self.K.append(f64(k))
                self.V.append(f64(v))
        assert attn.status() == 0
        self.table = torch.from_numpy(table).to(DEV)[:, :self.width]  # rows with a stride
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def run(self, attn=None, **kw):
        attn = attn or DecodeAttention(self.nh, self.nkv, self.d)
        lse = torch.full((len(self.lens), self.nh), 123.0, device=DEV)
        out, lse = attn.decode(self.q, self.cache, self.table, self.seq_lens, lse=lse, **kw)
        assert attn.status() == 0
        return out, lse

    def check(self, attn=None, **kw):
        out, lse = self.run(attn, **kw)
        host = {k: (f64(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
        want, wl, mag, reach = P.decode(f64(self.q), self.K, self.V, self.lens, **host)
        cap, slopes = kw.get("softcap", 0.0), host.get("slopes")
        n = max(max(self.lens), 1)
        eps_s = (self.d / 2 + 16) * U * reach + 16 * U * cap
        if slopes is not None:
            eps_s = eps_s + 2 * U * np.abs(slopes) * n
        rel = 2 * eps_s + 2.0 ** -20 + (n / 2 + 64) * U + (2.0 ** -11 if self.fmt == "e4m3" else 2.0 ** -16)
        close(out, want, 2.0 ** -8 * np.abs(want) + rel[..., None] * mag + 1e-30)
        got = f64(lse)
        empty = np.isneginf(wl)
        assert (np.isneginf(got) == empty).all()
        err = np.abs(got[~empty] - wl[~empty])
        tol = (eps_s + 2.0 ** -20 + 64 * U + 2 * U * np.abs(np.where(empty, 0, wl)))[~empty]
        assert (err <= tol).all(), (err.max(), tol[err.argmax()])
        return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 200]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d,page,layout", [
    (16, 16, 128, 16, "head"), (8, 8, 64, 1, "head"), (4, 2, 256, 24, "slot"), (15, 3, 128, 64, "layer"),
    (32, 4, 64, 7, "slot"), (12, 1, 128, 100, "head"), (16, 1, 256, 8, "head"), (48, 2, 64, 32, "slot"),
    (17, 1, 128, 16, "layer"), (9, 1, 256, 256, "head")])
def test_decode_edges(nh, nkv, d, page, layout, fmt):
    """Lengths around every tile and page border, every head grouping, masks
    that leave rows empty, and NaN wherever no sequence looks."""
    b = Batch(EDGES, nh, nkv, d, fmt, page, layout, seed=nh + d)
    attn = DecodeAttention(nh, nkv, d)
    b.check(attn)
    starts = torch.tensor([0, 1, 0, 3, 16, 5, 62, 64, 1, 99, -7, 16, 300, 65], dtype=torch.int32, device=DEV)
    slopes = torch.linspace(0.01, 0.5, nh, device=DEV)
    b.check(attn, starts=starts, softcap=30.0)
    b.check(attn, slopes=slopes, window=17)
    b.check(attn, starts=starts, window=1, scale=0.3)
    b.check(attn, starts=starts, window=64, slopes=slopes, softcap=5.0, scale=-0.1)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,nh,nkv,d,page", [
    ([5000], 4, 1, 128, 16), ([4096, 3], 16, 16, 64, 64), ([777, 20000, 1, 0, 333], 8, 2, 128, 48),
    ([2500] * 3, 10, 1, 256, 128)])
def test_decode_split_over_the_length(lens, nh, nkv, d, page, fmt):
    b = Batch(lens, nh, nkv, d, fmt, page, seed=len(lens))
    attn = DecodeAttention(nh, nkv, d)
    one = b.check(attn)
    b.check(attn, window=1999, softcap=20.0)
    # the same bits again, whatever ran in between, and on fewer SMs the same result to rounding
    again = b.run(attn)
    assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])
    b.check(DecodeAttention(nh, nkv, d, max_sms=7))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,nh,nkv,d,page", [
    ([9000, 10, 0, 4000], 6, 2, 128, 16), ([700] * 40, 5, 1, 64, 24), ([30001], 16, 1, 256, 64),
    ([i * 53 % 1500 for i in range(150)], 4, 2, 64, 32), ([6000, 6001], 12, 1, 128, 32)])
def test_decode_small_pieces(lens, nh, nkv, d, page, fmt):
    """Few SMs, so that each warp's piece of the list holds many segments: the same
    bits every time, and correct."""
    b = Batch(lens, nh, nkv, d, fmt, page, seed=len(lens) + d)
    for sms in (1, 3):
        attn = DecodeAttention(nh, nkv, d, max_sms=sms)
        one = b.check(attn, softcap=25.0)
        for _ in range(3):
            again = b.run(attn, softcap=25.0)
            assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


def test_decode_one_very_long_sequence():
    """One key/value head, 150001 keys: the split's deepest join."""
    for fmt in ("bf16", "e4m3"):
        Batch([150001], 2, 1, 64, fmt, 128, seed=5).check()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_many_sequences(fmt):
    lens = [(i * 37) % 150 for i in range(700)]
    Batch(lens, 4, 2, 64, fmt, 16, seed=9).check()


def test_decode_sharp_and_extreme_scores():
    """One key far above the rest, late or early; scores beyond f32 exp; value
    rows of very different sizes."""
    for fmt in ("bf16", "e4m3"):
        b = Batch([300, 300], 4, 2, 128, fmt, 16, seed=3)
        b.check(scale=60.0)
        b.check(scale=1e-30)
        b = Batch([200], 2, 2, 64, fmt, 16, seed=4)
        # the largest value row is one that no weight falls on
        attn = DecodeAttention(2, 2, 64)
        big = torch.full((1, 2, 64), 1.0e9, dtype=torch.bfloat16, device=DEV)
        key = (-1e3 * torch.sign(b.q[0].float())).to(torch.bfloat16)[None]
        slot = b.table[0, 0].long().view(1) * 16 + 3
        attn.write(b.cache, key, big, slot)
        b.K[0][3] = f64(key)[0] if fmt == "bf16" else cache_values(b.cache, 0)[int(b.table[0, 0]), :, 3]
        b.V[0][3] = cache_values(b.cache, 1)[int(b.table[0, 0]), :, 3]
        b.check()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_nan_stays_in_its_sequence(fmt):
    b = Batch([40, 80, 200], 4, 2, 64, fmt, 16, seed=8)
    clean, _ = b.run()
    attn = DecodeAttention(4, 2, 64)
    x = randn(gen(2), 1, 2, 64)
    y = x.clone()
    y[0, 1, 7] = float("nan")
    attn.write(b.cache, x, y, b.table[1, 2].long().view(1) * 16 + 5)  # position 37 of sequence 1
    out, _ = b.run()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
    assert torch.isfinite(out[1, :2]).all()
    assert torch.isnan(out[1, 2:, 7]).all() and torch.isfinite(out[1, 2:, :7]).all()
    # hidden by a start, it is not seen
    seen, _ = b.run(starts=torch.tensor([0, 38, 0], dtype=torch.int32, device=DEV))
    assert torch.isfinite(seen).all()
    # a NaN key makes its heads NaN
    attn.write(b.cache, y, x, b.table[1, 2].long().view(1) * 16 + 5)
    out, lse = b.run()
    assert torch.isnan(out[1, 2:]).all() and torch.isnan(lse[1, 2:]).all() and torch.isfinite(out[1, :2]).all()


def test_decode_reports_pages_and_lengths_outside():
    for fmt in ("bf16", "e4m3"):
        b = Batch([50, 70, 33], 4, 4, 64, fmt, 16, seed=6, width=6)
        attn = DecodeAttention(4, 4, 64)
        clean = attn.decode(b.q, b.cache, b.table, b.seq_lens)
        assert attn.status() == 0
        for bad in (-1, b.cache.n_pages, 2 ** 31 - 1):
            table = b.table.clone()
            table[1, 2] = bad
            out = attn.decode(b.q, b.cache, table, b.seq_lens)
            assert attn.status() == C["MOE_ERR_DEVICE"]
            assert torch.equal(out[0], clean[0]) and torch.equal(out[2], clean[2])
            K, V = b.K[1].copy(), b.V[1].copy()
            K[32:48] = V[32:48] = 0  # a page outside counts as zeros
            want, _, mag, _ = P.decode(f64(b.q)[1:2], [K], [V], [70])
            close(out[1:2], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag)
        # a length outside the table is cut to it, a negative one is empty
        table = b.table.clone()
        table[:, 5:] = 0
        table[0, 4:] = 0
        attn.decode(b.q, b.cache, table.clamp(0, b.cache.n_pages - 1), torch.tensor([50, 97, -3], dtype=torch.int32, device=DEV))
        assert attn.status() == C["MOE_ERR_DEVICE"]
        out = attn.decode(b.q, b.cache, b.table, torch.tensor([50, 70, -3], dtype=torch.int32, device=DEV))
        assert attn.status() == C["MOE_ERR_DEVICE"] and (out[2] == 0).all() and torch.equal(out[:2], clean[:2])


def test_decode_far_offsets():
    """Rows beyond 2^32 elements into the cache."""
    n_pages, page, d = 300, 64, 128
    stride = 1 << 24  # elements between pages: 300 pages span 5e9
    big = [torch.empty(n_pages * stride, dtype=torch.uint8, device=DEV) for _ in range(2)]
    kv = [t.as_strided((n_pages, 1, page, d), (stride, page * d, d, 1)) for t in big]
    sc = [torch.empty(n_pages, 1, page, device=DEV) for _ in range(2)]
    cache = PagedKVCache(*kv, *sc)
    attn = DecodeAttention(3, 1, d)
    g = gen(1)
    k, v, q = randn(g, 100, 1, d), randn(g, 100, 1, d), randn(g, 1, 3, d)
    table = torch.tensor([[299, 290]], dtype=torch.int32, device=DEV)
    j = torch.arange(100, device=DEV)
    slots = table[0].long()[j // page] * page + j % page
    attn.write(cache, k, v, slots)
    out = attn.decode(q, cache, table, torch.tensor([100], dtype=torch.int32, device=DEV))
    ko, vo = attn.read(cache, slots)
    assert attn.status() == 0
    (kc, ks), (vc, vs) = P.e4m3_row(f64(k)), P.e4m3_row(f64(v))
    tab = np.asarray(E4M3_TABLE)
    K, V = tab[kc] * ks[..., None], tab[vc] * vs[..., None]
    assert np.array_equal(f64(ko), K) and np.array_equal(f64(vo), V)  # e4m3 times 2^e fits bf16
    want, _, mag, _ = P.decode(f64(q), [K], [V], [100])
    close(out, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag)


def test_step_in_a_graph_and_on_another_stream():
    """append and decode captured once, replayed as the sequences grow, give
    the eager bits."""
    B, nh, nkv, d, page = 3, 8, 2, 128, 16
    g = gen(3)
    attn = DecodeAttention(nh, nkv, d, rope_freqs=rope_frequencies(d))
    w = torch.ones(d, device=DEV)
    table = torch.randperm(B * 40, generator=g, device=DEV).to(torch.int32).view(B, 40)
    steps = [randn(g, B, nh + 2 * nkv, d) for _ in range(5)]
    caches = [make_cache(B * 40, page, nkv, d, "e4m3", fill=1.0) for _ in range(2)]
    for c in caches:
        c.k.zero_()
        c.v.zero_()
    x = steps[0].clone()
    pos = torch.tensor([0, 30, 500], dtype=torch.int32, device=DEV)
    start_pos = pos.clone()
    lens = torch.empty_like(pos)
    out = torch.empty(B, nh, d, dtype=torch.bfloat16, device=DEV)

    def step(cache, stream=None):
        torch.add(pos, 1, out=lens)
        page_of = table.gather(1, (pos // page).long()[:, None])[:, 0].long()
        slots = page_of * page + pos % page
        q = attn.append(x[:, :nh], x[:, nh:nh + nkv], x[:, nh + nkv:], pos, slots, cache, w, w, stream=stream)
        attn.decode(q, cache, table, lens, out=out, stream=stream)
        pos.add_(1)

    eager = []
    for s in steps:
        x.copy_(s)
        step(caches[0])
        eager.append(out.clone())
    assert attn.status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pos.copy_(start_pos)
        step(caches[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[1])
    pos.copy_(start_pos)
    for s, want in zip(steps, eager):
        x.copy_(s)
        graph.replay()
        assert torch.equal(out, want)
    assert attn.status() == 0


def test_python_layer_refusals():
    attn = DecodeAttention(4, 2, 64, rope_freqs=rope_frequencies(64))
    cache = PagedKVCache.empty(4, 16, 2, 64, "e4m3")
    bf = torch.bfloat16
    q, k = torch.zeros(3, 4, 64, dtype=bf, device=DEV), torch.zeros(3, 2, 64, dtype=bf, device=DEV)
    pos, slots = torch.zeros(3, dtype=torch.int32, device=DEV), torch.arange(3, device=DEV)
    table, lens = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.ones(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: attn.norm_rope(q.float(), k, pos), lambda: attn.norm_rope(q, k[:2], pos),
                lambda: attn.norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos),
                lambda: attn.norm_rope(q, k, None), lambda: attn.norm_rope(q, k, pos.long()),
                lambda: attn.norm_rope(q.cpu(), k, pos), lambda: attn.norm_rope(q, k, pos, torch.ones(32, device=DEV)),
                lambda: attn.append(q, k, k, pos, slots.int(), cache), lambda: attn.write(cache, k, k[:, :1], slots),
                lambda: attn.write(cache, k, k, slots[:2]), lambda: attn.read(cache, slots, k_out=q),
                lambda: attn.decode(q, cache, table.long(), lens), lambda: attn.decode(q, cache, table[:2], lens),
                lambda: attn.decode(q, cache, table, lens.long()), lambda: attn.decode(q, cache, table, lens[:1]),
                lambda: attn.decode(q, cache, table, lens, slopes=torch.ones(2, device=DEV)),
                lambda: attn.decode(q, cache, table, lens, out=k), lambda: attn.decode(q, cache, table, None),
                lambda: attn.decode(q, cache, table, lens, lse=torch.ones(3, 4, dtype=torch.float64, device=DEV)),
                lambda: DecodeAttention(8, 4, 64).decode(q, cache, table, lens),
                lambda: PagedKVCache(cache.k, cache.v), lambda: PagedKVCache(cache.k.float(), cache.v.float()),
                lambda: PagedKVCache(cache.k, cache.v[:, :1], cache.k_scale, cache.v_scale),
                lambda: PagedKVCache.empty(1, 16, 2, 64, "fp4")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(Exception, match="moe_attn_decode"):
        attn.decode(q, cache, table, lens, softcap=-1.0)
    with pytest.raises(Exception, match="moe_attn_init"):
        DecodeAttention(4, 3, 64)
    # nothing to do
    none = torch.zeros(0, 4, 64, dtype=bf, device=DEV)
    assert attn.decode(none, cache, table[:0], lens[:0]).shape == (0, 4, 64)
    attn.write(cache, none[:, :2], none[:, :2], slots[:0])
    assert attn.status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d", [(8, 2, 64), (12, 12, 128), (16, 1, 128), (5, 1, 256), (40, 2, 64), (18, 1, 256)])
def test_decode_both_ways_of_small_calls(nh, nkv, d, fmt):
    """A page table that only just covers the lengths (clusters of CTAs per
    segment) and one that could hold far longer sequences (the cut list): the
    oracle's result both times, to the same bits every time."""
    attn = DecodeAttention(nh, nkv, d)
    for lens in ([1, 1000], [500, 0, 33], [64], [2, 31, 32, 33]):
        for width in (None, 2000):
            b = Batch(lens, nh, nkv, d, fmt, 16, seed=nh + len(lens), width=width)
            one = b.check(attn, softcap=20.0)
            again = b.run(attn, softcap=20.0)
            assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])
            b.check(attn, starts=torch.tensor([5] * len(lens), dtype=torch.int32, device=DEV), window=300)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d,B", [(32, 8, 64, 5), (12, 6, 128, 12), (36, 4, 128, 9), (8, 8, 64, 30), (60, 4, 64, 35),
                                        (5, 5, 256, 25), (16, 16, 128, 19)])
def test_decode_clusters_of_all_sizes(nh, nkv, d, B, fmt):
    """As many segments as leave clusters of eight, four, two CTAs or one,
    lengths from none to some tiles per warp: the oracle's result, to the same
    bits every time."""
    attn = DecodeAttention(nh, nkv, d)
    for S in (40, 300, 900):
        lens = [S * (i + 1) // B if i % 5 != 3 else i % 2 for i in range(B)]
        b = Batch(lens, nh, nkv, d, fmt, 16, seed=S + B)
        one = b.check(attn)
        again = b.run(attn)
        assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d,lens", [(4, 1, 64, [5000]), (7, 1, 128, [9000]), (6, 3, 128, [4097]), (8, 4, 256, [5001, 20]),
                                           (16, 4, 64, [9001, 0, 129]), (64, 4, 128, [30000, 2001]),
                                           (18, 2, 64, [9000, 1]), (64, 4, 128, [6000, 100, 3000, 0, 5999, 31])])
def test_decode_clusters_that_share_a_segment(nh, nkv, d, lens, fmt):
    """Sequences long enough for several clusters, and lengths that leave some of
    them nothing: the oracle's result, to the same bits every time."""
    attn = DecodeAttention(nh, nkv, d)
    for n in (lens, [x - x // 3 for x in lens], [min(x, 700) for x in lens], [min(x, 1) for x in lens]):
        b = Batch(n, nh, nkv, d, fmt, 16, seed=nh + d, width=(max(lens) + 15) // 16)
        one = b.check(attn)
        again = b.run(attn)
        assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])
        b.check(attn, starts=torch.tensor([9] * len(lens), dtype=torch.int32, device=DEV), window=3000)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_contexts_on_two_streams(fmt):
    """Contexts of their own on streams of their own, at the same time: the
    bits that each gives alone."""
    batches = [Batch([3000, 10, 700], 8, 2, 128, fmt, 32, seed=1), Batch([900] * 6, 4, 4, 64, fmt, 16, seed=2)]
    attns = [DecodeAttention(b.nh, b.nkv, b.d) for b in batches]
    alone = [b.run(a)[0].clone() for a, b in zip(attns, batches)]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w) for _ in range(10)] for w in alone]
    for i in range(10):
        for a, b, s, o in zip(attns, batches, streams, outs):
            a.decode(b.q, b.cache, b.table, b.seq_lens, out=o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(alone, outs):
        assert all(torch.equal(w, x) for x in o)
    assert all(a.status() == 0 for a in attns)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_example_step(fmt):
    """The example block: MoE beside the attention on another stream gives the
    bits of one stream, and the attention the oracle's result."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "scmoe_paged_decode.py")
    spec = importlib.util.spec_from_file_location("scmoe_paged_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    blocks = [ex.Block(3, 200, fmt, seed=4) for _ in range(2)]
    x = randn(gen(5), 3, blocks[0].hidden)
    for b in blocks:
        b.prompt(torch.tensor([150, 0, 33]))
    for _ in range(3):
        y = [b.step(x, overlap=i == 0) for i, b in enumerate(blocks)]
        assert torch.equal(y[0], y[1]) and torch.isfinite(y[0]).all()
    b = blocks[0]
    assert b.attn.status() == 0 and b.moe.status() == 0 and b.pos.tolist() == [153, 3, 36]
    # the third step's attention again, from what the cache holds
    qkv = (x @ b.w_qkv.T).view(3, -1, b.d)
    q, _ = b.attn.norm_rope(*b._heads(qkv)[:2], b.pos - 1, b.q_norm, b.k_norm)
    out = b.attn.decode(q, b.cache, b.table, b.pos)
    K, V = [], []
    for s, n in enumerate(b.pos.tolist()):
        j = torch.arange(n, device=DEV)
        k, v = b.attn.read(b.cache, b.table[s].long()[j // ex.PAGE] * ex.PAGE + j % ex.PAGE)
        K.append(f64(k))
        V.append(f64(v))
    want, _, mag, _ = P.decode(f64(q), K, V, b.pos.tolist())
    close(out, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag)


@pytest.mark.parametrize("fmt,big,nats", [("bf16", 1e9, 0.0), ("bf16", 1e30, 0.0), ("bf16", 1.0, 30.0),
                                          ("e4m3", 1e9, 0.0), ("e4m3", 1.0, 20.0)])
@pytest.mark.parametrize("nh,nkv,d", [(4, 2, 64), (16, 1, 64), (6, 2, 128), (12, 1, 128), (3, 1, 256)])
def test_decode_columns_that_the_heaviest_rows_leave_empty(nh, nkv, d, fmt, big, nats):
    """A value row that is far larger than the others, or whose key is far ahead,
    with zeros in all columns but one: the other columns are the sums of much
    smaller weights and keep their digits, each for itself.  Weights in 16 bits
    (2^-16), and for e4m3 off by 2^-48 of the largest weight times its value's
    scale, 448 of which are at most twice the large value; the rest as for all
    decode tests."""
    b = Batch([150, 700], nh, nkv, d, fmt, 16, seed=nh + d)
    b.q.copy_(b.q[:, :1].clone().expand(-1, nh, -1))
    attn = DecodeAttention(nh, nkv, d)
    for s, at in ((0, 3), (1, 411)):
        q = b.q[s, 0].double()
        key = (q * (nats * d ** 0.5 / float(q @ q))).to(torch.bfloat16).expand(1, nkv, d).contiguous()
        row = torch.zeros(1, nkv, d, dtype=torch.bfloat16, device=DEV)
        row[..., 1] = big
        page = int(b.table[s, at // 16])
        attn.write(b.cache, key, row, torch.tensor([16 * page + at % 16], device=DEV))
        b.K[s][at] = cache_values(b.cache, 0)[page, :, at % 16]
        b.V[s][at] = cache_values(b.cache, 1)[page, :, at % 16]
    out, _ = b.run(attn)
    want, _, mag, reach = P.decode(f64(b.q), b.K, b.V, b.lens)
    rel = 2 * (d / 2 + 16) * U * reach + 2.0 ** -20 + (700 / 2 + 64) * U + 2.0 ** -16
    tol = 2.0 ** -8 * np.abs(want) + rel[..., None] * mag
    if fmt == "e4m3":
        tol = tol + 2.0 ** -47 * 700 * mag[..., 1:2]
    close(out, want, tol)


def test_outputs_are_of_the_calls_stream():
    """A call on another stream than the current one: memory that the current
    stream's queued work still uses is not handed out for its outputs."""
    T, nh, nkv, d = 64, 8, 2, 128
    b = Batch([40] * T, nh, nkv, d, "bf16", 16, seed=11)
    attn = DecodeAttention(nh, nkv, d)
    want, rows = b.run(attn)[0].clone(), randn(gen(4), T, nkv, d)
    slots = torch.arange(T, device=DEV)
    nowhere = -1 - slots
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    calls = {"norm_rope": lambda **k: attn.norm_rope(b.q, rows, None, **k)[0],
             "append": lambda **k: attn.append(b.q, rows, rows, None, nowhere, b.cache, **k),
             "decode": lambda **k: attn.decode(b.q, b.cache, b.table, b.seq_lens, **k),
             "read": lambda **k: attn.read(b.cache, slots, **k)[0]}
    for name, call in calls.items():
        for stream in (side, side.cuda_stream):
            old = torch.empty(T, nh if name != "read" else nkv, d, dtype=torch.bfloat16, device=DEV)
            at = old.data_ptr()
            torch.cuda._sleep(2_000_000)
            old.fill_(1.0)  # queued behind the sleep
            del old
            out = call(stream=stream)
            assert out.data_ptr() != at
            side.synchronize()
            if name == "decode":
                assert torch.equal(out, want)
            elif name != "read":
                assert torch.equal(out, b.q)
            torch.cuda.synchronize()
    assert attn.status() == 0


def test_rotation_by_negative_frequencies():
    """A negative frequency undoes what its opposite does, at positions up to the
    ends of the int32 range: each angle lies 2^-17 or so beside a half turn, so that
    its sine shows an error of the angle in its own bf16 digits.  The angle is off
    by 2^-64 turns per position, and by f32 roundings of its rest."""
    from fractions import Fraction
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    at = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 10 ** 9 + 7]
    freqs = [-(float(pi) * (2 * i + 1) + 1e-5 * (i + 1)) / abs(p) for p in at for i in range(2)]
    x = torch.zeros(len(at), 1, 64, dtype=torch.bfloat16, device=DEV)
    x[..., :8] = 1.0  # the first elements of the pairs
    pos = torch.tensor(at, dtype=torch.int32, device=DEV)
    back = DecodeAttention(1, 1, 64, rope_freqs=freqs)
    forth = DecodeAttention(1, 1, 64, rope_freqs=[-f for f in freqs])
    want = np.zeros((len(at), 8))
    for t, p in enumerate(at):
        for i, f in enumerate(freqs):
            a = Fraction(f) * p
            turns = round(a / pi)
            want[t, i] = (-1) ** turns * np.sin(float(a - turns * pi))
    assert (np.abs(want) < 2e-5).sum() >= 8
    far = np.abs(np.array(at, np.float64))[:, None] * (2 * np.pi * 2.0 ** -64)
    y, z = back.norm_rope(x, x, pos)[0], forth.norm_rope(x, x, pos)[0]
    close(y[:, 0, 8:16], want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + far)
    close(z[:, 0, 8:16], -want, (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + far)
    assert torch.equal(y[:, 0, :8], z[:, 0, :8]) and torch.equal(y[:, 0, 8:16], -z[:, 0, 8:16])


@pytest.mark.parametrize("d,R,inter", [(64, 0, False), (128, 128, False), (256, 64, True)])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
def test_norm_of_rows_whose_squares_leave_f32(d, R, inter, eps):
    """Rows up to bf16's largest value and down to its smallest: their sum of
    squares is beyond f32 or below it, their norm is not.  Large rows (and tiny
    ones where eps is as small) have outputs like any other's; ordinary rows and
    rows with infinities beside them stay as they are."""
    nh = nkv = 6
    g = gen(d)
    sizes = torch.tensor([2.0 ** 126, 2.0 ** 64, 1.0, 2.0 ** -60, 2.0 ** -80, 2.0 ** -120], device=DEV)
    x = torch.rand(7, nh, d, generator=g, device=DEV) + 0.5  # within a factor of three
    x = x * torch.where(torch.rand(7, nh, d, generator=g, device=DEV) < 0.5, -1.0, 1.0) * sizes[None, :, None]
    q = x.to(torch.bfloat16)
    k = q.flip(1).contiguous()
    w = 1 + 0.2 * torch.rand(d, generator=g, device=DEV)
    pos = torch.arange(7, dtype=torch.int32, device=DEV) * 1000 if R else None
    freqs = rope_frequencies(R) if R else []
    attn = DecodeAttention(nh, nkv, d, rope_freqs=freqs or None, interleaved=inter)
    qo, ko = attn.norm_rope(q, k, pos, w, w, eps=eps)
    e = float(np.float32(eps))
    for got, x in ((qo, q), (ko, k)):
        want, tol = _want_rows(x, w, pos, freqs, inter, e)
        close(got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -134 + tol)
    cache = make_cache(7, 1, nkv, d, "bf16", fill=0.0)
    assert torch.equal(attn.append(q, k, k, pos, torch.arange(7, device=DEV), cache, w, w, eps=eps), qo)
    assert torch.equal(cache.k[:, :, 0], ko) and torch.equal(cache.v[:, :, 0], k)
    # without a weight nothing is scaled; an infinity makes its row zeros and a NaN
    plain = DecodeAttention(nh, nkv, d)
    assert all(torch.equal(a, b) for a, b in zip(plain.norm_rope(q, k, None), (q, k)))
    q[3, 2, 5], q[4, 0, 7], q[5, 1] = float("inf"), float("-inf"), 0.0
    zero = torch.zeros((), dtype=torch.bfloat16, device=DEV)
    qi, ki = plain.norm_rope(q, k, None, w, w, eps=eps)
    for t, h, i in ((3, 2, 5), (4, 0, 7)):
        bad = torch.zeros(d, dtype=torch.bool, device=DEV)
        bad[i] = True
        assert torch.equal(torch.isnan(qi[t, h]), bad) and (qi[t, h][~bad] == zero).all()
    assert (torch.isnan(qi[5, 1]) if eps == 0 else qi[5, 1] == zero).all() and torch.isfinite(ki).all()


def test_errors_right_after_a_status_are_kept():
    """The flag is cleared before moe_attn_status returns: an error on a stream
    that does not wait for the default one, right after it, is reported."""
    attn = DecodeAttention(2, 1, 64)
    cache = make_cache(2, 8, 1, 64, "bf16", fill=1.0)
    x, bad = randn(gen(1), 1, 1, 64), torch.tensor([16], device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert attn.status() == 0
    for _ in range(200):
        attn.write(cache, x, x, bad, stream=side)
        assert attn.status() == C["MOE_ERR_DEVICE"]
    assert attn.status() == 0 and (cache.k == 1).all()


# Page tables so wide that every call of few sequences is cut as a list.
WIDE = 1 << 21


def cut_as_a_list(b, attn):
    """b's calls on attn are cut as a list of tiles."""
    return attn.decode_clusters(b.cache, len(b.lens), b.width) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d,sms", [(5, 1, 64, 14), (8, 1, 128, 20), (3, 1, 256, 20), (16, 1, 64, 40), (12, 1, 128, 40),
                                          (4, 2, 64, 28)])
@pytest.mark.parametrize("lens", [[20000], [50000, 20, 0, 4000, 1]])
def test_decode_list_joins_many_groups_of_parts(lens, nh, nkv, d, sms, fmt):
    """A list whose longest segment spans some 40 CTAs: parts are joined in groups
    of 16, then three groups.  Pieces of less than four tiles per warp, and, in the
    longer list, of more, where segments count for more than their tiles.  The
    oracle's result, to the same bits every time."""
    b = Batch(lens, nh, nkv, d, fmt, 64, seed=nh + d + len(lens), width=WIDE // 64)
    attn = DecodeAttention(nh, nkv, d, max_sms=sms)
    assert cut_as_a_list(b, attn)
    one = b.check(attn)
    for _ in range(2):
        again = b.run(attn)
        assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])
    b.check(attn, softcap=25.0, window=19000)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[150001], [150001, 20000, 0, 90000, 7]])
def test_decode_list_over_the_device(lens, fmt):
    """The list on all SMs, segments of hundreds of CTAs."""
    b = Batch(lens, 2, 1, 64, fmt, 128, seed=len(lens), width=WIDE // 128)
    attn = DecodeAttention(2, 1, 64)
    assert cut_as_a_list(b, attn)
    one = b.check(attn)
    again = b.run(attn)
    assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nh,nkv,d", [(8, 2, 64), (12, 12, 128), (16, 1, 128), (5, 1, 256), (40, 2, 64), (18, 1, 256)])
def test_decode_lists_of_small_calls(nh, nkv, d, fmt):
    """Few short sequences with page tables that could hold far longer ones: the
    list; with tables that only just cover them, clusters."""
    attn = DecodeAttention(nh, nkv, d)
    for lens in ([1, 1000], [500, 0, 33], [64], [2, 31, 32, 33]):
        b = Batch(lens, nh, nkv, d, fmt, 16, seed=nh + len(lens), width=WIDE // 16)
        assert cut_as_a_list(b, attn)
        one = b.check(attn, softcap=20.0)
        again = b.run(attn, softcap=20.0)
        assert torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])
        b.check(attn, starts=torch.tensor([5] * len(lens), dtype=torch.int32, device=DEV), window=300)
        b.table, b.width = b.table[:, :(max(lens) + 15) // 16], (max(lens) + 15) // 16
        assert not cut_as_a_list(b, attn)
        b.check(attn, softcap=20.0)


def test_decode_clusters_tells_the_way():
    attn = DecodeAttention(32, 8, 128)
    cache = PagedKVCache.empty(4, 16, 8, 128, "bf16")
    assert attn.decode_clusters(cache, 0, 10) == 0 and attn.decode_clusters(cache, 1, 64) == 1
    assert attn.decode_clusters(cache, 1, 1000) > 1 and attn.decode_clusters(cache, 512, 1000) == 0
    with pytest.raises(Exception, match="moe_attn_decode_clusters"):
        attn.decode_clusters(cache, 1, 0)
    with pytest.raises(ValueError):
        attn.decode_clusters(PagedKVCache.empty(4, 16, 4, 128, "bf16"), 1, 64)
    attn.close()
    with pytest.raises(ValueError):
        attn.decode_clusters(cache, 1, 64)


def test_decode_of_an_empty_batch():
    attn = DecodeAttention(4, 2, 64)
    cache = PagedKVCache.empty(4, 16, 2, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    for width in (0, 3):
        table, lens = torch.empty(0, width, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
        out, lse = attn.decode(q, cache, table, lens, lse=torch.empty(0, 4, device=DEV))
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert attn.status() == 0


def test_outputs_of_calls_on_the_default_streams_handle():
    """Handle 0, while another stream is the current one: outputs are of the
    default stream's memory."""
    attn = DecodeAttention(8, 2, 128)
    q, k = randn(gen(1), 64, 8, 128), randn(gen(2), 64, 2, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        old = torch.empty(64, 8, 128, dtype=torch.bfloat16, device=DEV)
        at = old.data_ptr()
        torch.cuda._sleep(2_000_000)
        old.fill_(1.0)
        del old
        out, _ = attn.norm_rope(q, k, None, stream=0)
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(out, q) and attn.status() == 0
