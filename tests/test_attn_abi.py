"""Host-side refusals of the paged attention's C ABI, and the Python layer's:
every one is decided before any CUDA call, so no GPU is needed.

The calls need a context, which only a GPU can give.  What the checks read of
it is its configuration, the first member; a zeroed block that starts with one
stands in for it, and no call below gets past its checks.
"""
import ctypes
import math

import pytest

import __graft_entry__ as entry
import fp8_routed_expert_gb300 as moe
from fp8_routed_expert_gb300._lib import AttnConfig, PagedKVDesc

ARG, SHAPE, ALIGN = (moe.C["MOE_ERR_" + n] for n in ("ARG", "SHAPE", "ALIGN"))
NH, NKV, D, R = 8, 2, 128, 64
P = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def L():
    entry.build()
    return moe.lib()


def _config(freqs=None, **kw):
    freqs = [0.5] * (R // 2) if freqs is None else freqs
    arr = (ctypes.c_double * max(1, len(freqs)))(*freqs)
    cfg = dict(n_heads=NH, n_kv_heads=NKV, head_dim=D, rope_dim=R, interleaved=0, max_sms=0, device=0,
               rope_freqs=ctypes.addressof(arr))
    cfg.update(kw)
    c = AttnConfig(**cfg)
    c.keep = arr
    return c


@pytest.fixture(scope="module")
def ctx():
    c = _config()
    block = ctypes.create_string_buffer(4096)
    ctypes.memmove(block, ctypes.byref(c), ctypes.sizeof(c))
    return block


def _kv(**kw):
    f = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=4, page_stride=NKV * 16 * D, head_stride=16 * D, slot_stride=D,
             scale_page_stride=NKV * 16, scale_head_stride=16, scale_slot_stride=1, page_size=16,
             format=moe.C["MOE_KV_E4M3"])
    f.update(kw)
    return PagedKVDesc(**f)


@pytest.mark.parametrize("kw,rc", [
    (dict(head_dim=96), SHAPE), (dict(n_heads=9), SHAPE), (dict(n_kv_heads=0), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(n_heads=2048, n_kv_heads=2), SHAPE), (dict(rope_dim=24), SHAPE), (dict(rope_dim=256), SHAPE),
    (dict(rope_dim=-16), SHAPE), (dict(max_sms=-1), SHAPE), (dict(device=-1), SHAPE), (dict(interleaved=2), ARG),
    (dict(rope_freqs=None), ARG), (dict(freqs=[math.nan] * 32), ARG), (dict(freqs=[math.inf] * 32), ARG)])
def test_bad_configs(L, kw, rc):
    h = ctypes.c_void_p(77)
    assert L.moe_attn_init(ctypes.byref(h), ctypes.byref(_config(**kw))) == rc
    assert h.value is None


def test_nulls(L, ctx):
    h = ctypes.c_void_p(77)
    assert L.moe_attn_init(None, None) == ARG and L.moe_attn_init(ctypes.byref(h), None) == ARG and h.value is None
    L.moe_attn_free(None)
    assert L.moe_attn_status(None) == ARG
    kv = _kv()
    assert L.moe_attn_norm_rope(None, P, 1024, P, 256, P, 1, None, None, 0.0, P, 1024, P, 256, None) == ARG
    assert L.moe_attn_append(ctx, None, P, 1024, P, 256, P, 256, P, P, 1, None, None, 0.0, P, 1024, None) == ARG
    assert L.moe_attn_write(None, ctypes.addressof(kv), P, 256, P, 256, P, 1, None) == ARG
    assert L.moe_attn_read(ctx, None, P, 1, P, 256, P, 256, None) == ARG
    assert L.moe_attn_decode(None, ctypes.addressof(kv), P, 1024, P, 4, 4, P, None, 1, 1.0, 0.0, None, 0, P, None,
                             None) == ARG


def _norm(L, ctx, **kw):
    a = dict(q=P, qs=NH * D, k=P, ks=NKV * D, pos=P, T=3, wq=P, wk=P, eps=1e-6, qo=P, qos=NH * D, ko=P, kos=NKV * D)
    a.update(kw)
    return L.moe_attn_norm_rope(ctx, *a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(T=1 << 31), SHAPE), (dict(q=None), ARG), (dict(ko=None), ARG), (dict(pos=None), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(eps=math.inf), ARG), (dict(qs=NH * D - 8), SHAPE),
    (dict(kos=0), SHAPE), (dict(ks=-NKV * D), SHAPE), (dict(qs=NH * D + 4), ALIGN), (dict(q=P + 8), ALIGN),
    (dict(qo=P + 2), ALIGN), (dict(wq=P + 4), ALIGN), (dict(pos=P + 2), ALIGN), (dict(qs=1 << 40), SHAPE)])
def test_norm_rope_refusals(L, ctx, kw, rc):
    assert _norm(L, ctx, **kw) == rc


def test_no_tokens_is_no_work(L, ctx):
    assert _norm(L, ctx, T=0, q=None) == 0
    desc = _kv()
    kv = ctypes.addressof(desc)
    assert L.moe_attn_write(ctx, kv, None, 0, None, 0, None, 0, None) == 0
    assert L.moe_attn_read(ctx, kv, None, 0, None, 0, None, 0, None) == 0
    assert L.moe_attn_decode(ctx, kv, None, 0, None, 0, 1, None, None, 0, 1.0, 0.0, None, 0, None, None, None) == 0


@pytest.mark.parametrize("kw,rc", [
    (dict(format=7), ARG), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE), (dict(page_size=0), SHAPE),
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG), (dict(v_scale=None), ARG),
    (dict(k=P + 8), ALIGN), (dict(slot_stride=D + 8), ALIGN), (dict(head_stride=-16), SHAPE),
    (dict(scale_slot_stride=-1), SHAPE), (dict(v_scale=P + 2), ALIGN), (dict(page_stride=1 << 50), SHAPE),
    (dict(format=0, slot_stride=D + 4), ALIGN)])
def test_cache_refusals(L, ctx, kw, rc):
    kv = _kv(**kw)
    ref = ctypes.addressof(kv)
    assert L.moe_attn_write(ctx, ref, P, NKV * D, P, NKV * D, P, 1, None) == rc
    assert L.moe_attn_read(ctx, ref, P, 1, P, NKV * D, P, NKV * D, None) == rc
    assert L.moe_attn_append(ctx, ref, P, NH * D, P, NKV * D, P, NKV * D, P, P, 1, None, None, 0.0, P, NH * D,
                             None) == rc
    assert L.moe_attn_decode(ctx, ref, P, NH * D, P, 4, 4, P, None, 1, 1.0, 0.0, None, 0, P, None, None) == rc


def test_write_read_append_refusals(L, ctx):
    kv = _kv()
    ref = ctypes.addressof(kv)
    rows = (P, NKV * D)
    assert L.moe_attn_write(ctx, ref, *rows, *rows, None, 1, None) == ARG
    assert L.moe_attn_write(ctx, ref, *rows, *rows, P + 4, 1, None) == ALIGN
    assert L.moe_attn_write(ctx, ref, P, 8, *rows, P, 1, None) == SHAPE
    assert L.moe_attn_read(ctx, ref, None, 1, *rows, *rows, None) == ARG
    assert L.moe_attn_read(ctx, ref, P, 1, None, NKV * D, *rows, None) == ARG
    assert L.moe_attn_append(ctx, ref, P, NH * D, *rows, *rows, P, None, 1, None, None, 0.0, P, NH * D, None) == ARG
    assert L.moe_attn_append(ctx, ref, P, NH * D, *rows, None, NKV * D, P, P, 1, None, None, 0.0, P, NH * D,
                             None) == ARG


@pytest.mark.parametrize("kw,rc", [
    (dict(B=-1), ARG), (dict(B=(1 << 20) + 1), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 27), SHAPE),
    (dict(table_stride=-1), SHAPE), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG), (dict(softcap=-1.0), ARG),
    (dict(softcap=math.nan), ARG), (dict(window=-1), ARG), (dict(table=None), ARG), (dict(lens=None), ARG),
    (dict(out=None), ARG), (dict(q=None), ARG), (dict(lens=P + 2), ALIGN), (dict(starts=P + 1), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(lse=P + 2), ALIGN), (dict(slopes=P + 2), ALIGN), (dict(qs=8), SHAPE)])
def test_decode_refusals(L, ctx, kw, rc):
    a = dict(q=P, qs=NH * D, table=P, table_stride=4, max_pages=4, lens=P, starts=None, B=2, scale=1.0, softcap=0.0,
             slopes=None, window=0, out=P, lse=None)
    a.update(kw)
    kv = _kv()
    assert L.moe_attn_decode(ctx, ctypes.addressof(kv), *a.values(), None) == rc


def test_rope_frequencies():
    f = moe.rope_frequencies(64)
    assert len(f) == 32 and f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64))


def test_outputs_come_from_the_memory_of_the_calls_stream(monkeypatch):
    """An output that a call makes is allocated while its stream is the current
    one.  Streams, memory and the native calls are stand-ins."""
    import torch

    from fp8_routed_expert_gb300 import attention

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream = handle

    class Use:
        def __init__(self, stream):
            self.handle = stream.cuda_stream

        def __enter__(self):
            current.append(self.handle)

        def __exit__(self, *exc):
            current.pop()

    class Rows:
        shape = (3,)

    current, made, ran = [5], [], []
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(current[-1]))
    monkeypatch.setattr(attention, "_current_raw_stream", lambda index: current[-1])

    class Native:
        def __getattr__(self, name):
            return lambda *a: ran.append(a[-1]) or 0

    a = object.__new__(moe.DecodeAttention)
    a.n_heads, a.n_kv_heads, a.head_dim, a.device, a._index = NH, NKV, D, None, 0
    a._ctx, a._b, a._scale = (), Native(), 1.0
    cache = type("Cache", (), {"_native": ()})()
    x = Rows()
    calls = (lambda s: a.norm_rope(x, x, x, stream=s), lambda s: a.append(x, x, x, x, x, cache, stream=s),
             lambda s: a.read(cache, x, stream=s), lambda s: a.decode(x, cache, x, x, stream=s))
    for given, used in ((None, 5), (Stream(7), 7), (9, 9)):
        for call, outputs in zip(calls, (2, 1, 2, 1)):
            made.clear(), ran.clear()
            call(given)
            assert made == [used] * outputs and ran == [used] and current == [5]


def _refused_by_all(L, ctx, kv, T=1):
    ref = ctypes.addressof(kv)
    return {L.moe_attn_write(ctx, ref, P, NKV * D, P, NKV * D, P, T, None),
            L.moe_attn_read(ctx, ref, P, T, P, NKV * D, P, NKV * D, None),
            L.moe_attn_append(ctx, ref, P, NH * D, P, NKV * D, P, NKV * D, P, P, T, None, None, 0.0, P, NH * D, None),
            L.moe_attn_decode(ctx, ref, P, NH * D, P, 4, 4, P, None, T, 1.0, 0.0, None, 0, P, None, None)}


@pytest.mark.parametrize("fmt", ["BF16", "E4M3"])
def test_caches_whose_offsets_leave_the_address_range(L, ctx, fmt):
    """Strides that each are within bounds, but whose products with the numbers of
    pages, heads or slots are not; the largest that still fit are taken (no tokens:
    no work)."""
    row = dict(BF16=2, E4M3=1)[fmt]
    base = dict(format=moe.C["MOE_KV_" + fmt], n_pages=1, page_size=1, page_stride=0, head_stride=0, slot_stride=0,
                scale_page_stride=0, scale_head_stride=0, scale_slot_stride=0)
    top = (1 << 31) - 1
    for kw in (dict(n_pages=top, page_stride=1 << 40), dict(page_size=top, slot_stride=1 << 40),
               dict(n_pages=1 << 22, page_stride=1 << 40, page_size=1 << 22, slot_stride=1 << 40)):
        assert _refused_by_all(L, ctx, _kv(**{**base, **kw})) == {SHAPE}
    for kw in (dict(scale_page_stride=1 << 40, n_pages=top), dict(scale_slot_stride=1 << 40, page_size=top)):
        if fmt == "E4M3":
            assert _refused_by_all(L, ctx, _kv(**{**base, **kw})) == {SHAPE}
    # (2^31 - 2) pages of 2^31 bytes, less a row
    fits = _kv(**{**base, "n_pages": top, "page_stride": (1 << 31) // row})
    assert _refused_by_all(L, ctx, fits, T=0) == {0}
    assert L.moe_attn_decode(ctx, ctypes.addressof(_kv()), P, NH * D, P, 1 << 41, 4, P, None, 1, 1.0, 0.0, None, 0, P,
                             None, None) == SHAPE


def test_decode_clusters_refusals(L, ctx):
    desc = _kv()
    kv = ctypes.addressof(desc)
    assert L.moe_attn_decode_clusters(None, kv, 1, 4) == ARG and L.moe_attn_decode_clusters(ctx, None, 1, 4) == ARG
    assert L.moe_attn_decode_clusters(ctx, kv, -1, 4) == ARG and L.moe_attn_decode_clusters(ctx, kv, 0, 4) == 0
    for B, pages in (((1 << 20) + 1, 4), (1, 0), (1, 1 << 27)):
        assert L.moe_attn_decode_clusters(ctx, kv, B, pages) == SHAPE
    bad = _kv(slot_stride=D + 8)
    assert L.moe_attn_decode_clusters(ctx, ctypes.addressof(bad), 1, 4) == ALIGN


def test_no_sequences_need_no_page_table(L, ctx):
    """B = 0 is no work whatever the page table's width, none included."""
    desc = _kv()
    kv = ctypes.addressof(desc)
    for pages in (0, 1, 9):
        assert L.moe_attn_decode(ctx, kv, None, 0, None, 0, pages, None, None, 0, 1.0, 0.0, None, 0, None, None, None) == 0
        assert L.moe_attn_decode_clusters(ctx, kv, 0, pages) == 0
    assert L.moe_attn_decode(ctx, kv, None, 0, None, 0, -1, None, None, 0, 1.0, 0.0, None, 0, None, None, None) == SHAPE
