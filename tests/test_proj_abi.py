"""Host-side refusals of the prompts' attention and of the projections: every one is
decided before any CUDA call, so no GPU is needed.

The calls need a context, which only a GPU can give.  What the checks read of it is
its configuration, the first member; a zeroed block that starts with one stands in
for it, and no call below gets past its checks.
"""
import ctypes
import math

import pytest
import torch

import __graft_entry__ as entry
import fp8_routed_expert_gb300 as moe
from fp8_routed_expert_gb300 import projection
from fp8_routed_expert_gb300._lib import AttnConfig

ARG, SHAPE, ALIGN = (moe.C["MOE_ERR_" + n] for n in ("ARG", "SHAPE", "ALIGN"))
NH, NKV, D = 8, 2, 128
P = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def L():
    entry.build()
    return moe.lib()


@pytest.fixture(scope="module")
def ctx():
    c = AttnConfig(n_heads=NH, n_kv_heads=NKV, head_dim=D)
    block = ctypes.create_string_buffer(4096)
    ctypes.memmove(block, ctypes.byref(c), ctypes.sizeof(c))
    return block


@pytest.fixture(scope="module")
def pctx():
    return ctypes.create_string_buffer(4096)


def _prefill(L, ctx, **kw):
    a = dict(q=P, qs=NH * D, Tq=5, k=P, ks=NKV * D, v=P, vs=NKV * D, Tk=7, q_starts=P, k_starts=P, B=2, causal=1, scale=1.0, cap=0.0,
             slopes=P, window=0, out=P, outs=NH * D, lse=P)
    a.update(kw)
    return L.moe_attn_prefill(ctx, *a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(Tq=-1), ARG), (dict(Tk=-1), ARG), (dict(Tq=1 << 31), SHAPE), (dict(Tk=1 << 31), SHAPE), (dict(B=-1), ARG),
    (dict(B=(1 << 20) + 1), SHAPE), (dict(causal=2), ARG), (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG),
    (dict(cap=-1.0), ARG), (dict(cap=math.inf), ARG), (dict(window=-1), ARG), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(v=None), ARG), (dict(out=None), ARG), (dict(q_starts=None), ARG), (dict(k_starts=None), ARG), (dict(qs=NH * D - 8), SHAPE),
    (dict(ks=0), SHAPE), (dict(vs=-NKV * D), SHAPE), (dict(outs=NH * D + 4), ALIGN), (dict(q=P + 8), ALIGN), (dict(v=P + 2), ALIGN),
    (dict(q_starts=P + 2), ALIGN), (dict(slopes=P + 1), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ks=1 << 40), SHAPE)])
def test_prefill_refusals(L, ctx, kw, rc):
    assert _prefill(L, ctx, **kw) == rc
    assert L.moe_attn_prefill(None, *[0] * 11, 0, 0.0, 0.0, None, 0, None, 0, None, None) == ARG


def test_no_prompts_are_no_work(L, ctx):
    none = dict(q=None, k=None, v=None, out=None, q_starts=None, k_starts=None)
    assert _prefill(L, ctx, B=0, **none) == 0 and _prefill(L, ctx, Tq=0, **none) == 0


def test_proj_nulls(L, pctx):
    h = ctypes.c_void_p(77)
    assert L.moe_proj_init(None, 0, 0) == ARG
    for device, sms in ((-1, 0), (0, -1)):
        assert L.moe_proj_init(ctypes.byref(h), device, sms) == SHAPE and h.value is None
    L.moe_proj_free(None)
    assert L.moe_proj_status(None) == ARG


def _norm(L, pctx, **kw):
    a = dict(x=P, xs=256, r=P, rs=256, T=3, H=256, w=P, eps=1e-6, ro=P, ros=256, out=P, outs=256, codes=P, cs=256, scales=P, sr=1, sb=3)
    a.update(kw)
    return L.moe_proj_norm(pctx, *a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(T=-1), ARG), (dict(T=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=100), SHAPE), (dict(H=16392), SHAPE), (dict(H=-8), SHAPE),
    (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(x=None), ARG), (dict(r=None), ARG), (dict(ro=None), ARG),
    (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(r=None, ro=None, out=None, codes=None, scales=None), ARG),
    (dict(xs=248), SHAPE), (dict(outs=0), SHAPE), (dict(rs=-256), SHAPE), (dict(cs=128), SHAPE), (dict(xs=1 << 40), SHAPE),
    (dict(xs=260), ALIGN), (dict(ros=258), ALIGN), (dict(cs=260), ALIGN), (dict(x=P + 8), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(codes=P + 4), ALIGN), (dict(scales=P + 2), ALIGN), (dict(w=P + 4), ALIGN), (dict(sr=0), SHAPE), (dict(sb=-1), SHAPE)])
def test_norm_refusals(L, pctx, kw, rc):
    assert _norm(L, pctx, **kw) == rc
    assert L.moe_proj_norm(None, P, 256, None, 0, 1, 256, None, 0.0, None, 0, P, 256, None, 0, None, 0, 0, None) == ARG


def _matmul(L, pctx, **kw):
    a = dict(a=P, lda=256, sa=P, sr=1, sb=5, M=5, w=P, ldw=256, sw=P, N=40, K=256, out=P, outs=40)
    a.update(kw)
    return L.moe_proj_matmul(pctx, *a.values(), None)


@pytest.mark.parametrize("kw,rc", [
    (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=-1), ARG), (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE),
    (dict(K=(1 << 31) - 255), SHAPE), (dict(a=None), ARG), (dict(w=None), ARG), (dict(sa=None), ARG), (dict(sw=None), ARG),
    (dict(out=None), ARG), (dict(lda=240), SHAPE), (dict(ldw=0), SHAPE), (dict(outs=32), SHAPE), (dict(lda=264), ALIGN),
    (dict(ldw=257), ALIGN), (dict(outs=44), ALIGN), (dict(a=P + 8), ALIGN), (dict(w=P + 1), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(sa=P + 2), ALIGN), (dict(sw=P + 2), ALIGN), (dict(sr=0), SHAPE), (dict(sb=0), SHAPE)])
def test_matmul_refusals(L, pctx, kw, rc):
    assert _matmul(L, pctx, **kw) == rc
    assert L.moe_proj_matmul(None, P, 256, P, 1, 5, 5, P, 256, P, 40, 256, P, 40, None) == ARG


def test_nothing_to_project_is_no_work(L, pctx):
    assert _norm(L, pctx, T=0, x=None) == 0
    assert _matmul(L, pctx, M=0, a=None, out=None) == 0 and _matmul(L, pctx, N=0, w=None, out=None) == 0


def test_outputs_come_from_the_memory_of_the_calls_stream(monkeypatch):
    """Stand-ins for torch and the binding: what a call allocates and where it runs."""
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

    class Made:
        def t(self):
            return self

        def __getitem__(self, i):
            return self

    class Rows:
        shape = (3, 256)

    current, made, ran = [5], [], []
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(current[-1]) or Made())
    monkeypatch.setattr(projection, "_current_raw_stream", lambda index: current[-1])

    class Native:
        def __getattr__(self, name):
            return lambda *a: ran.append(a[-1]) or 0

    p = object.__new__(moe.Projection)
    p.device, p._index, p._ctx, p._b = None, 0, (), Native()
    x = Rows()
    calls = (lambda s: p.norm(x, stream=s), lambda s: p.norm_quant(x, stream=s), lambda s: p.matmul(x, x, x, x, stream=s))
    for given, used in ((None, 5), (Stream(7), 7), (9, 9)):
        for call, outputs in zip(calls, (1, 2, 1)):
            made.clear(), ran.clear()
            call(given)
            assert made == [used] * outputs and ran == [used] and current == [5]


def test_bits_of_the_prompts_weights(L, ctx):
    assert L.moe_attn_prefill_bits(None, 8) == ARG
    assert [L.moe_attn_prefill_bits(ctx, b) for b in (0, 7, 9, 32, -8)] == [SHAPE] * 5
