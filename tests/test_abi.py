"""The C-ABI library loads and behaves on the host side (no GPU needed).

No compute call is made: config validation, NULL handling and error strings
all run before any CUDA call.
"""
import ctypes

import pytest

import __graft_entry__ as entry
import fp8_routed_expert_gb300 as moe
from fp8_routed_expert_gb300._lib import MoEConfig


@pytest.fixture(scope="module")
def L():
    entry.build()
    return moe.lib()


def test_exports_every_declared_function(L):
    names = moe.exported_functions()
    assert {"moe_init", "moe_layer_forward", "moe_free", "moe_get_routing", "moe_status",
            "moe_strerror", "moe_layer_forward_host"} <= set(names)
    for n in names:
        assert hasattr(L, n), n


def _init(L, **kw):
    cfg = dict(max_tokens=8, hidden=256, n_experts=8, inter=128, max_top_k=2, device=0)
    cfg.update(kw)
    h = ctypes.c_void_p(1234)
    rc = L.moe_init(ctypes.byref(h), ctypes.byref(MoEConfig(**cfg)))
    return rc, h


@pytest.mark.parametrize("kw", [dict(hidden=200), dict(inter=100), dict(hidden=0),
                                dict(n_experts=0), dict(n_experts=2000), dict(max_top_k=0),
                                dict(max_top_k=9), dict(max_top_k=33, n_experts=64),
                                dict(max_tokens=0), dict(hidden=65536 + 128),
                                dict(max_tokens=1 << 40)])
def test_bad_configs_rejected_before_cuda(L, kw):
    rc, h = _init(L, **kw)
    assert rc == moe.C["MOE_ERR_SHAPE"]
    assert h.value is None  # *out cleared


def test_null_arguments(L):
    assert L.moe_init(None, None) == moe.C["MOE_ERR_ARG"]
    h = ctypes.c_void_p()
    assert L.moe_init(ctypes.byref(h), None) == moe.C["MOE_ERR_ARG"]
    L.moe_free(None)  # no-op
    assert L.moe_layer_forward(None, None, 0, None, None, None, None, None, None, 1, None,
                               None) == moe.C["MOE_ERR_ARG"]
    assert L.moe_status(None) == moe.C["MOE_ERR_ARG"]
    assert L.moe_set_path(None, 0) == moe.C["MOE_ERR_ARG"]
    assert L.moe_resolve_path(None, 1) == moe.C["MOE_ERR_ARG"]
    assert L.moe_selftest_wait_timeout(None, 1000, None, None) == moe.C["MOE_ERR_ARG"]
    assert L.moe_cache_init(None, None, None, None, 1) == moe.C["MOE_ERR_ARG"]
    h = ctypes.c_void_p(99)
    assert L.moe_cache_init(ctypes.byref(h), None, None, None, 1) == moe.C["MOE_ERR_ARG"]
    assert h.value is None
    assert L.moe_cache_forward(None, None, 1, None, None, None, None, 1, None, None) == moe.C["MOE_ERR_ARG"]
    assert L.moe_cache_prefetch(None, None, 0) == moe.C["MOE_ERR_ARG"]
    assert L.moe_cache_stats(None, None, 0) == moe.C["MOE_ERR_ARG"]
    L.moe_cache_free(None)


def test_error_strings(L):
    for name, code in moe.C.items():
        if name.startswith("MOE_ERR_") or name == "MOE_OK":
            s = L.moe_strerror(code).decode()
            assert s and s != "unknown error", name
    assert L.moe_strerror(12345).decode() == "unknown error"
    for k in range(moe.C["MOE_K_COUNT"]):
        assert L.moe_kernel_name(k).decode() != "unknown"


def test_init_without_gpu_reports_cuda_error(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    rc, h = _init(L)
    assert rc in (moe.C["MOE_ERR_CUDA"], moe.C["MOE_ERR_UNSUPPORTED"])
    assert h.value is None


def test_outputs_come_from_the_memory_of_the_calls_stream(monkeypatch):
    """An output that a call makes is allocated while its stream is the current
    one.  Streams, memory, tensors and the library are stand-ins."""
    import torch

    from fp8_routed_expert_gb300 import layer

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

    class Tensor:
        is_cuda = True

        def __init__(self, dtype, *shape):
            self.dtype, self.shape = dtype, shape

        def dim(self):
            return len(self.shape)

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return 0

        def numel(self):
            return 0

        def element_size(self):
            return 0

    class Library:
        def __getattr__(self, name):
            return lambda *a: ran.append(a[-1]) or 0

    def make(*a, **k):
        made.append(current[-1])
        return Tensor(None)

    current, made, ran = [5], [], []
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(current[-1]))
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(torch, "empty_like", make)
    monkeypatch.setattr(layer, "lib", Library)
    H, E, I = 256, 8, 128
    u8, f32 = torch.uint8, torch.float32
    m = object.__new__(moe.MoELayer)
    m.cfg, m.device, m._h = MoEConfig(8, H, E, I, 2, 0), 0, None
    c = object.__new__(moe.ExpertCache)
    c.layer, c._h = m, None
    x, rw = Tensor(torch.bfloat16, 3, H), Tensor(f32, E, H)
    fp8 = (Tensor(u8, E, 2 * I, H), Tensor(f32, E, 2 * I // 128, H // 128), Tensor(u8, E, H, I),
           Tensor(f32, E, H // 128, I // 128))
    fp4 = (Tensor(u8, E, 2 * I, H // 2), Tensor(u8, E, 2 * I, H // 16), Tensor(f32, E), Tensor(u8, E, H, I // 2),
           Tensor(u8, E, H, I // 16), Tensor(f32, E))
    calls = ((lambda s: m.forward(x, rw, None, *fp8, 2, stream=s), 1),
             (lambda s: m.forward_nvfp4(x, rw, None, *fp4, 2, stream=s), 1),
             (lambda s: m.routing(3, 2, stream=s), 6), (lambda s: m.debug_buffer("h", f32, 1, stream=s), 1),
             (lambda s: c.forward(x, rw, None, fp8[1], fp8[3], 2, stream=s), 1))
    for given, used in ((None, 5), (Stream(7), 7), (9, 9)):
        for call, outputs in calls:
            made.clear(), ran.clear()
            call(given)
            assert made == [used] * outputs and ran == [used] and current == [5]


def test_handle_zero_is_the_default_stream(monkeypatch):
    """The memory of a call on handle 0 is the default stream's."""
    import torch

    from fp8_routed_expert_gb300.layer import _memory_of
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: ("external", handle, device.index))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device.index))
    assert _memory_of(0, 3) == ("default", 3) and _memory_of(7, 2) == ("external", 7, 2)
