"""Attention over a paged key/value cache: the serving form of the attention
beside the MoE.  ``PagedKVCache`` describes the cache, ``DecodeAttention`` is
the context whose calls norm and rotate heads, write and read the cache, attend
to it and attend within whole prompts (moe_attn_* of include/fp8moe.h, where each
call's arithmetic, layouts and errors are stated).  Every step runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import C, AttnConfig, PagedKVDesc, check, lib, torch_binding
from .layer import _memory_of, _stream_handle

_BF16 = torch.bfloat16

# The current stream's handle of a device.  A small decode step is a few
# microseconds, and building a torch.cuda.Stream object for each call costs
# about three (on Grace); this query costs a tenth of one.  For the same reason
# the calls go through the native binding, which checks their tensors.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def rope_frequencies(rope_dim: int, theta: float = 10000.0) -> list[float]:
    """The usual frequencies theta^(-2i/R), i < R/2, in radians per position."""
    return [theta ** (-2.0 * i / rope_dim) for i in range(rope_dim // 2)]


class PagedKVCache:
    """Key/value pages in device memory: ``k`` and ``v`` of shape [n_pages,
    n_kv_heads, page_size, head_dim], bf16, or uint8 (e4m3 codes) with f32
    ``k_scale`` / ``v_scale`` [n_pages, n_kv_heads, page_size].  The tensors
    may be views with any strides whose rows are contiguous (a permuted
    layout, one layer of a larger allocation); ``v`` has ``k``'s strides."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if k.dim() != 4 or not k.is_cuda or k.dtype not in (_BF16, torch.uint8):
            raise ValueError("k must be a cuda bf16 or uint8 tensor [n_pages, n_kv_heads, page_size, head_dim]")
        if v.dtype != k.dtype or v.shape != k.shape or v.device != k.device or v.stride() != k.stride():
            raise ValueError("v must match k in type, shape, strides and device")
        if k.stride(3) != 1:
            raise ValueError("the rows of k and v must be contiguous")
        e4m3 = k.dtype == torch.uint8
        if e4m3:
            for s in (k_scale, v_scale):
                if s is None or s.dtype != torch.float32 or s.shape != k.shape[:3] or s.device != k.device:
                    raise ValueError(f"an e4m3 cache needs f32 scales {tuple(k.shape[:3])} on its device")
            if k_scale.stride() != v_scale.stride():
                raise ValueError("v_scale must have k_scale's strides")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.format = "e4m3" if e4m3 else "bf16"
        self.device = k.device
        ss = k_scale.stride() if e4m3 else (0, 0, 0)
        self._desc = PagedKVDesc(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
                                 v_scale.data_ptr() if e4m3 else None, self.n_pages, *k.stride()[:3], *ss,
                                 self.page_size, C["MOE_KV_E4M3"] if e4m3 else C["MOE_KV_BF16"])
        self._native = (ctypes.addressof(self._desc), self.n_kv_heads, self.head_dim, k.get_device())

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, format: str = "bf16",
              device: int = 0) -> "PagedKVCache":
        """A new cache, rows of one (page, head) next to each other.  Memory is
        not initialised: positions are attended to only once written."""
        if format not in ("bf16", "e4m3"):
            raise ValueError(f"format must be 'bf16' or 'e4m3', got {format!r}")
        dev = torch.device("cuda", device)
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        dt = _BF16 if format == "bf16" else torch.uint8
        kv = [torch.empty(shape, dtype=dt, device=dev) for _ in range(2)]
        sc = [torch.empty(shape[:3], dtype=torch.float32, device=dev) for _ in range(2)] if format == "e4m3" else []
        return cls(*kv, *sc)


class DecodeAttention:
    """A context for one head layout (moe_attn_init).  ``rope_freqs``: radians
    per position of each rotated pair (``rope_frequencies``), None for no
    rotation; its length is half the rotated elements of a head.  One context
    serves one stream at a time.  ``prefill_bits``: what the weights of ``prefill``
    keep for their product with the values, 8 bits, or 16 at 1.1 to 1.5 times the time.

    ``stream`` of a call is the torch stream, or its handle, that its kernels run
    on (None: the current one).  Outputs that are not given are allocated from
    that stream's memory.  Other tensors of the call, and its outputs where they
    are used elsewhere, are the caller's to order (``wait_stream``) and to keep
    (``record_stream``)."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, rope_freqs=None,
                 interleaved: bool = False, device: int = 0, max_sms: int = 0, prefill_bits: int = 8):
        freqs = [] if rope_freqs is None else [float(f) for f in rope_freqs]
        arr = (ctypes.c_double * max(len(freqs), 1))(*freqs)
        self.cfg = AttnConfig(n_heads, n_kv_heads, head_dim, 2 * len(freqs), int(interleaved), max_sms, device,
                              ctypes.addressof(arr) if freqs else None)
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.rope_dim = 2 * len(freqs)
        self.device, self._index = torch.device("cuda", device), device
        self._ctx = None  # what the binding takes, while the context is open
        self._b = torch_binding()
        self._scale = 1.0 / math.sqrt(head_dim) if head_dim > 0 else 0.0
        h = ctypes.c_void_p()
        check(lib().moe_attn_init(ctypes.byref(h), ctypes.byref(self.cfg)), "moe_attn_init")
        self.cfg.rope_freqs = None  # read during the call only
        self._h = h
        if prefill_bits != 8:
            check(lib().moe_attn_prefill_bits(h, prefill_bits), "moe_attn_prefill_bits")
        self._ctx = (h.value, n_heads, n_kv_heads, head_dim, self.rope_dim, device)

    def close(self) -> None:
        self._ctx = None
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().moe_attn_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def status(self) -> int:
        return lib().moe_attn_status(self._h)

    def _stream(self, stream) -> int | None:
        if stream is None and _current_raw_stream is not None:
            return _current_raw_stream(self._index)
        return _stream_handle(stream)

    def _new(self, T: int, heads: int, stream) -> torch.Tensor:
        if stream is not None:
            with _memory_of(stream, self._index):
                return self._new(T, heads, None)
        return torch.empty((T, heads, self.head_dim), dtype=_BF16, device=self.device)

    # -- operators -------------------------------------------------------

    def norm_rope(self, q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor | None,
                  q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                  eps: float = 1e-6, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                  stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """RMS norm (where a weight f32 [d] is given) and rotation of q bf16
        [T, n_heads, d] and k bf16 [T, n_kv_heads, d]; positions int32 [T].
        q_out / k_out may be q / k."""
        if q_out is None:
            q_out = self._new(q.shape[0], self.n_heads, stream)
        if k_out is None:
            k_out = self._new(k.shape[0], self.n_kv_heads, stream)
        rc = self._b.norm_rope(self._ctx, q, k, positions, q_weight, k_weight, eps, q_out, k_out,
                               self._stream(stream))
        if rc:
            check(rc, "moe_attn_norm_rope")
        return q_out, k_out

    def append(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
               slots: torch.Tensor, cache: PagedKVCache, q_weight: torch.Tensor | None = None,
               k_weight: torch.Tensor | None = None, eps: float = 1e-6, q_out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
        """norm_rope whose keys, and the values as they are, go into the
        cache's slots (int64 [T]: page * page_size + slot, negative to store
        nothing).  Returns the queries."""
        if q_out is None:
            q_out = self._new(q.shape[0], self.n_heads, stream)
        rc = self._b.append(self._ctx, cache._native, q, k, v, positions, slots, q_weight, k_weight, eps, q_out,
                            self._stream(stream))
        if rc:
            check(rc, "moe_attn_append")
        return q_out

    def write(self, cache: PagedKVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, stream=None) -> None:
        """k and v bf16 [T, n_kv_heads, d] into the cache's slots, quantised
        if it is e4m3."""
        rc = self._b.write(self._ctx, cache._native, k, v, slots, self._stream(stream))
        if rc:
            check(rc, "moe_attn_write")

    def read(self, cache: PagedKVCache, slots: torch.Tensor, k_out: torch.Tensor | None = None,
             v_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """The rows of the slots as bf16 [T, n_kv_heads, d] (zeros for a
        negative slot)."""
        if k_out is None:
            k_out = self._new(slots.shape[0], self.n_kv_heads, stream)
        if v_out is None:
            v_out = self._new(slots.shape[0], self.n_kv_heads, stream)
        rc = self._b.read(self._ctx, cache._native, slots, k_out, v_out, self._stream(stream))
        if rc:
            check(rc, "moe_attn_read")
        return k_out, v_out

    def decode(self, q: torch.Tensor, cache: PagedKVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
               scale: float | None = None, softcap: float = 0.0, slopes: torch.Tensor | None = None,
               window: int = 0, starts: torch.Tensor | None = None, out: torch.Tensor | None = None,
               lse: torch.Tensor | None = None, stream=None):
        """Attention of one new token per sequence: q bf16 [B, n_heads, d],
        page_table int32 [B, max_pages], seq_lens int32 [B] (the new token
        counted).  ``scale`` is 1/sqrt(d) by default; softcap > 0 caps the
        scores by a tanh, ``slopes`` f32 [n_heads] adds slope * (j - newest
        position), ``window`` > 0 and ``starts`` int32 [B] hide earlier
        positions.  Returns out bf16 [B, n_heads, d], or (out, lse) if ``lse``
        f32 [B, n_heads] is given."""
        if out is None:
            out = self._new(q.shape[0], self.n_heads, stream)
        rc = self._b.decode(self._ctx, cache._native, q, page_table, seq_lens, starts,
                            self._scale if scale is None else scale, softcap, slopes, window, out, lse,
                            self._stream(stream))
        if rc:
            check(rc, "moe_attn_decode")
        return out if lse is None else (out, lse)

    def prefill(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_starts: torch.Tensor,
                k_starts: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
                softcap: float = 0.0, slopes: torch.Tensor | None = None, window: int = 0,
                out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
        """Attention of prompts packed one after another: q bf16 [Tq, n_heads, d],
        k and v bf16 [Tk, n_kv_heads, d]; sequence b's rows begin at q_starts[b] and
        k_starts[b] (int32 [B + 1], the last one the end; k_starts None: q_starts).
        Its last query is its last key's token, so a chunk of a prompt comes with the
        keys and values before it (``read``).  Options as for ``decode``; without
        ``causal`` later keys are visible too.  Returns out bf16 [Tq, n_heads, d], or
        (out, lse) if ``lse`` f32 [Tq, n_heads] is given; rows outside the sequences
        are left as they are."""
        if out is None:
            out = self._new(q.shape[0], self.n_heads, stream)
        rc = self._b.prefill(self._ctx, q, k, v, q_starts, q_starts if k_starts is None else k_starts, causal,
                             self._scale if scale is None else scale, softcap, slopes, window, out, lse,
                             self._stream(stream))
        if rc:
            check(rc, "moe_attn_prefill")
        return out if lse is None else (out, lse)

    def decode_clusters(self, cache: PagedKVCache, batch: int, max_pages: int) -> int:
        """How ``decode`` splits a call of ``batch`` sequences with page tables of
        ``max_pages`` columns: clusters of CTAs per sequence and group of heads, or
        0 where all sequences' tiles are cut evenly over the device."""
        if self._ctx is None:
            raise ValueError("the context is closed")
        if (cache.n_kv_heads, cache.head_dim) != (self.n_kv_heads, self.head_dim):
            raise ValueError(f"the cache holds {cache.n_kv_heads} heads of {cache.head_dim}; "
                             f"the context has {self.n_kv_heads} of {self.head_dim}")
        n = lib().moe_attn_decode_clusters(self._h, ctypes.addressof(cache._desc), batch, max_pages)
        if n < 0:
            check(n, "moe_attn_decode_clusters")
        return n
