"""Projections around the attention and the MoE, in the experts' weight format:
the hidden states' norm with the residual's addition and an 8-bit output, and the
product of 8-bit rows with 8-bit weights (moe_proj_* of include/fp8moe.h, where each
call's arithmetic, layouts and errors are stated).  Every step runs in the library's
kernels.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import check, lib, torch_binding
from .attention import _current_raw_stream
from .layer import _memory_of, _stream_handle

BLOCK = 128  # columns (and rows of the weights) that share a scale


class Projection:
    """A context of one device (moe_proj_init); ``max_sms``: the SMs a call may fill,
    and the CTAs that it has at most, 0 for all.

    ``stream`` of a call is the torch stream, or its handle, that its kernels run on
    (None: the current one).  Outputs that are not given are allocated from that
    stream's memory.  Other tensors of the call, and its outputs where they are used
    elsewhere, are the caller's to order and to keep."""

    def __init__(self, device: int = 0, max_sms: int = 0):
        self.device, self._index = torch.device("cuda", device), device
        self._ctx = None  # what the binding takes, while the context is open
        self._b = torch_binding()
        h = ctypes.c_void_p()
        check(lib().moe_proj_init(ctypes.byref(h), device, max_sms), "moe_proj_init")
        self._h = h
        self._ctx = (h.value, device)

    def close(self) -> None:
        self._ctx = None
        if getattr(self, "_h", None) is not None and self._h.value:
            lib().moe_proj_free(self._h)
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
        return lib().moe_proj_status(self._h)

    def _stream(self, stream) -> int | None:
        if stream is None and _current_raw_stream is not None:
            return _current_raw_stream(self._index)
        return _stream_handle(stream)

    def _new(self, shape, dtype, stream) -> torch.Tensor:
        if stream is not None:
            with _memory_of(stream, self._index):
                return self._new(shape, dtype, None)
        return torch.empty(shape, dtype=dtype, device=self.device)

    def norm(self, x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
             eps: float = 1e-6, residual_out: torch.Tensor | None = None, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
        """RMS norm of x bf16 [T, H] (where a weight f32 [H] is given), or of
        bf16(x + residual), which goes to ``residual_out`` (None: residual itself is
        overwritten).  Returns bf16 [T, H]."""
        if out is None:
            out = self._new(x.shape, torch.bfloat16, stream)
        if residual_out is None:
            residual_out = residual
        rc = self._b.norm(self._ctx, x, residual, weight, eps, residual_out, out, None, None, self._stream(stream))
        if rc:
            check(rc, "moe_proj_norm")
        return out

    def norm_quant(self, x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, residual_out: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                   scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """``norm`` as e4m3 codes uint8 [T, H] with f32 scales [T, ceil(H / 128)], and in
        bf16 too if ``out`` is given.  Without a weight the rows are quantised as they
        are.  The scales may have any positive strides; new ones lie block by block,
        as ``matmul`` reads them fastest."""
        if codes is None:
            codes = self._new(x.shape, torch.uint8, stream)
        if scales is None:
            T, H = x.shape
            scales = self._new((-(-H // BLOCK), T), torch.float32, stream).t()
        if residual_out is None:
            residual_out = residual
        rc = self._b.norm(self._ctx, x, residual, weight, eps, residual_out, out, codes, scales, self._stream(stream))
        if rc:
            check(rc, "moe_proj_norm")
        return codes, scales

    def matmul(self, codes: torch.Tensor, scales: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
               out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Rows (e4m3 codes uint8 [M, K], scales f32 [M, ceil(K / 128)]) times weights
        (codes uint8 [N, K], scales f32 [ceil(N / 128), ceil(K / 128)]), transposed:
        bf16 [M, N].  Rows of codes and weights begin 16-byte aligned."""
        if out is None:
            M, N = codes.shape[0], w.shape[0]
            out = self._new((M, -(-N // 8) * 8), torch.bfloat16, stream)[:, :N]
        rc = self._b.matmul(self._ctx, codes, scales, w, w_scale, out, self._stream(stream))
        if rc:
            check(rc, "moe_proj_matmul")
        return out
