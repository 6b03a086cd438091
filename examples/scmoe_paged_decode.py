"""Decode steps of a shortcut-connected MoE block over a paged cache.

Per step, for every sequence's new token: the query, key and value heads are
projected (a plain matrix product), normed and rotated, the key and value rows
put into the sequence's page (``DecodeAttention.append``), and the new token
attends to its sequence's pages (``DecodeAttention.decode``).  The routed MoE
of the same hidden state runs beside it on another stream, and its output is
added at the end of the block.

    python examples/scmoe_paged_decode.py --batch 8 --prompt 1000 --steps 32 --cache e4m3
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from fp8_routed_expert_gb300 import DecodeAttention, MoELayer, PagedKVCache, rope_frequencies  # noqa: E402

PAGE = 32


class Block:
    """One block: attention weights, MoE weights, and a paged cache that grows
    with its sequences."""

    def __init__(self, batch: int, max_len: int, cache: str = "e4m3", hidden: int = 2048, n_heads: int = 16,
                 n_kv_heads: int = 16, n_experts: int = 64, inter: int = 1024, top_k: int = 8, seed: int = 0):
        dev = torch.device("cuda", 0)
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        d = 128
        self.batch, self.hidden, self.n_heads, self.n_kv, self.d, self.top_k = batch, hidden, n_heads, n_kv_heads, d, top_k
        randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        bf16 = lambda t: t.to(torch.bfloat16)  # noqa: E731
        self.w_qkv = bf16(randn((n_heads + 2 * n_kv_heads) * d, hidden) * hidden ** -0.5)
        self.w_out = bf16(randn(hidden, n_heads * d) * (n_heads * d) ** -0.5)
        self.q_norm, self.k_norm = torch.ones(d, device=dev), torch.ones(d, device=dev)
        # experts: e4m3 codes of N(0, 1) values with one scale per 128 x 128 block
        codes = lambda *s: randn(*s).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        self.moe_args = (randn(n_experts, hidden) * 0.02, None, codes(n_experts, 2 * inter, hidden),
                         torch.full((n_experts, 2 * inter // 128, hidden // 128), 0.02, device=dev),
                         codes(n_experts, hidden, inter),
                         torch.full((n_experts, hidden // 128, inter // 128), 0.02, device=dev))
        self.moe = MoELayer(batch, hidden, n_experts, inter, top_k)
        self.attn = DecodeAttention(n_heads, n_kv_heads, d, rope_freqs=rope_frequencies(d))
        # sequence b's pages, in an order of their own
        width = -(-max_len // PAGE)
        self.cache = PagedKVCache.empty(batch * width, PAGE, n_kv_heads, d, cache)
        order = torch.randperm(batch * width, generator=g, device=dev)
        self.table = order.to(torch.int32).view(batch, width).contiguous()
        self.pos = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.moe_stream = torch.cuda.Stream()

    def slots(self, pos: torch.Tensor) -> torch.Tensor:
        """Where each sequence's row of position pos lies."""
        page = self.table.gather(1, (pos // PAGE).long()[:, None])[:, 0].long()
        return page * PAGE + pos % PAGE

    def prompt(self, lengths: torch.Tensor, seed: int = 1) -> None:
        """Fills the caches with prompts of the given lengths (int64 [batch], on
        the host): their normed and rotated keys, and values."""
        g = torch.Generator(device=self.table.device)
        g.manual_seed(seed)
        for b, n in enumerate(lengths.tolist()):
            if n == 0:
                continue
            x = torch.randn(n, self.hidden, generator=g, device=self.table.device).to(torch.bfloat16)
            qkv = (x @ self.w_qkv.T).view(n, -1, self.d)
            j = torch.arange(n, dtype=torch.int32, device=self.table.device)
            slots = self.table[b].long()[(j // PAGE).long()] * PAGE + j % PAGE
            self.attn.append(*self._heads(qkv), j, slots, self.cache, self.q_norm, self.k_norm)
        self.pos.copy_(lengths.to(torch.int32))

    def _heads(self, qkv: torch.Tensor):
        a, b = self.n_heads, self.n_heads + self.n_kv
        return qkv[:, :a], qkv[:, a:b], qkv[:, b:]

    def step(self, x: torch.Tensor, overlap: bool = True) -> torch.Tensor:
        """x bf16 [batch, hidden], the hidden states of the sequences' newest
        tokens; returns the block's output."""
        main = torch.cuda.current_stream()
        side = self.moe_stream if overlap else main
        side.wait_stream(main)
        with torch.cuda.stream(side):
            y = self.moe.forward(x, *self.moe_args, self.top_k)
        qkv = (x @ self.w_qkv.T).view(self.batch, -1, self.d)
        q = self.attn.append(*self._heads(qkv), self.pos, self.slots(self.pos), self.cache, self.q_norm, self.k_norm)
        self.pos += 1
        o = self.attn.decode(q, self.cache, self.table, self.pos)
        o = o.view(self.batch, -1) @ self.w_out.T
        main.wait_stream(side)
        x.record_stream(side)
        y.record_stream(main)
        return x + o + y


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt; the others are shorter")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="e4m3")
    ap.add_argument("--serial", action="store_true", help="MoE and attention on one stream")
    a = ap.parse_args()
    block = Block(a.batch, a.prompt + a.steps + 8, a.cache)
    block.prompt(torch.tensor([max(1, a.prompt * (b + 1) // a.batch) for b in range(a.batch)]))
    x = torch.randn(a.batch, block.hidden, device="cuda").to(torch.bfloat16)
    for _ in range(4):
        block.step(x, not a.serial)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        y = block.step(x, not a.serial)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    assert block.attn.status() == 0 and block.moe.status() == 0 and torch.isfinite(y).all()
    print(f"{a.batch} sequences of up to {a.prompt} tokens, {a.cache} cache: {t * 1e6:.0f} us a step, "
          f"{a.batch / t:.0f} tokens/s through the block")


if __name__ == "__main__":
    main()
