"""A multi-adapter serving loop in small: prompts, then single tokens, of one attention layer.

Each step builds its maps and pages on the GPU (``lora_batch_plan``), projects the rows to q, k and
v with every request's adapter added (``lora_delta_fused`` on the plan's ``seq_slot``), stores the new
keys and values in the 4-bit cache (``lora_kv4_append`` at the plan's ``slot_map``) and attends over it
(``lora_kv4_attention``).  A request that is done gives its pages back (``lora_pages_release``).

    python examples/serve_step.py
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lora_delta_gb300 as ld

HIDDEN, Q_HEADS, KV_HEADS, D, PAGE = 256, 8, 2, 64, 16
WIDTHS = (Q_HEADS * D, KV_HEADS * D, KV_HEADS * D)


class Server:
    """One layer's weights, adapters and cache, and the requests' lengths, pages and slots."""

    def __init__(self, req_slot, max_tokens: int, num_pages: int, seed: int = 0, dev="cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, device=dev, generator=g) * std).bfloat16()

        def ints(x):
            return torch.tensor(x, dtype=torch.int32, device=dev)

        self.weight = normal(HIDDEN, sum(WIDTHS), std=HIDDEN ** -0.5)
        self.pool = ld.LoraPool(HIDDEN, WIDTHS, max_loras=3, R=16, device=dev)
        for slot, rank in enumerate((16, 8, 4)):
            self.pool.pack(slot, [normal(rank, HIDDEN, std=HIDDEN ** -0.5) for _ in WIDTHS],
                           [normal(w, rank, std=rank ** -0.5) for w in WIDTHS], alpha=float(rank), rank=rank)
        self.cache = ld.Kv4Cache.empty(num_pages, PAGE, KV_HEADS, D, device=dev)
        B = len(req_slot)
        self.req_slot, self.ctx = ints(req_slot), ints([0] * B)
        self.table = torch.full((B, -(-max_tokens // PAGE)), -1, dtype=torch.int32, device=dev)
        self.free, self.free_count = torch.arange(num_pages, dtype=torch.int32, device=dev), ints([num_pages])
        self.err = ld.new_error_word(dev)

    def step(self, x, new_len, max_new: int):
        """The rows ``x`` [n, HIDDEN] of ``new_len`` [B] new tokens a request: the attention's output
        [n, Q_HEADS, D], the plan and the projections."""
        plan = ld.BatchPlan(len(self.ctx), len(x), PAGE, x.device)
        ld.lora_batch_plan(plan, self.ctx, new_len, self.table, req_slot=self.req_slot, free_pages=self.free,
                           free_count=self.free_count, err=self.err)
        qkv = x @ self.weight
        ld.lora_delta_fused(qkv, x, plan.seq_slot, self.pool, err=self.err)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split(WIDTHS, 1))
        ld.lora_kv4_append(self.cache, k, v, plan.slot_map, err=self.err)
        out = torch.empty(len(x), Q_HEADS, D, dtype=x.dtype, device=x.device)
        ld.lora_kv4_attention(out, q, self.cache, self.table, plan.row_start, plan.seq_len, max_new, err=self.err)
        self.ctx = plan.seq_len.clone()
        return out, plan, qkv

    def release(self, done):
        """The pages of the requests with ``done[b] != 0`` back to the free ones."""
        ld.lora_pages_release(done, self.ctx, self.table, PAGE, self.free, self.free_count, err=self.err)
        self.ctx = torch.where(done != 0, 0, self.ctx).int()


def main():
    dev, prompts = "cuda", [37, 5, 64, 1]
    server = Server(req_slot=[0, 2, -1, 1], max_tokens=128, num_pages=24, dev=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(sum(prompts), HIDDEN, device=dev, generator=g).bfloat16()
    out, plan, _ = server.step(x, torch.tensor(prompts, dtype=torch.int32, device=dev), max(prompts))
    print("prompts:", tuple(out.shape), "lengths", plan.seq_len.tolist(), "free pages", server.free_count.item())
    one = torch.ones(len(prompts), dtype=torch.int32, device=dev)
    for i in range(3):
        x = torch.randn(len(prompts), HIDDEN, device=dev, generator=g).bfloat16()
        out, plan, _ = server.step(x, one, 1)
        print(f"token {i}:", tuple(out.shape), "slots", plan.slot_map.tolist(), "adapters", plan.seq_slot.tolist())
    server.release(torch.tensor([1, 0, 1, 0], dtype=torch.int32, device=dev))
    print("released: free pages", server.free_count.item(), "errors", ld.lora_get_error(server.err))


if __name__ == "__main__":
    main()
