"""A layer of routed experts with adapters, in small: the experts' base products and the LoRA deltas around them.

The tokens are sorted by expert (``lora_moe_dispatch``); the first product takes the gate and up delta of each row's adapter
ahead of its activation (``lora_moe_fc1_delta`` on the sorted rows, then ``lora_moe_linear``); the second is followed by the
down delta in place (``lora_moe_w2_delta``); ``lora_moe_combine`` weighs the rows and adds them to the residual.

    python examples/moe_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lora_delta_gb300 as ld


class MoeLayer:
    """E experts of inner width I, ``L`` adapters of rank ``rank``; bfloat16 as the deltas are."""

    def __init__(self, H=256, I=128, E=8, top_k=2, L=3, rank=16, scale=2.0, seed=0, dev="cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, device=dev, generator=g) * std).bfloat16()

        self.H, self.I, self.E, self.top_k, self.L, self.rank, self.scale = H, I, E, top_k, L, rank, scale
        self.router = torch.randn(H, E, device=dev, generator=g) * H ** -0.5
        self.w13, self.w2 = normal(E, 2 * I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5)
        # banks [E, L, rank, in] and [E, L, out, rank], and the tables of the experts' addresses
        self.a13 = [normal(E, L, rank, H, std=H ** -0.5) for _ in range(2)]
        self.b13 = [normal(E, L, I, rank, std=rank ** -0.5) for _ in range(2)]
        self.a2, self.b2 = normal(E, L, rank, I, std=I ** -0.5), normal(E, L, H, rank, std=rank ** -0.5)

        def table(*banks):
            return torch.tensor([[b[e].data_ptr() for e in range(E)] for b in banks], dtype=torch.int64, device=dev)

        self.ptr = table(*self.a13), table(*self.b13), table(self.a2)[0].contiguous(), table(self.b2)[0].contiguous()
        self.err = ld.new_error_word(dev)

    def route(self, x):
        """Weights [T, top_k] and experts of the tokens."""
        top, ids = torch.topk(x.float() @ self.router, self.top_k, dim=1)
        return torch.softmax(top, 1).contiguous(), ids.int().contiguous()

    def forward(self, x, weights, ids, lora):
        """x [T, H] and its experts' part; ``lora`` [T] int32 names each token's adapter, -1 for none."""
        T, P, dev = len(x), len(x) * self.top_k, x.device
        H, I, E, R, err = self.H, self.I, self.E, self.rank, self.err
        plan = ld.MoePlan(T, self.top_k, E, dev)
        rows, y = (torch.empty(P, H, dtype=x.dtype, device=dev) for _ in range(2))
        delta, act = torch.empty(P, 1, 2 * I, dtype=x.dtype, device=dev), torch.empty(P, I, dtype=x.dtype, device=dev)
        ld.lora_moe_dispatch(rows, x, ids, plan, lora_ids=lora, err=err)
        experts, (a13, b13, a2, b2) = plan.row_expert.view(P, 1), self.ptr
        ld.lora_moe_fc1_delta(delta, rows, a13, R * H, b13, I * R, False, experts, plan.row_lora, E, I, R, self.L, self.scale, err=err)
        ld.lora_moe_linear(act, rows, self.w13, plan, delta=delta.view(P, 2 * I), activation="silu", gated=True, err=err)
        ld.lora_moe_linear(y, act, self.w2, plan, err=err)
        ld.lora_moe_w2_delta(y.view(P, 1, H), act, a2, R * I, b2, H * R, experts, plan.row_lora, E, H, R, self.L, self.scale, err=err)
        out = torch.empty_like(x)
        ld.lora_moe_combine(out, y, plan, weights=weights, residual=x)
        return out, plan


def main():
    layer = MoeLayer()
    g = torch.Generator(device="cuda").manual_seed(1)
    for T in (64, 1):
        x = torch.randn(T, layer.H, device="cuda", generator=g).bfloat16()
        lora = torch.randint(-1, layer.L, (T,), dtype=torch.int32, device="cuda", generator=g)
        out, plan = layer.forward(x, *layer.route(x), lora)
        print(f"{T} tokens:", tuple(out.shape), "rows of the experts", plan.seg_start.diff().tolist(), "errors",
              ld.lora_get_error(layer.err))


if __name__ == "__main__":
    main()
