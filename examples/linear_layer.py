"""Trains a stack of a decayed linear attention layer and a selective layer on a delayed
copy for a few steps, then runs packed prompts and decodes from their states with 4-bit
weights.

    python examples/linear_layer.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from gated_deltanet_chunked_gdn_gb300.linear_layer import LinearLayer, Stack
from gated_deltanet_chunked_gdn_gb300.selective_layer import SelectiveLayer


def main(width=64, steps=100):
    torch.manual_seed(0)
    stack = Stack([LinearLayer(width, 1, 2, K=64, V=64), SelectiveLayer(width, 128, rank=32)], width)
    head = torch.nn.Parameter(torch.randn(width, width, device="cuda").bfloat16() * width ** -0.5)
    opt = torch.optim.Adam([*stack.parameters(), head], lr=1e-2)
    losses = []
    for _ in range(steps):
        u = torch.randn(8, 128, width, device="cuda").bfloat16()
        want = torch.roll(u, 2, dims=1).float()
        loss = ((stack(u) @ head).float() - want)[:, 2:].square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"delayed copy: loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    stack.quantize_()
    lens = [100, 7, 300]
    cu = torch.tensor([0, 100, 107, 407], dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    states = stack.new_states(6)
    u = torch.randn(1, sum(lens), width, device="cuda").bfloat16()
    stack.prompt(u, states, slots, cu)
    token = torch.randn(3, width, device="cuda").bfloat16()
    for _ in range(4):
        out = stack.step(token, states, slots)
    print(f"decoded 4 tokens of {len(lens)} sequences, |out| {out.float().norm():.2f}")
    return losses, out


if __name__ == "__main__":
    main()
