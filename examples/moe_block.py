#!/usr/bin/env python
"""A pre-norm MoE transformer block's feed-forward half, built from the
library's layers and trained for a few steps on a synthetic task:

    h      = layer_norm(x)                           bfloat16
    logits = linear(h, Wgate)                        float32 [T, E]
    ids, w = router(logits, k)                       sigmoid scores, balance bias
    y      = moe(h, W, ids, w)                       the routed experts, float32
    s      = linear(h, Wup, bup, "gelu")             the shared expert
    out    = linear(s, Wdown, residual = x + y)      float32

After every step the balance bias moves against each expert's load, as in
routing without an auxiliary loss.

    python examples/moe_block.py [--tokens 4096] [--hidden 2048] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import variable_size_expert_gb300 as mgg  # noqa: E402


class MoEBlock(torch.nn.Module):
    """out = x + moe(h) + shared(h), h = layer_norm(x); weights are kept in
    bfloat16, the norm's and biases in float32."""

    def __init__(self, hidden: int, shared: int, experts: int, k: int, groups: int = 1,
                 topk_groups: int = 1, device="cuda", generator=None):
        super().__init__()

        def weight(*shape):
            w = torch.randn(*shape, device=device, generator=generator) / shape[-1] ** 0.5
            return torch.nn.Parameter(w.bfloat16())

        self.k, self.groups, self.topk_groups = k, groups, topk_groups
        self.norm_w = torch.nn.Parameter(torch.ones(hidden, device=device))
        self.norm_b = torch.nn.Parameter(torch.zeros(hidden, device=device))
        self.gate = weight(experts, hidden)
        self.experts = weight(experts, hidden, hidden)
        self.up, self.up_b = weight(shared, hidden), torch.nn.Parameter(torch.zeros(shared, device=device))
        self.down = weight(hidden, shared)
        self.register_buffer("balance", torch.zeros(experts, device=device))
        # the word that every layer's kernels report errors in
        self.register_buffer("status", mgg.new_status(device), persistent=False)

    def forward(self, x: torch.Tensor):
        """x [T, hidden] float32 (the residual stream) -> (out, expert_ids)."""
        h = mgg.layer_norm(x, self.norm_w, self.norm_b, out_dtype=torch.bfloat16)
        logits = mgg.linear(h, self.gate, out_dtype=torch.float32, status=self.status)
        ids, w = mgg.router(logits, self.k, scoring="sigmoid", bias=self.balance, groups=self.groups,
                            topk_groups=self.topk_groups, status=self.status)
        y = mgg.moe(h, self.experts, ids, w, status=self.status)
        s = mgg.linear(h, self.up, self.up_b, "gelu", status=self.status)
        return mgg.linear(s, self.down, residual=x + y, out_dtype=torch.float32, status=self.status), ids

    @torch.no_grad()
    def rebalance(self, ids: torch.Tensor, rate: float = 1e-3) -> torch.Tensor:
        load = torch.bincount(ids.flatten(), minlength=self.balance.numel()).float()
        self.balance += rate * torch.sign(load.mean() - load)
        return load


def train(tokens=4096, hidden=2048, shared=2048, experts=8, k=2, steps=20, lr=0.02, seed=0, log=print):
    """Fits the block to a fixed random map of its input; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = MoEBlock(hidden, shared, experts, k, generator=g)
    x = torch.randn(tokens, hidden, device="cuda", generator=g)
    target = x + torch.tanh(x.roll(1, 1)) + 0.1 * torch.randn(tokens, hidden, device="cuda", generator=g)
    params = list(block.parameters())
    losses = []
    for step in range(steps):
        out, ids = block(x)
        loss = (out - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in params:      # normalised gradient steps: one rate fits every layer
                p.sub_((lr * p.float().norm() / (p.grad.float().norm() + 1e-6)
                        * p.grad.float()).to(p.dtype) if p.dim() > 1 else lr * p.grad)
                p.grad = None
        load = block.rebalance(ids)
        losses.append(loss.item())
        if error := mgg.read_status(block.status):
            raise RuntimeError(f"step {step}: the kernels report error bits {error:#x}")
        log(f"step {step:3d}  loss {losses[-1]:.4f}  load {int(load.min())}..{int(load.max())}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    train(tokens=a.tokens, hidden=a.hidden, shared=a.hidden, experts=a.experts, steps=a.steps)
