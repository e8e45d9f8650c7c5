"""The layers together (examples/moe_block.py): the block's forward and every
parameter's gradient against float64 autograd of the same block, and a few
training steps."""
import os
import sys

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block
    return moe_block


def test_block_against_float64():
    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, F, E, k = 150, 128, 96, 8, 2
    block = ex.MoEBlock(H, F, E, k, groups=4, topk_groups=2, generator=g)
    block.balance.copy_(0.05 * torch.randn(E, device="cuda", generator=g))
    x = torch.randn(T, H, device="cuda", generator=g).requires_grad_()
    out, ids = block(x)
    dy = torch.randn(T, H, device="cuda", generator=g)
    (out * dy).sum().backward()

    # the same block in float64 on the CPU, the experts chosen held fixed;
    # h is rounded to bfloat16 as the block's own activations are
    p = {n: R.d(v).requires_grad_() for n, v in block.named_parameters()}
    xd = R.d(x).requires_grad_()
    h, _, _ = R.norm_forward(xd, p["norm_w"], p["norm_b"], 1e-5)
    h = h + (h.detach().float().bfloat16().double() - h.detach())
    i = ids.cpu().long()
    w = R.weights_of(h @ p["gate"].t(), i, torch.ones(T, k, dtype=torch.bool), "sigmoid", True, 1.0)
    per = torch.einsum("tk,enk->ten", h, p["experts"])
    y = (per.gather(1, i[:, :, None].expand(T, k, H)) * w[:, :, None]).sum(1)
    s = R.act(h @ p["up"].t() + p["up_b"], "gelu")
    ref = xd + y + s @ p["down"].t()
    (ref * R.d(dy)).sum().backward()
    # bfloat16 activations and gradients between the layers: at most five
    # roundings of root mean square 1.7e-3 each meet in one value
    for name, got, want in [("out", out, ref)] + [("x", x.grad, xd.grad)] + [
            (n, v.grad, p[n].grad) for n, v in block.named_parameters()]:
        err = float((R.d(got) - want.detach()).norm() / want.detach().norm())
        assert err <= 9e-3, (name, err)


def test_training_lowers_the_loss():
    ex = _example()
    losses = ex.train(tokens=512, hidden=256, shared=256, experts=8, steps=15, log=lambda s: None)
    assert losses[-1] < 0.8 * losses[0], losses
    again = ex.train(tokens=512, hidden=256, shared=256, experts=8, steps=1, log=lambda s: None)
    assert abs(again[0] - losses[0]) <= 1e-5 * losses[0]
