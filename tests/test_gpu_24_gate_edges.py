"""The expert choice where its arithmetic is at its ends."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("E", [16, 200, 600])
@pytest.mark.parametrize("renorm", [False, True])
def test_sigmoid_gradient_of_sure_choices(dtype, E, renorm):
    """Logits from -60 to 60: the slope p (1 - p) keeps its relative accuracy on
    both sides, where 1 - p is far below p's last bit.

    1 + exp(l), the division and the products round by U each, exp is within
    2 ulp (4 U): 16 U of w (1 - p) |g - dot|, and of the terms of dot."""
    T, k, scale = 61, 4, 2.5
    g = torch.Generator(device=DEV).manual_seed(E)
    logits = (torch.rand(T, E, generator=g, device=DEV) * 120 - 60).to(dtype)
    logits[0] = torch.linspace(10, 40, E, device=DEV).to(dtype)     # every choice is sure
    ids, w = mgg.select_experts(logits, k, "sigmoid", renormalize=renorm, scale=scale)
    dw = torch.randn(T, k, generator=g, device=DEV)
    st = mgg.new_status(DEV)
    got = mgg.select_experts_backward(dw, logits, ids, w, "sigmoid", renorm, scale, status=st)
    assert mgg.read_status(st) == 0
    l, i, wd, gd = R.d(logits), ids.cpu().long(), R.d(w), R.d(dw)
    dot = (gd * wd).sum(1, keepdim=True) / scale if renorm else torch.zeros(T, 1).double()
    mag = (gd * wd).abs().sum(1, keepdim=True) / scale if renorm else torch.zeros(T, 1).double()
    slope = wd * torch.sigmoid(-l.gather(1, i))
    ref = torch.zeros(T, E).double().scatter_(1, i, slope * (gd - dot))
    tol = torch.zeros(T, E).double().scatter_(1, i, 16 * R.U * slope * (gd.abs() + mag))
    R.within(got, ref, tol + R.rounding(dtype, ref) * 1.01, "dlogits")
    assert (got.gather(1, ids.long()) != 0).float().mean() > 0.9    # a sure choice still learns


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [16, 200, 600])
def test_bias_that_is_no_number(scoring, E):
    """An expert whose key is NaN or -inf by its bias fills a row only after all
    others, lowest index first, with weight 0."""
    T, k = 33, 8
    g = torch.Generator(device=DEV).manual_seed(E)
    logits = torch.randn(T, E, generator=g, device=DEV)
    bias = torch.full((E,), float("nan"), device=DEV)
    bias[::2] = -float("inf")
    bias[3], bias[E - 2], bias[E // 2] = 0.0, 0.1, -0.2
    ids, w = mgg.select_experts(logits, k, scoring, bias, renormalize=False)
    live = torch.tensor([3, E // 2, E - 2])
    assert torch.equal(ids[:, :3].cpu().long().sort(1).values, live.expand(T, 3))
    p, _, _ = R.scores(logits, scoring)
    R.within(w[:, :3], p.gather(1, ids[:, :3].cpu().long()), 16 * R.U, "weights")
    rest = [e for e in range(E) if e not in live.tolist()][:k - 3]
    assert torch.equal(ids[:, 3:].cpu(), torch.tensor(rest).int().expand(T, k - 3))
    assert not w[:, 3:].any()
