"""How a group of experts is scored: by its best key or its two best, with
either scoring; the rule without a word is the scoring's own."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _reference(logits, k, scoring, bias, groups, topk_groups, two):
    """(ids, rows sure of them): the definition in float64; a row is sure where
    no group and no expert is within 1e-5 of changing places (the keys are
    float32 sums of values below 2: 2e-7)."""
    z = R.d(logits)
    p = torch.softmax(z, 1) if scoring == "softmax" else torch.sigmoid(z)
    key = z if scoring == "softmax" and bias is None and not two else p + (0 if bias is None else R.d(bias))
    T, E = z.shape
    best = key.view(T, groups, E // groups).sort(dim=2, descending=True).values
    score = best[:, :, :2].sum(2) if two and E // groups > 1 else best[:, :, 0]
    order, pick = score.sort(dim=1, descending=True)
    sure = torch.ones(T, dtype=torch.bool)
    if topk_groups < groups:
        sure &= order[:, topk_groups - 1] - order[:, topk_groups] > 1e-5
    keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, pick[:, :topk_groups], True)
    key = torch.where(keep.repeat_interleave(E // groups, 1), key, torch.full_like(key, -1e300))
    srt, ids = key.sort(dim=1, descending=True)
    sure &= (srt[:, :k] - srt[:, 1:k + 1] > 1e-5).all(1)
    return ids[:, :k], sure


# (experts, groups): lane groups, groups of odd numbers of lanes, groups that
# share lanes, groups of one expert, more than 256 experts
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (224, 4), (60, 10), (16, 16), (480, 6)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_rules(E, groups, scoring, with_bias):
    T, tg = 700, max(2, groups // 2)
    k = min(6, tg * (E // groups) - 1)
    g = torch.Generator(device=DEV).manual_seed(E)
    logits = torch.randn(T, E, generator=g, device=DEV)
    bias = 0.3 * torch.rand(E, generator=g, device=DEV) if with_bias else None
    got = {}
    for rule in ("best", "two best", None):
        ids, w = mgg.select_experts(logits, k, scoring, bias, groups, tg, group_score=rule)
        two = rule == "two best" or (rule is None and scoring == "sigmoid")
        want, sure = _reference(logits, k, scoring, bias, groups, tg, two)
        assert sure.float().mean() > 0.9
        assert torch.equal(ids.cpu().long()[sure], want[sure])
        got[rule] = ids
        again, w2 = mgg.router(logits, k, scoring, bias, groups, tg, group_score=rule)
        assert torch.equal(again, ids) and torch.equal(w2, w)
    if E // groups > 1:
        assert not torch.equal(got["best"], got["two best"])
    else:
        assert torch.equal(got["best"], got["two best"])
