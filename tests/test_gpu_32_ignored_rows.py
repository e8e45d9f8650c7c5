"""Tokens that do not count, whatever their hidden states hold: NaN, infinities and
the largest finite numbers in rows of x whose target is ignored or lies outside the
vocabulary leave the loss and both gradients as they are, bit for bit."""
import math

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import step_ref as S
from variable_size_expert_gb300 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _inputs(T, K, V, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    W = (torch.randn(V, K, generator=g, device=DEV) / K ** 0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device=DEV)
    off = torch.rand(T, generator=g, device=DEV) < 0.4
    off[0], off[-1] = True, T == 1
    return x, W, t, off


def _both(x, W, t, reduction, **kw):
    st = mgg.new_status(DEV)
    loss, lse, w = mgg.linear_cross_entropy_forward(x, W, t, reduction=reduction, z_loss=1e-3, status=st)
    dloss = torch.linspace(-1.0, 2.0, len(t), device=DEV) if reduction == "none" else torch.tensor(1.7, device=DEV)
    dx, dW = mgg.linear_cross_entropy_backward(dloss, x, W, t, lse, w, z_loss=1e-3, status=st, **kw)
    return loss, dx, dW, mgg.read_status(st)


# every way that the gradients go: one pass over W (up to 4 tokens), d in two parts (up
# to 128), one part with x's rows on 64-byte lines and off them, W's pieces copied (2048
# tokens on), clusters
@pytest.mark.parametrize("T,K,V", [(1, 64, 300), (2, 1032, 700), (4, 2056, 3000), (5, 4096, 300), (32, 520, 20001),
                                   (70, 64, 700), (128, 264, 515), (129, 576, 130), (200, 128, 4097), (255, 72, 1000),
                                   (300, 192, 1000), (513, 1032, 513), (2050, 40, 700)])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_rows_that_do_not_count(T, K, V, reduction):
    x, W, t, off = _inputs(T, K, V, T + K)
    t = torch.where(off, S.IGNORE, t)
    want = _both(x, W, t, reduction)
    assert all(torch.isfinite(v).all() for v in want[:3]) and want[3] == 0
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(BF).max):
        y = torch.where(off[:, None], bad, x)
        got = _both(y, W, t, reduction)
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3])), bad
        dW = _both(y, W, t, reduction, need_dx=False)[2]
        dx = _both(y, W, t, reduction, need_dW=False)[1]
        assert torch.equal(dW, want[2]) and torch.equal(dx, want[1])


@pytest.mark.parametrize("T", [3, 100, 300])
def test_bad_targets_and_pieces(T, monkeypatch):
    """The same of targets outside the vocabulary, over pieces of it."""
    monkeypatch.setenv("MGG_VOCAB_PIECE", "256")
    x, W, t, off = _inputs(T, 72, 1000, T)
    for dtype in (torch.int64, torch.int32):
        u = torch.where(off, 1000, t).to(dtype)
        want = _both(x, W, u, "mean")
        got = _both(torch.where(off[:, None], math.nan, x), W, u, "mean")
        assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
        assert got[3] == want[3] == L.MGG_DEV_BAD_TARGET


def test_differentiable_call_and_strided_rows():
    x, W, t, off = _inputs(140, 96, 600, 9)
    t = torch.where(off, S.IGNORE, t)
    wide = torch.full((140, 112), math.nan, dtype=BF, device=DEV)
    wide[:, 8:104] = torch.where(off[:, None], math.nan, x)
    grads = []
    for v in (x, wide[:, 8:104]):
        a, b = v.detach().requires_grad_(), W.clone().requires_grad_()
        mgg.linear_cross_entropy(a, b, t).backward()
        grads.append((a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*grads))
    assert not grads[1][0][off].any()
