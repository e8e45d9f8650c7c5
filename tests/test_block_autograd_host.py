"""The differentiable calls' own part, on the CPU: the kernels behind them are
stood in for by torch operations, which autograd does not see through."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import block, ops


def _norm(x, w, b, eps, out_dtype):
    mean = x.mean(1)
    rstd = (x.var(1, correction=0) + eps) ** -0.5
    return (x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd


def _norm_backward(dy, x, w, mean, rstd, bias, ws):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


class Host:
    """What block.py asks of the compiled entry; keeps the status words given."""

    def __init__(self):
        self.status = []

    layer_norm_forward = staticmethod(_norm)
    layer_norm_backward = staticmethod(_norm_backward)

    def select_experts(self, logits, k, *_):
        w, ids = torch.softmax(logits, 1).topk(k, 1)
        return ids.int(), w

    def select_experts_backward(self, g, logits, ids, w, scoring, renorm, scale, status):
        self.status.append(status)
        return torch.zeros_like(logits).scatter(1, ids.long(), g * w)

    def linear_forward(self, x, W, b, act, res, out_dtype, save_pre, status, out):
        self.status.append(status)
        z = x @ W.t() + (0 if b is None else b)
        out = torch.tanh(z) if act else z
        out = out if res is None else out + res
        return (out, z) if save_pre else out

    def linear_backward(self, dy, x, W, pre, act, bias_dtype, need_dx, need_dW, status, ws):
        self.status.append(status)
        dz = dy if pre is None else dy * (1 - torch.tanh(pre) ** 2)
        return dz @ W, dz.t() @ x, dz.sum(0) if bias_dtype else None


@pytest.fixture
def host(monkeypatch):
    h = Host()
    monkeypatch.setattr(block, "_host", h)
    return h


def _second(f, x):
    """The gradient of a gradient penalty beside another term."""
    (g,) = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    (g.square().sum() + x.pow(3).sum()).backward()


def test_second_gradients_are_refused(host, monkeypatch):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 8, generator=g, requires_grad=True)
    w, b = torch.randn(8, generator=g), torch.randn(8, generator=g)
    W = torch.randn(3, 8, generator=g)
    monkeypatch.setattr(ops, "moe_forward", lambda x, W, ids, tw, **_: (x @ W[0].t(), None))
    monkeypatch.setattr(ops, "moe_backward", lambda dy, x, W, r, k, **_: (dy @ W[0], torch.zeros_like(W),
                                                                        torch.zeros(5, 1)))
    ids, tw = torch.zeros(5, 1, dtype=torch.int32), torch.ones(5, 1)
    for f in (lambda v: mgg.layer_norm(v, w, b), lambda v: mgg.router(v, 2)[1],
              lambda v: mgg.linear(v, W, None, "gelu"), lambda v: mgg.moe(v, W[None], ids, tw)):
        with pytest.raises(RuntimeError, match="once_differentiable"):
            _second(f, x)


def test_first_gradients(host):
    x = torch.randn(5, 8, generator=torch.Generator().manual_seed(1), requires_grad=True)
    W = torch.ones(3, 8, requires_grad=True)
    mgg.linear(x, W).sum().backward()
    assert torch.equal(x.grad, torch.full((5, 8), 3.0)) and W.grad.shape == (3, 8)


def test_one_status_word_serves_both_directions(host, monkeypatch):
    """The word a caller gives reaches every kernel call that can report an
    error, and no other word is made."""
    st = torch.zeros(1, dtype=torch.int32)
    made = []
    for m in (block, ops):
        monkeypatch.setattr(m, "new_status", lambda dev: made.append(dev) or torch.zeros(1).int())
    seen = []
    monkeypatch.setattr(ops, "moe_forward",
                        lambda x, W, ids, tw, status=None: seen.append(status) or (x @ W[0].t(), None))
    monkeypatch.setattr(ops, "moe_backward",
                        lambda dy, x, W, r, k, status=None: seen.append(status) or
                        (dy @ W[0], torch.zeros_like(W), torch.zeros(5, 1)))
    x = torch.randn(5, 8, generator=torch.Generator().manual_seed(2), requires_grad=True)
    W = torch.ones(8, 8)
    mgg.linear(x, W, None, "gelu", status=st).sum().backward()
    mgg.router(x, 2, status=st)[1].sum().backward()
    mgg.moe(x, W[None], torch.zeros(5, 1).int(), torch.ones(5, 1), status=st).sum().backward()
    words = host.status + seen
    assert len(words) == 5 and all(w is st for w in words) and not made
    mgg.linear(x, W).sum().backward()
    assert len(made) == 2       # without one: a word for each direction
