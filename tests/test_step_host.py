"""Refusals of the losses and the optimiser, checked before the device is
touched: the C ABI's status codes, the torch API's exceptions on CPU tensors and
for operands elsewhere, and the differentiable calls' own part."""
import ctypes
import math
import os

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests.test_block_devices_host import BF, F, I, Claim
from variable_size_expert_gb300 import block, step

FAKE = 0x10000      # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    from variable_size_expert_gb300 import _lib, build
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(build.HOST)):
        g.build()
    return _lib.load()


def test_balance_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al, dt = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT, L.MGG_ERR_DTYPE

    def f(l=FAKE, d=1, ldl=16, ids=FAKE, mask=None, T=4, E=16, k=2, B=1, sc=0, loss=FAKE, counts=FAKE, slope=FAKE,
          st=FAKE):
        return lib.mgg_balance_loss(l, d, ldl, ids, mask, T, E, k, B, sc, loss, counts, slope, st, FAKE, 1 << 30, None)
    for kw, want in ((dict(l=None), inv), (dict(ids=None), inv), (dict(loss=None), inv), (dict(counts=None), inv),
                     (dict(slope=None), inv), (dict(st=None), inv), (dict(T=-1), inv), (dict(E=0), inv),
                     (dict(E=1025, ldl=1025), inv), (dict(k=0), inv), (dict(k=33), inv), (dict(ldl=15), inv),
                     (dict(B=0), inv), (dict(B=3), inv), (dict(sc=2), inv), (dict(sc=0x100), inv), (dict(d=2), dt),
                     (dict(l=FAKE + 2), al), (dict(ids=FAKE + 1), al), (dict(slope=FAKE + 2), al), (dict(T=(1 << 30) + 1), inv)):
        assert f(**kw) == want, kw

    def b(g=FAKE, l=FAKE, d=1, slope=FAKE, T=4, E=16, B=1, sc=0, out=FAKE):
        return lib.mgg_balance_loss_backward(g, l, d, 16, slope, None, T, E, B, sc, out, None)
    for kw, want in ((dict(g=None), inv), (dict(l=None), inv), (dict(slope=None), inv), (dict(out=None), inv),
                     (dict(E=17), inv), (dict(B=3), inv), (dict(sc=5), inv), (dict(d=3), dt), (dict(out=FAKE + 2), al)):
        assert b(**kw) == want, kw
    assert b(T=0, l=None, out=None) == L.MGG_OK
    ws = lambda T, B, E: lib.mgg_workspace_bytes(L.MGG_OP_BALANCE, T, B, E, 0, 0, 1)  # noqa: E731
    assert ws(0, 1, 8) == 0 and ws(10, 3, 8) == 0 and ws(4, 1, 2000) == 0
    # the sums and the counts of a sequence's block at least
    assert ws(4096, 64, 128) >= 64 * 128 * 8


def test_cross_entropy_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT

    def f(x=FAKE, ldx=64, W=FAKE, t=FAKE, i64=1, T=4, K=64, V=24, red=2, zl=0.0, loss=FAKE, lse=FAKE, w=FAKE, st=FAKE):
        return lib.mgg_linear_cross_entropy(x, ldx, W, t, i64, -100, T, K, V, red, zl, loss, lse, w, st, FAKE, 1 << 40,
                                            None)
    for kw, want in ((dict(x=None), inv), (dict(W=None), inv), (dict(t=None), inv), (dict(loss=None), inv),
                     (dict(lse=None), inv), (dict(w=None), inv), (dict(st=None), inv), (dict(T=-1), inv),
                     (dict(K=0), inv), (dict(V=0), inv), (dict(ldx=56), inv), (dict(red=3), inv), (dict(red=-1), inv),
                     (dict(zl=-1.0), inv), (dict(zl=math.nan), inv), (dict(zl=math.inf), inv), (dict(K=60), al),
                     (dict(ldx=68), al), (dict(x=FAKE + 8), al), (dict(W=FAKE + 8), al), (dict(t=FAKE + 4), al),
                     (dict(i64=0, t=FAKE + 2), al), (dict(lse=FAKE + 2), al), (dict(T=(1 << 30) + 1), inv),
                     (dict(V=(1 << 30) + 1), inv), (dict(K=(1 << 30) + 8, ldx=1 << 31), inv)):
        assert f(**kw) == want, kw

    def b(g=FAKE, w=FAKE, x=FAKE, W=FAKE, t=FAKE, lse=FAKE, T=4, K=64, V=24, zl=0.0, dx=FAKE, dW=FAKE, st=FAKE):
        return lib.mgg_linear_cross_entropy_backward(g, 0, w, x, K, W, t, 1, -100, lse, T, K, V, zl, dx, dW, st, FAKE,
                                                     1 << 40, None)
    for kw, want in ((dict(g=None), inv), (dict(w=None), inv), (dict(x=None), inv), (dict(W=None), inv),
                     (dict(t=None), inv), (dict(lse=None), inv), (dict(st=None), inv), (dict(V=0), inv),
                     (dict(zl=-0.5), inv), (dict(K=60), al), (dict(dx=FAKE + 8), al), (dict(dW=FAKE + 8), al),
                     (dict(g=FAKE + 2), al)):
        assert b(**kw) == want, kw
    ws = lambda op, T, V, K: lib.mgg_workspace_bytes(op, T, 0, 0, V, K, 0)  # noqa: E731
    assert ws(L.MGG_OP_VOCAB_FORWARD, 0, 8, 8) == ws(L.MGG_OP_VOCAB_BACKWARD, 4, 0, 8) == 0
    # a pair a tile and token; a piece of the logits' gradient, bounded whatever V
    assert ws(L.MGG_OP_VOCAB_FORWARD, 1000, 25600, 64) >= 100 * 1000 * 8
    assert ws(L.MGG_OP_VOCAB_BACKWARD, 1000, 4096, 64) >= 1000 * 4096 * 2
    assert ws(L.MGG_OP_VOCAB_BACKWARD, 8192, 1 << 20, 1024) < 512 << 20


def test_piece_setting(lib, monkeypatch):
    from variable_size_expert_gb300 import _lib as L
    ws = lambda: lib.mgg_workspace_bytes(L.MGG_OP_VOCAB_BACKWARD, 1000, 0, 0, 65536, 1024, 0)  # noqa: E731
    whole = ws()
    monkeypatch.setenv("MGG_VOCAB_PIECE", "1000")
    assert ws() < whole / 4
    monkeypatch.setenv("MGG_VOCAB_PIECE", "none")
    assert ws() == whole


def test_adamw_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al, dt = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT, L.MGG_ERR_DTYPE

    def f(bits=32, pd=1, gd=1, lr=1e-3, lrd=None, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, sd=None, gs=None, count=1,
          second=None, **kw):
        a = dict(param=FAKE, master=None, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=None,
                 exp_avg_sq_scale=None, n=8)
        ts = [L.AdamwTensor(**{**a, **kw}), L.AdamwTensor(**{**a, **kw, **(second or {})})]
        return lib.mgg_adamw_step((L.AdamwTensor * 2)(*ts), 2 if second else count, pd, gd, bits, lr, lrd, b1, b2, eps,
                                  wd, step, sd, gs, None)
    for kw, want in ((dict(param=None), inv), (dict(grad=None), inv), (dict(exp_avg=None), inv),
                     (dict(exp_avg_sq=None), inv), (dict(n=-1), inv), (dict(count=-1), inv), (dict(bits=16), inv),
                     (dict(bits=8), inv), (dict(bits=8, exp_avg_scale=FAKE), inv), (dict(b1=1.0), inv),
                     (dict(b2=-0.1), inv), (dict(b1=math.nan), inv), (dict(lr=-1.0), inv), (dict(lr=math.inf), inv),
                     (dict(eps=-1e-8), inv), (dict(wd=math.nan), inv), (dict(step=0), inv), (dict(step=-3), inv),
                     (dict(master=FAKE), inv), (dict(pd=0, second=dict(master=FAKE)), inv), (dict(pd=2), dt),
                     (dict(gd=7), dt), (dict(param=FAKE + 2), al), (dict(pd=0, param=FAKE + 1), al),
                     (dict(grad=FAKE + 2), al), (dict(exp_avg=FAKE + 1), al), (dict(gs=FAKE + 1), al),
                     (dict(sd=FAKE + 2), al), (dict(lrd=FAKE + 2), al)):
        assert f(**kw) == want, kw
    assert f(count=0) == L.MGG_OK and f(n=0, param=None) == L.MGG_OK
    assert lib.mgg_adamw_step(None, 1, 1, 1, 32, 0.1, None, 0.9, 0.9, 0.0, 0.0, 1, None, None, None) == inv


def test_torch_api_refusals(lib):
    x, b = torch.zeros(4, 64), torch.zeros(4, 64).bfloat16()
    ids, t, st = torch.zeros(4, 2).int(), torch.zeros(4).long(), torch.zeros(1).int()
    cases = [
        (ValueError, lambda: mgg.balance_loss_forward(x, ids, status=st)),                 # not on a GPU
        (ValueError, lambda: mgg.balance_loss_forward(x, ids, scoring="tanh", status=st)),
        (TypeError, lambda: mgg.balance_loss_forward([1.0], ids, status=st)),
        (ValueError, lambda: mgg.balance_loss_backward(x[0, 0], x, x[:1])),
        (ValueError, lambda: mgg.linear_cross_entropy_forward(b, b, t, status=st)),
        (TypeError, lambda: mgg.linear_cross_entropy_forward(x, b, t, status=st)),
        (ValueError, lambda: mgg.linear_cross_entropy_forward(b, b, t, reduction="max", status=st)),
        (ValueError, lambda: mgg.linear_cross_entropy_backward(x[0, 0], b, b, t, x[:, 0], x[0, :1], status=st)),
        (ValueError, lambda: mgg.adamw_step([x], [x], [x], [x], 1)),
        (TypeError, lambda: mgg.adamw_step(3, [x], [x], [x], 1)),
        (TypeError, lambda: mgg.adamw_step([1.0], [x], [x], [x], 1)),
        (ValueError, lambda: mgg.adamw_step([x], [], [x], [x], 1)),
        (TypeError, lambda: mgg.adamw_step([x], [x], [x], [x], "1")),
        (ValueError, lambda: mgg.adamw_state([x], 16)),
    ]
    for i, (want, f) in enumerate(cases):
        with pytest.raises(want):
            f()
            pytest.fail(f"case {i} was not refused")


T, K, V, E, k = 4, 64, 24, 16, 2
CALLS = {
    "balance_loss_forward": (lambda logits, expert_ids, mask, status:
                             mgg.balance_loss_forward(logits, expert_ids, mask=mask, status=status),
                             dict(logits=((T, E), F), expert_ids=((T, k), I), mask=((T,), torch.bool),
                                  status=((1,), I))),
    "balance_loss_backward": (lambda dloss, logits, slope, mask:
                              mgg.balance_loss_backward(dloss, logits, slope, mask=mask),
                              dict(dloss=((), F), logits=((T, E), F), slope=((1, E), F), mask=((T,), torch.bool))),
    "linear_cross_entropy_forward": (lambda x, W, targets, status:
                                     mgg.linear_cross_entropy_forward(x, W, targets, status=status),
                                     dict(x=((T, K), BF), W=((V, K), BF), targets=((T,), torch.long),
                                          status=((1,), I))),
    "linear_cross_entropy_backward": (lambda dloss, x, W, targets, lse, weight, status:
                                      mgg.linear_cross_entropy_backward(dloss, x, W, targets, lse, weight,
                                                                        status=status),
                                      dict(dloss=((), F), x=((T, K), BF), W=((V, K), BF), targets=((T,), torch.long),
                                           lse=((T,), F), weight=((1,), F), status=((1,), I))),
}
CASES = [(c, a) for c, (_, args) in CALLS.items() for a in list(args)[1:]]


@pytest.mark.parametrize("call,arg", CASES, ids=[f"{c}-{a}" for c, a in CASES])
@pytest.mark.parametrize("where", ["cuda:1", "cpu"])
def test_operand_elsewhere(lib, call, arg, where):
    f, args = CALLS[call]
    ts = {n: Claim(s, d, where if n == arg else "cuda:0") for n, (s, d) in args.items()}
    with pytest.raises(ValueError, match=f"^{arg} must be on the first argument's device"):
        f(**ts)


class Host:
    """What step.py asks of the compiled entry, in torch operations; keeps the
    status words given."""

    def __init__(self):
        self.status = []

    def balance_loss_forward(self, logits, ids, scoring, mask, sequences, status, ws):
        self.status.append(status)
        return torch.softmax(logits, 1).mean(0)[0].detach(), torch.zeros(1, logits.shape[1]).int(), logits[:1].detach()

    def balance_loss_backward(self, dloss, logits, slope, scoring, mask):
        return dloss * torch.ones_like(logits)

    def linear_cross_entropy_forward(self, x, W, t, ignore, reduction, z_loss, status, ws):
        self.status.append(status)
        return (x @ W.t()).sum().detach(), torch.zeros(len(x)), torch.ones(1)

    def linear_cross_entropy_backward(self, g, x, W, t, lse, weight, ignore, z_loss, need_dx, need_dW, status, ws):
        self.status.append(status)
        assert g.is_contiguous()
        return (g * torch.ones_like(x) if need_dx else None), (g * torch.ones_like(W) if need_dW else None)


def test_autograd_of_the_losses(monkeypatch):
    host = Host()
    monkeypatch.setattr(block, "_host", host)
    st = torch.zeros(1).int()
    z, x, W = (torch.randn(5, 8, requires_grad=True) for _ in range(3))
    ids, t = torch.zeros(5, 2).int(), torch.zeros(5).long()
    loss, counts = mgg.balance_loss(z, ids, status=st)
    assert not counts.requires_grad
    (2 * loss + 3 * mgg.linear_cross_entropy(x, W, t, status=st)).backward()
    assert torch.equal(z.grad, torch.full((5, 8), 2.0)) and torch.equal(x.grad, torch.full((5, 8), 3.0))
    assert torch.equal(W.grad, torch.full((5, 8), 3.0)) and all(s is st for s in host.status) and len(host.status) == 3
    # one operand without a gradient
    mgg.linear_cross_entropy(x.detach(), W, t, status=st).backward()
    made = []
    monkeypatch.setattr(step, "new_status", lambda dev: made.append(dev) or torch.zeros(1).int())
    mgg.linear_cross_entropy(x, W, t).backward()
    assert len(made) == 2       # without one: a word for each direction
    for f in (lambda v: mgg.balance_loss(v, ids)[0], lambda v: mgg.linear_cross_entropy(v, W, t)):
        (g,) = torch.autograd.grad(f(x).square(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.square().sum() + x.pow(3).sum()).backward()


def test_adamw_state_of_any_iterable():
    ps = [torch.zeros(3, 5), torch.zeros(300), torch.zeros(0)]
    for bits, blocks in ((32, None), (8, [1, 2, 0])):
        m, v, ms, vs = mgg.adamw_state(iter(ps), bits)
        assert [x.shape for x in m] == [x.shape for x in v] == [x.shape for x in ps]
        assert ms is None and vs is None if blocks is None else [len(x) for x in ms] == [len(x) for x in vs] == blocks


def test_adamw_class_keeps_its_own_count(monkeypatch):
    calls = []
    monkeypatch.setattr(step, "adamw_step", lambda *a: calls.append(a))
    ps = [torch.nn.Parameter(torch.ones(3, 4).bfloat16()), torch.nn.Parameter(torch.ones(300)),
          torch.nn.Parameter(torch.ones(5))]
    opt = mgg.AdamW(ps, lr=0.1, bits=8)
    assert [m is None for m in opt.masters] == [False, True, True] and opt.exp_avg[1].dtype == torch.float8_e4m3fn
    assert opt.exp_avg_scale[1].shape == (2,) and opt.exp_avg[0].shape == (3, 4)
    ps[0].grad, ps[1].grad = torch.ones(3, 4).bfloat16(), torch.ones(300)
    opt.step()
    opt.step()
    assert len(calls) == 4 and [c[4] for c in calls] == [1, 1, 2, 2]
    assert [len(c[0]) for c in calls] == [1, 1, 1, 1] and calls[1][9] is None and calls[0][9][0] is opt.masters[0]
    opt.zero_grad()
    opt.step()
    assert len(calls) == 4 and opt.count == 3
