"""The AdamW class without a GPU: what a refused step leaves behind."""
import os

import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import block, step


@pytest.fixture(scope="module")
def host():
    import __graft_entry__ as g
    from variable_size_expert_gb300 import build
    if not os.path.exists(build.HOST):
        g.build()
    return block._host


def _params():
    ps = [torch.nn.Parameter(torch.ones(3, 4).bfloat16()), torch.nn.Parameter(torch.ones(300))]
    for p in ps:
        p.grad = torch.ones_like(p)
    return ps


def test_a_refused_step_is_not_counted(host, monkeypatch):
    opt = mgg.AdamW(_params())
    with pytest.raises(ValueError, match="CUDA"):
        opt.step()                              # the first call's own refusal
    assert opt.count == 0
    calls = []
    monkeypatch.setattr(step, "adamw_step", lambda *a: calls.append(a))
    opt.step()
    assert opt.count == 1 and [c[4] for c in calls] == [1, 1]


def test_the_check_refuses_what_the_step_refuses(host):
    x = torch.zeros(4)
    good = ([x], [x], [x], [x], 1, 1e-3, 0.9, 0.99, 1e-8, 0.0, None, None, None, None)
    for at, bad in ((0, 3), (0, [1.0]), (1, []), (4, "1"), (5, "x"), (11, [x]), (0, [x])):
        args = good[:at] + (bad,) + good[at + 1:]
        kinds = []
        for f in (host.adamw_step, host.adamw_check):
            with pytest.raises((TypeError, ValueError)) as e:
                f(*args)
            kinds.append((e.type, str(e.value)))
        assert kinds[0] == kinds[1], at
    assert host.adamw_check(*([[]] * 4), *good[4:]) is None


def test_masters_take_over_what_was_written(monkeypatch):
    monkeypatch.setattr(step, "adamw_step", lambda *a: None)
    ps = _params() + [torch.nn.Parameter(torch.ones(5).bfloat16())]
    opt = mgg.AdamW(ps)
    assert [m is None for m in opt.masters] == [False, True, False]
    opt.masters[0].add_(1e-4)                  # (bits that bfloat16 does not hold)
    low = opt.masters[0].clone()
    assert torch.equal(low.bfloat16(), ps[0].detach())
    opt.step()
    assert torch.equal(opt.masters[0], low)    # nothing was written
    with torch.no_grad():
        ps[0][1, 2] = 7.0
        ps[2].fill_(2.0)
    opt.step()
    low[1, 2] = 7.0
    assert torch.equal(opt.masters[0], low)
    assert (opt.masters[2] == 1).all()         # (no gradient yet: when one comes)
    ps[2].grad = torch.ones(5).bfloat16()
    opt.step()
    assert (opt.masters[2] == 2).all()
    ps[0].data.fill_(3.0)                      # (counts no version)
    opt.step()
    assert torch.equal(opt.masters[0], low)
    opt.sync_masters()
    assert (opt.masters[0] == 3).all()
    with torch.inference_mode():
        q = torch.ones(4).bfloat16()
        q.grad = torch.ones(4).bfloat16()
        mgg.AdamW([q]).step()
