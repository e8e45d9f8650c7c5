"""The AdamW class where a step is refused: nothing of it has happened, neither an
update nor a count."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _model(seed=0):
    """Parameters of two mixes of types, with gradients."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ps = [torch.nn.Parameter(torch.randn(20, 30, generator=g, device=DEV).to(dt))
          for dt in (torch.bfloat16, torch.float32, torch.bfloat16)]
    for p in ps:
        p.grad = torch.randn(20, 30, generator=g, device=DEV).to(p.dtype)
    return ps


def _held(opt):
    lists = (opt.params, opt.masters, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale)
    ts = [t.detach() for l in lists if l is not None for t in l if t is not None]
    return [(t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).clone() for t in ts] + [
        torch.as_tensor(opt.count).clone().cpu()]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_changes_nothing(bits, capturable):
    ps, qs = _model(), _model()
    opt, ref = (mgg.AdamW(x, lr=1e-2, bits=bits, capturable=capturable) for x in (ps, qs))
    opt.step()
    ref.step()
    before = _held(opt)
    good = ps[1].grad
    bad = (torch.zeros(30, 20, device=DEV).t(),       # not contiguous
           )
    for grad in bad:
        ps[1].grad = grad
        with pytest.raises(ValueError):
            opt.step()
        assert _same(_held(opt), before)
    ps[1].grad = good
    with pytest.raises(ValueError):
        opt.step(grad_scale=torch.ones(2, device=DEV))
    assert _same(_held(opt), before)
    for lr, betas, want in ((-1.0, (0.9, 0.999), L.MggError), (1e-2, (1.0, 0.999), L.MggError), ("x", (0.9, 0.9), TypeError)):
        opt.lr, opt.betas = lr, betas
        with pytest.raises(want):
            opt.step()
        assert _same(_held(opt), before)
    opt.lr, opt.betas = 1e-2, (0.9, 0.999)
    opt.step()
    ref.step()
    assert _same(_held(opt), _held(ref))
