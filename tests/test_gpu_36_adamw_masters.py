"""Masters of the AdamW class follow what is written into their parameters between
two steps: weights that are loaded, elements that are clamped."""
import pytest
import torch

import variable_size_expert_gb300 as mgg

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _param(seed=0, n=3000):
    g = torch.Generator(device=DEV).manual_seed(seed)
    p = torch.nn.Parameter(torch.randn(n, generator=g, device=DEV).to(BF))
    p.grad = torch.randn(n, generator=g, device=DEV).to(BF)
    return p


def test_loaded_weights_are_stepped_on():
    """From loaded weights the step is that of an optimiser whose masters they are
    (but for elements that are loaded as they were: those keep their master)."""
    p, q = _param(), _param()
    opt, ref = mgg.AdamW([p], lr=1e-2), mgg.AdamW([q], lr=1e-2)
    opt.step()
    ref.step()
    loaded = _param(7).detach()
    as_they_were = loaded == p.detach()
    assert 0 < int(as_they_were.sum()) < 100
    torch.nn.ParameterList([p]).load_state_dict({"0": loaded})
    ref.masters[0].copy_(torch.where(as_they_were, ref.masters[0], loaded.float()))
    with torch.no_grad():
        q.copy_(loaded)
    opt.step()
    ref.step()
    assert torch.equal(p, q) and torch.equal(opt.masters[0], ref.masters[0])
    assert (p.float() - loaded.float()).abs().max() < 0.1


def test_a_resumed_run_keeps_its_masters():
    """Params and masters of a checkpoint, both loaded: the masters' bits stay."""
    p, q = _param(), _param(3)
    opt, ref = mgg.AdamW([q], lr=1e-2), mgg.AdamW([p], lr=1e-2)
    for _ in range(3):
        ref.step()
    with torch.no_grad():
        q.copy_(p)
    q.grad = p.grad
    for a, b in zip(opt.masters + opt.exp_avg + opt.exp_avg_sq, ref.masters + ref.exp_avg + ref.exp_avg_sq):
        a.copy_(b)
    opt.count = ref.count
    opt.step()
    ref.step()
    assert torch.equal(p, q) and torch.equal(opt.masters[0], ref.masters[0])


def test_what_was_not_written_keeps_its_bits():
    p = _param()
    opt = mgg.AdamW([p], lr=1e-3)
    opt.step()
    held = opt.masters[0].clone()
    low = p.detach().float() < 0.5
    with torch.no_grad():
        p.clamp_(min=0.5)
    opt.sync_masters()
    assert torch.equal(opt.masters[0], torch.where(low, 0.5, held))
    assert not torch.equal(opt.masters[0], p.detach().float())      # (bits below bfloat16's)
    opt.step()
    assert torch.equal(p.detach(), opt.masters[0].to(BF))


def test_written_before_the_first_step_and_behind_the_versions():
    p = _param()
    opt = mgg.AdamW([p], lr=1e-2, weight_decay=0.0)
    with torch.no_grad():
        p.fill_(3.0)
    p.grad.zero_()
    opt.step()
    assert (p == 3).all() and (opt.masters[0] == 3).all()
    p.data.fill_(5.0)                       # (.data counts no version)
    opt.sync_masters()
    opt.step()
    assert (p == 5).all() and (opt.masters[0] == 5).all()


def test_captured_steps_keep_their_masters():
    """Nothing is written between the steps: a replay adds up below bfloat16's bits."""
    p, q = _param(), _param()
    opt, ref = (mgg.AdamW([x], lr=1e-5, capturable=True) for x in (p, q))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step()
    torch.cuda.current_stream().wait_stream(side)
    ref.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for _ in range(4):
        graph.replay()
        ref.step()
    torch.cuda.synchronize()
    assert torch.equal(opt.masters[0], ref.masters[0]) and torch.equal(p, q)
