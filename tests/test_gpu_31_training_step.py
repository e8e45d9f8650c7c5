"""The losses and the optimiser together, as a training step uses them: every
gradient against float64 autograd, the example's token model for a few steps,
and a whole step captured and replayed."""
import os
import sys

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R
from tests import step_ref as S
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block
    return moe_block


def _rounded(v):
    """v with its bfloat16 rounding, the rounding's gradient the identity."""
    return v + (v.detach().float().bfloat16().double() - v.detach())


def test_gradients_against_float64():
    ex = _example()
    g = torch.Generator(device=DEV).manual_seed(5)
    V, T, H, E, k, aux = 300, 140, 128, 8, 2, 0.5
    model = ex.TokenModel(V, H, E, k, generator=g)
    text = torch.randint(0, V, (T,), device=DEV, generator=g)
    targets = torch.where(torch.rand(T, device=DEV, generator=g) < 0.2, S.IGNORE, text.flip(0))
    loss, ce = model(text, targets, aux)
    loss.backward()
    assert mgg.read_status(model.block.status) == 0

    p = {n: R.d(v).requires_grad_() for n, v in model.named_parameters()}
    b = {n[6:]: v for n, v in p.items() if n.startswith("block.")}
    t = text.cpu()
    x = p["embedding"][t]
    h = _rounded(R.norm_forward(x, b["norm_w"], b["norm_b"], 1e-5)[0])
    logits = h @ b["gate"].t()
    # the experts chosen are those of the kernels, held fixed
    with torch.no_grad():
        hk = mgg.layer_norm(model.embedding[text], model.block.norm_w, model.block.norm_b, out_dtype=torch.bfloat16)
        ids, _ = mgg.router(mgg.linear(hk, model.block.gate, out_dtype=torch.float32), k, "sigmoid",
                            bias=model.block.balance)
    i = ids.cpu().long()
    w = R.weights_of(logits, i, torch.ones(T, k, dtype=torch.bool), "sigmoid", True, 1.0)
    per = torch.einsum("tk,enk->ten", h, b["experts"])
    y = (per.gather(1, i[:, :, None].expand(T, k, H)) * w[:, :, None]).sum(1)
    s = R.act(h @ b["up"].t() + b["up_b"], "gelu")
    out = x + y + s @ b["down"].t()
    z = _rounded(R.norm_forward(out, p["norm_w"], p["norm_b"], 1e-5)[0]) @ p["head"].t()
    on = targets.cpu() >= 0
    ref_ce = (torch.logsumexp(z, 1) - z.gather(1, targets.cpu().clamp(min=0)[:, None])[:, 0])[on].mean()
    a = torch.sigmoid(logits)
    share = E * torch.bincount(i.flatten(), minlength=E).double() / (k * T)
    ref = ref_ce + aux * (share * (a / a.sum(1, keepdim=True)).mean(0)).sum()
    ref.backward()
    assert abs(ce.item() - ref_ce.item()) <= 9e-3 * abs(ref_ce.item())
    # bfloat16 activations and gradients between the layers: of the seven roundings
    # of root mean square 1.7e-3 that one path holds, at most six meet in one value
    # beside its own: sqrt(7) * 1.7e-3, and twice that for their unequal sizes
    for n, v in model.named_parameters():
        err = float((R.d(v.grad) - p[n].grad).norm() / p[n].grad.norm())
        assert err <= 9e-3, (n, err)


@pytest.mark.parametrize("bits", [32, 8])
def test_token_model_trains(bits):
    losses = _example().train_tokens(vocabulary=501, tokens=700, hidden=128, experts=8, steps=3, bits=bits,
                                     log=lambda s: None)
    assert len(losses) == 3 and all(l == l and l < 50 for l in losses)


def test_balance_loss_in_the_block_example():
    losses = _example().train(tokens=256, hidden=128, shared=128, experts=8, steps=2, aux=0.1, log=lambda s: None)
    assert all(l == l for l in losses)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_captured_and_replayed(bits):
    """Losses, gradients and update in one graph, its replays against eager
    steps from the same start."""
    T, H, E, V, k = 96, 64, 8, 700, 2

    def fresh():
        g = torch.Generator(device=DEV).manual_seed(1)
        ps = [torch.nn.Parameter((torch.randn(*s, generator=g, device=DEV) / H ** 0.5).bfloat16())
              for s in ((E, H), (V, H))]
        return ps, mgg.AdamW(ps, lr=1e-2, bits=bits, capturable=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device=DEV)
    st = mgg.new_status(DEV)

    def step(ps, opt):
        gate, head = ps
        logits = mgg.linear(x, gate, out_dtype=torch.float32, status=st)
        ids, w = mgg.router(logits, k, status=st)
        aux, counts = mgg.balance_loss(logits, ids, status=st)
        loss = mgg.linear_cross_entropy(x, head, t, status=st) + aux + w.sum() * 1e-3
        loss.backward()
        opt.step()
        opt.zero_grad()
        return loss.detach(), counts
    ps, opt = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ps, opt)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, counts = step(ps, opt)
    got = []
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got.append((loss.item(), counts.clone()))
    qs, ref = fresh()
    step(qs, ref)
    for l, c in got:
        rl, rc = step(qs, ref)
        assert l == rl.item() and torch.equal(c, rc)
    assert all(torch.equal(a, b) for a, b in zip(ps, qs)) and mgg.read_status(st) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, do not meet."""
    x = torch.randn(300, 128, device=DEV).bfloat16()
    Ws = [(torch.randn(2000 + 300 * i, 128, device=DEV) / 11).bfloat16() for i in range(2)]
    t = torch.randint(0, 2000, (300,), device=DEV)
    alone = [mgg.linear_cross_entropy_forward(x, W, t)[:2] for W in Ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Ws]
    for _ in range(20):
        outs = []
        for s, W in zip(streams, Ws):
            with torch.cuda.stream(s):
                outs.append(mgg.linear_cross_entropy_forward(x, W, t)[:2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, r in zip(outs, alone) for a, b in zip(o, r))
