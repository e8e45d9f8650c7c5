"""AdamW over many tensors against float64: every mix of types, 32- and 8-bit
moments, sizes around the blocks and pieces, unaligned views, many tensors,
steps and rates on the device, captured steps, values that are not finite."""
import math

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R
from tests import step_ref as S

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
OPT = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def _case(sizes, pt, gt, master, bits, seed, offset=0):
    """Lists as adamw_step takes them, moments of earlier steps in them."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(n, dtype=F, std=1.0):
        return (torch.randn(n + offset, generator=g, device=DEV) * std).to(dtype)[offset:]
    w = [rand(n) for n in sizes]
    p = [x.to(pt) if offset == 0 else torch.cat([x.new_zeros(offset), x]).to(pt)[offset:] for x in w]
    grads = [rand(n, gt, 1e-2) for n in sizes]
    m, v, ms, vs = mgg.adamw_state(p, bits)
    for i, n in enumerate(sizes):
        m0, v0 = rand(n, std=3e-3), rand(n, std=1e-2).square()
        if bits == 32:
            m[i], v[i] = m0, v0 if offset else v0.clone()
        else:
            for val, codes, scale in ((m0, m[i], ms[i]), (v0.sqrt(), v[i], vs[i])):
                pad = torch.zeros(-(-n // 256) * 256, device=DEV)
                pad[:n] = val
                b = pad.view(-1, 256)
                scale.copy_(b.abs().amax(1) / 448 if n else scale)
                q = (b / scale.clamp(min=1e-30)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten()[:n]
                codes.view(torch.uint8).copy_(q)
    return p, grads, m, v, ms, vs, w if master else None


def _value(codes, scale):
    n = codes.numel()
    return R.d(codes.float()) * R.d(scale).repeat_interleave(256)[:n]


def _check(case, t, scale=None, step=None, lr=None, **more):
    p, g, m, v, ms, vs, masters = case
    opt = {**OPT, **more}
    held = masters if masters is not None else p
    before = [(R.d(held[i]), R.d(g[i].float()), R.d(m[i]) if ms is None else _value(m[i], ms[i]),
               R.d(v[i]) if vs is None else _value(v[i], vs[i]).square()) for i in range(len(p))]
    mgg.adamw_step(p, g, m, v, t if step is None else step, **{**opt, "lr": opt["lr"] if lr is None else lr},
                   masters=masters, exp_avg_scale=ms, exp_avg_sq_scale=vs, grad_scale=scale)
    for i, (p0, g0, m0, v0) in enumerate(before):
        rp, rm, rv, tol = S.adamw(p0, g0, m0, v0, t, opt["lr"], opt["betas"], opt["eps"], opt["weight_decay"],
                                  1.0 if scale is None else R.d(scale))
        R.within(held[i], rp, tol + (R.rounding(BF, rp) if held[i].dtype == BF else 0.0), f"p[{i}]")
        if masters is not None:
            assert torch.equal(p[i], masters[i].bfloat16())
        if ms is None:
            mag = opt["betas"][0] * m0.abs() + g0.abs()
            R.within(m[i], rm, 4 * R.U * mag + 1e-38, f"m[{i}]")
            R.within(v[i], rv, 8 * R.U * rv + 1e-38, f"v[{i}]")
            continue
        for codes, sc, ref, second in ((m[i], ms[i], rm, False), (v[i], vs[i], rv.sqrt(), True)):
            val, rs, near = S.grid8(ref, t, second)
            R.within(sc, rs, 8 * R.U * rs + 1e-38, "scale")
            # f32 arithmetic moves value / scale by some 8 U of at most 16 codes
            bad = (R.d(codes.float()) != val) & (near > 1e-5)
            assert not bad.any(), (i, second, int(bad.sum()))


SIZES = [1, 0, 7, 8, 255, 256, 257, 1000, 2048, 2049, 5000]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,master", [(F, F, False), (F, BF, False), (BF, BF, False), (BF, F, False),
                                          (BF, BF, True), (BF, F, True)])
def test_types_and_sizes(pt, gt, master, bits):
    case = _case(SIZES, pt, gt, master, bits, 1)
    for t in (1, 2, 100):
        _check(case, t, torch.tensor([0.3], device=DEV) if t == 2 else None)


@pytest.mark.parametrize("bits", [32, 8])
def test_unaligned_views(bits):
    for offset in (1, 3, 4):
        case = _case([300, 2300], F, BF, False, bits, 2, offset)
        if bits == 8:  # codes off their eight-byte boundaries too
            for t in (case[2], case[3]):
                for i, c in enumerate(t):
                    t[i] = torch.cat([c.view(torch.uint8)[:1], c.view(torch.uint8)])[1:].view(torch.float8_e4m3fn)
        _check(case, 5)


@pytest.mark.parametrize("count", [23, 24, 25, 400, 401, 900])
@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(count, bits):
    _check(_case([1 + 37 * i % 700 for i in range(count)], BF, BF, True, bits, count), 3)


def test_large_tensor_and_edges_between_pieces():
    _check(_case([3_000_001, 5, 1 << 20], F, BF, False, 32, 4), 7)


@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.9, 0.999), (0.5, 0.9999)])
@pytest.mark.parametrize("t", [1, 3, 100000])
def test_bias_corrections(betas, t):
    _check(_case([700], F, F, False, 32, 5), t, betas=betas, weight_decay=0.0)
    _check(_case([700], F, F, False, 32, 5), t, betas=betas, step=torch.tensor([t], dtype=torch.int32, device=DEV),
           lr=torch.tensor(OPT["lr"], device=DEV))


def test_zero_gradients_and_state():
    p = [torch.ones(600, device=DEV)]
    for bits in (32, 8):
        m, v, ms, vs = mgg.adamw_state(p, bits)
        mgg.adamw_step(p, [torch.zeros_like(p[0])], m, v, 1, **{**OPT, "weight_decay": 0.0}, exp_avg_scale=ms,
                       exp_avg_sq_scale=vs)
        assert (p[0] == 1).all() and not m[0].float().any() and not v[0].float().any()


def test_what_is_not_finite_stays_where_it_is():
    for bits in (32, 8):
        case = _case([1024], F, F, False, bits, 6)
        g = case[1][0]
        g[5], g[300], g[700] = math.nan, math.inf, -math.inf
        mgg.adamw_step(case[0], case[1], case[2], case[3], 4, **OPT, exp_avg_scale=case[4], exp_avg_sq_scale=case[5])
        odd = torch.zeros(1024, dtype=torch.bool, device=DEV)
        odd[[5, 300, 700]] = True
        assert torch.isfinite(case[0][0][~odd]).all()
        for s in case[2] + case[3]:
            assert torch.isfinite(s.float()[~odd]).all() and not torch.isfinite(s.float()[odd]).any()


def test_a_state_that_is_not_a_number_stays_one():
    """A code of NaN in either moment, as a step on a NaN gradient left it."""
    for at in (2, 3):
        case = _case([512], F, F, False, 8, 7)
        case[at][0].view(torch.uint8)[300] = 0x7F
        mgg.adamw_step(case[0], case[1], case[2], case[3], 4, **OPT, exp_avg_scale=case[4], exp_avg_sq_scale=case[5])
        for s in (case[0][0], case[at][0]):
            odd = ~torch.isfinite(s.float())
            assert odd[300] and int(odd.sum()) == 1


def test_second_moment_of_eight_bits_never_vanishes():
    """A gradient far below its block's largest: sqrt(v) stays a code above zero,
    so that its element does not leap."""
    p = [torch.zeros(256, device=DEV)]
    g = torch.full((256,), 1e-9, device=DEV)
    g[0] = 1.0
    m, v, ms, vs = mgg.adamw_state(p, 8)
    for t in range(1, 20):
        mgg.adamw_step(p, [g], m, v, t, lr=1e-3, betas=(0.9, 0.99), exp_avg_scale=ms, exp_avg_sq_scale=vs)
        assert (v[0].float() > 0).all()
    assert p[0].abs().max() <= 20 * 2e-3


def test_eight_bit_moments_follow_the_gradients():
    """Changes of less than a code add up: sqrt(v) of gradients that fall by
    half follows the float32 moment, where rounding to nearest would stay."""
    n = 4096
    gen = torch.Generator(device=DEV).manual_seed(0)
    size = torch.exp(0.5 * torch.randn(n, generator=gen, device=DEV))
    p = [torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)]
    a, b = mgg.adamw_state(p[:1], 8), mgg.adamw_state(p[1:], 32)
    for t in range(1, 1501):
        g = size * torch.randn(n, generator=gen, device=DEV) * (1.0 if t < 500 else 0.5)
        mgg.adamw_step(p[:1], [g], a[0], a[1], t, exp_avg_scale=a[2], exp_avg_sq_scale=a[3], betas=(0.9, 0.995))
        mgg.adamw_step(p[1:], [g], b[0], b[1], t, betas=(0.9, 0.995))
    ratio = (a[1][0].float().view(-1, 256) * a[3][0][:, None]).flatten() / b[1][0].sqrt()
    assert abs(ratio.mean().item() - 1) < 0.05, ratio.mean()
    assert ratio.std().item() < 0.3, ratio.std()


def test_class_mixes_types_and_skips_what_has_no_gradient():
    params = [torch.nn.Parameter(torch.randn(40, 30, device=DEV).bfloat16()), torch.nn.Parameter(torch.randn(7, device=DEV)),
              torch.nn.Parameter(torch.randn(5, device=DEV))]
    opt = mgg.AdamW(params, **OPT)
    want = []
    for p in params[:2]:
        p.grad = torch.randn(p.shape, device=DEV).to(p.dtype)
        z = torch.zeros(p.numel(), dtype=torch.double)
        want.append(S.adamw(R.d(p).flatten(), R.d(p.grad).flatten(), z, z, 1, OPT["lr"], OPT["betas"], OPT["eps"],
                            OPT["weight_decay"]))
    left = params[2].detach().clone()
    opt.step()
    R.within(opt.masters[0].flatten(), want[0][0], want[0][3], "master")
    assert torch.equal(params[0].detach(), opt.masters[0].bfloat16())
    R.within(params[1].flatten(), want[1][0], want[1][3], "p")
    assert torch.equal(params[2].detach(), left)
    opt.zero_grad()
    assert all(p.grad is None for p in params)


def test_a_graph_that_kept_the_old_parameters_notices():
    params = [torch.nn.Parameter(torch.randn(300, device=DEV).to(dt)) for dt in (BF, F)]
    opt = mgg.AdamW(params, **OPT)
    kept = sum(p.square().float().sum() for p in params)
    for p in params:
        p.grad = torch.ones_like(p)
    at = [p._version for p in params]
    opt.step()
    assert all(p._version > a for p, a in zip(params, at))
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()
    with torch.inference_mode():  # a tensor without versions
        q, g = torch.ones(40, device=DEV), torch.ones(40, device=DEV)
        m, v, _, _ = mgg.adamw_state([q])
        mgg.adamw_step([q], [g], m, v, 1)
        assert not q.eq(1).any()
    mgg.adamw_step([q], [g], m, v, 2)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_count_on(bits):
    def fresh():
        g = torch.Generator(device=DEV).manual_seed(3)
        p = torch.nn.Parameter(torch.randn(3000, generator=g, device=DEV))
        p.grad = torch.randn(3000, generator=g, device=DEV)
        return p
    lr = torch.tensor(1e-2, device=DEV)
    p, q = fresh(), fresh()
    opt = mgg.AdamW([p], lr=lr, bits=bits, capturable=True)
    ref = mgg.AdamW([q], lr=1e-2, bits=bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        opt.step()
    torch.cuda.current_stream().wait_stream(side)
    ref.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    for t in range(3):
        if t == 2:
            lr.fill_(5e-3)
            ref.lr = 5e-3
        graph.replay()
        ref.step()
    torch.cuda.synchronize()
    assert opt.count.item() == 4 and ref.count == 4
    assert (p - q).abs().max().item() <= 4 * 8 * R.U * (1e-2 + q.abs().max().item())


def test_refusals():
    def t(*shape, dtype=F):
        return torch.zeros(*shape, dtype=dtype, device=DEV)
    p, g = [t(300), t(5)], [t(300), t(5)]
    m, v = [t(300), t(5)], [t(300), t(5)]
    m8, v8, ms, vs = mgg.adamw_state(p, 8)
    flat = t(400)
    cases = [
        (ValueError, lambda: mgg.adamw_step(p, g[:1], m, v, 1)),
        (ValueError, lambda: mgg.adamw_step(p, g, m[:1], v, 1)),
        (ValueError, lambda: mgg.adamw_step(p, [t(300), t(4)], m, v, 1)),
        (TypeError, lambda: mgg.adamw_step(p, [t(300), t(5, dtype=BF)], m, v, 1)),
        (TypeError, lambda: mgg.adamw_step([t(300), t(5, dtype=BF)], g, m, v, 1)),
        (TypeError, lambda: mgg.adamw_step([x.half() for x in p], g, m, v, 1)),
        (TypeError, lambda: mgg.adamw_step(p, g, m8, v8, 1)),
        (TypeError, lambda: mgg.adamw_step(p, g, m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs)),
        (ValueError, lambda: mgg.adamw_step(p, g, m8, v8, 1, exp_avg_scale=ms)),
        (ValueError, lambda: mgg.adamw_step(p, g, m8, v8, 1, exp_avg_scale=[t(1), t(1)], exp_avg_sq_scale=vs)),
        (ValueError, lambda: mgg.adamw_step([p[0], t(10)[::2]], g, m, v, 1)),
        (ValueError, lambda: mgg.adamw_step([p[0], p[0]], [g[0], g[0]], [m[0], m[0]], [v[0], v[0]], 1)),
        (ValueError, lambda: mgg.adamw_step([flat[:300], flat[299:304]], g, m, v, 1)),
        (ValueError, lambda: mgg.adamw_step([x.cpu() for x in p], g, m, v, 1)),
        (ValueError, lambda: mgg.adamw_step(p, [x.cpu() for x in g], m, v, 1)),
        (ValueError, lambda: mgg.adamw_step(p, g, m, v, torch.tensor([1], device=DEV))),
        (ValueError, lambda: mgg.adamw_step(p, g, m, v, 1, grad_scale=t(2))),
        (RuntimeError, lambda: mgg.adamw_step(p, g, m, v, 0)),
        (RuntimeError, lambda: mgg.adamw_step(p, g, m, v, 1, betas=(1.0, 0.9))),
        (RuntimeError, lambda: mgg.adamw_step(p, g, m, v, 1, lr=-1.0)),
        (RuntimeError, lambda: mgg.adamw_step(p, g, m, v, 1, masters=[t(300), t(5)])),
        (ValueError, lambda: mgg.adamw_state(p, 4)),
    ]
    for i, (want, f) in enumerate(cases):
        with pytest.raises(want):
            f()
            pytest.fail(f"case {i} was not refused")
    mgg.adamw_step([], [], [], [], 1)
