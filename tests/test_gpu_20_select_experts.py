"""The expert choice and its gradient against float64: exact ids where the
keys are the logits themselves (ties included), optimality within rounding
where they are computed scores, masks, groups, and gradients by the chain
rule and by differences."""
import math

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
NINF = -math.inf
# a score is within 8 U of its value (exp within 2 ulp, sum, divide, times),
# softmax's sum adds its depth; keys p + bias add one rounding of at most 2
TOL = 64 * R.U


def _logits(T, E, dt, seed, coarse=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = 1.5 * torch.randn(T, E, generator=g, device=DEV)
    if coarse:
        l = (l * 2).round() / 2        # many equal logits
    return l.to(dt), g


def _check(logits, k, scoring, bias=None, groups=1, topk_groups=1, renorm=True, scale=1.0):
    ids, w = mgg.select_experts(logits, k, scoring=scoring, bias=bias, groups=groups,
                                topk_groups=topk_groups, renormalize=renorm, scale=scale)
    T, E = logits.shape
    assert ids.shape == w.shape == (T, k) and ids.dtype == torch.int32 and w.dtype == F
    rid, rw, key = R.select(logits, k, scoring, bias, groups, topk_groups, renorm, scale)
    i = ids.cpu().long()
    assert ((i >= 0) & (i < E)).all()
    assert (i.sort(1).values.diff(dim=1) > 0).all(), "ids repeat"
    if scoring == "softmax" and bias is None:
        assert torch.equal(i, rid)
    else:
        # best first, and nothing better left out, within the scores' rounding
        got, best = key.gather(1, i), key.gather(1, rid)
        same = (got == best) | ((got - best).abs() <= TOL * 2)
        assert same.all(), "not the best keys in order"
    # the weights of the ids that were chosen
    p, _, _ = R.scores(logits, scoring)
    chosen = torch.where(key.gather(1, i) > NINF, p.gather(1, i), torch.zeros(T, k).double())
    rw = R.weigh(chosen, renorm, scale)
    R.within(w, rw, TOL * rw + 1e-38, "weights")
    return ids, w


@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 8, 2), (9, 31, 5), (64, 33, 4),
                                   (65, 64, 8), (7, 96, 6), (129, 128, 8), (17, 160, 32),
                                   (40, 256, 8), (5, 257, 7), (6, 512, 16), (3, 1000, 3),
                                   (4, 1024, 32)])
def test_choice(T, E, k, scoring, dt):
    l, g = _logits(T, E, dt, T * 7 + E)
    bias = 0.3 * torch.randn(E, generator=g, device=DEV) if (T + E) % 2 else None
    _check(l, k, scoring, renorm=k > 2, scale=1.0 if E % 3 else 2.5)
    if bias is not None:
        _check(l, k, scoring, bias=bias)


@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(scoring, dt):
    l, _ = _logits(200, 96, dt, 3, coarse=True)
    ids, _ = _check(l, 12, scoring)
    # equal logits have equal scores: the order is the stable one of the logits
    ref = torch.sort(l.float().cpu(), dim=1, descending=True, stable=True).indices[:, :12]
    assert torch.equal(ids.cpu().long(), ref)
    l = torch.zeros(5, 70, dtype=dt, device=DEV)
    l[:, ::2] = -0.0
    ids, w = _check(l, 6, scoring)
    assert torch.equal(ids.cpu(), torch.arange(6, dtype=torch.int32).expand(5, 6))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,tg,k", [(16, 2, 1, 4), (24, 3, 2, 8), (64, 8, 4, 6), (256, 8, 4, 8),
                                           (160, 8, 3, 6), (12, 12, 5, 5), (1024, 32, 4, 16),
                                           (96, 4, 4, 8), (100, 5, 2, 30)])
def test_groups(E, groups, tg, k, scoring):
    l, g = _logits(77, E, F, E + groups)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV) if scoring == "sigmoid" else None
    _check(l, k, scoring, bias=bias, groups=groups, topk_groups=tg, scale=2.5)
    _check(l, k, scoring, groups=groups, topk_groups=tg, renorm=False)


@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_masks(scoring, dt, groups):
    l, g = _logits(12, 48, dt, 8)
    low = torch.finfo(dt).min
    l[0] = NINF                       # nothing left
    l[1] = low                        # nothing left, masked with the lowest value
    l[2] = float("nan")
    l[3, 1:] = NINF                   # one expert left
    l[3, 0] = 2.0
    l[4, 10:] = low                   # fewer than k left
    l[5, 7] = float("inf")            # certain
    l[6, 3] = float("nan")            # one expert masked among others
    l[7] = NINF
    l[7, 40] = low
    l[7, 41] = -100.0                 # unlikely, but not masked
    l[8, :24] = low                   # whole groups masked
    bias = torch.randn(48, generator=g, device=DEV).abs() * 3 if scoring == "sigmoid" else None
    tg = 2 if groups > 1 else 1
    ids, w = _check(l, 8, scoring, bias=bias, groups=groups, topk_groups=tg)
    assert torch.isfinite(w).all()
    for r in (0, 1, 2):
        assert torch.equal(ids[r].cpu(), torch.arange(8, dtype=torch.int32)) and not w[r].any()
    assert ids[3, 0] == 0 and float(w[3, 0]) == pytest.approx(1.0, abs=1e-6) and not w[3, 1:].any()
    assert ids[7, 0] == 41
    if bias is None:
        assert ids[5, 0] == 7
    assert 3 not in ids[6, w[6] > 0].tolist()
    if scoring == "softmax":
        assert float(w[5, 0]) == 1.0


def test_row_slices_and_no_rows():
    g = torch.Generator(device=DEV).manual_seed(4)
    wide = torch.randn(19, 75, generator=g, device=DEV)
    for off, n in ((0, 64), (3, 64), (8, 60)):
        l = wide[:, off:off + n]
        a = _check(l, 5, "sigmoid")
        b = mgg.select_experts(l.contiguous(), 5, scoring="sigmoid")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ids, w = mgg.select_experts(torch.empty(0, 16, device=DEV), 3)
    assert ids.shape == w.shape == (0, 3)
    d = mgg.select_experts_backward(w, torch.empty(0, 16, device=DEV), ids, w)
    assert d.shape == (0, 16)


# ---------------------------------------------------------------- gradient
@pytest.mark.parametrize("dt", [F, BF])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (33, 31, 4), (50, 64, 8), (9, 200, 6),
                                   (21, 256, 8), (3, 1000, 32)])
def test_gradient(T, E, k, scoring, renorm, dt):
    l, g = _logits(T, E, dt, T + 13 * E)
    scale = 2.5 if E > 8 else 1.0
    ids, w = mgg.select_experts(l, k, scoring=scoring, renormalize=renorm, scale=scale)
    gw = torch.randn(T, k, generator=g, device=DEV)
    st = mgg.new_status(DEV)
    d = mgg.select_experts_backward(gw, l, ids, w, scoring=scoring, renormalize=renorm,
                                    scale=scale, status=st)
    assert d.dtype == dt and mgg.read_status(st) == 0
    z = R.d(l).requires_grad_()
    i = ids.cpu().long()
    ref_w = R.weights_of(z, i, torch.ones(T, k, dtype=torch.bool), scoring, renorm, scale)
    (ref_w * R.d(gw)).sum().backward()
    # every term is w_j times a difference of g and a weighted mean of g
    mag = (R.d(w) * R.d(gw).abs()).sum(1, keepdim=True) + R.d(w).amax(1, keepdim=True) * R.d(gw).abs().amax(1, keepdim=True)
    R.within(d, z.grad, 2 * TOL * mag + R.rounding(dt, z.grad) * 1.01, "dlogits")
    # and against central differences of the float64 weights
    v = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).double()
    h = 1e-5

    def loss(zz):
        return float((R.weights_of(zz, i, torch.ones(T, k, dtype=torch.bool), scoring, renorm,
                                   scale) * R.d(gw)).sum())
    num = (loss(R.d(l) + h * v) - loss(R.d(l) - h * v)) / (2 * h)
    tol = float((2 * TOL * mag * v.abs()).sum() + (R.rounding(dt, z.grad) * v.abs()).sum()) + 1e-7
    assert abs(float((R.d(d) * v).sum()) - num) <= tol + 1e-6 * abs(num)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_gradient_with_masks(scoring, renorm):
    l, g = _logits(6, 40, F, 77)
    l[0] = NINF
    l[1, 3:] = torch.finfo(F).min
    l[2, ::2] = float("nan")
    ids, w = mgg.select_experts(l, 5, scoring=scoring, renormalize=renorm)
    gw = torch.randn(6, 5, generator=g, device=DEV)
    gw[0] = float("nan")               # nothing was chosen there: takes no part
    d = mgg.select_experts_backward(gw, l, ids, w, scoring=scoring, renormalize=renorm)
    assert torch.isfinite(d).all() and not d[0].any() and not d[1, 3:].any() and not d[2, ::2].any()
    z = torch.where(l > torch.finfo(F).min, l, torch.full_like(l, NINF)).cpu().double()[1:]
    z.requires_grad_()
    live = (w[1:] > 0).cpu()
    ref = R.weights_of(z, ids[1:].cpu().long(), live, scoring, renorm, 1.0)
    (ref * R.d(gw[1:])).sum().backward()
    R.within(d[1:], z.grad.nan_to_num(0.0), 4 * TOL * 10, "dlogits")


def test_gradient_bad_ids_and_repeats():
    l, g = _logits(4, 20, F, 5)
    ids, w = mgg.select_experts(l, 3, scoring="sigmoid", renormalize=False)
    gw = torch.randn(4, 3, generator=g, device=DEV)
    bad = ids.clone()
    bad[1, 1], bad[2, 0] = 20, -1
    st = mgg.new_status(DEV)
    d = mgg.select_experts_backward(gw, l, bad, w, scoring="sigmoid", renormalize=False, status=st)
    from variable_size_expert_gb300 import _lib as L
    assert mgg.read_status(st) == L.MGG_DEV_BAD_EXPERT_ID
    good = mgg.select_experts_backward(gw, l, ids, w, scoring="sigmoid", renormalize=False)
    assert torch.equal(d[0], good[0]) and torch.equal(d[3], good[3])
    assert int((d[1] != 0).sum()) == 2 and int((d[2] != 0).sum()) == 2
    same = ids.clone()
    same[:] = 4                        # equal ids add up
    d = mgg.select_experts_backward(gw, l, same, w, scoring="sigmoid", renormalize=False)
    s = torch.sigmoid(l[:, 4]).cpu().double()
    R.within(d[:, 4], (R.d(w) * R.d(gw)).sum(1) * (1 - s), 16 * TOL, "repeats")
    assert int((d != 0).sum()) <= 4


def test_router_feeds_moe():
    """The differentiable choice in front of the fused layer: gradients reach
    the logits through the routing weights."""
    g = torch.Generator(device=DEV).manual_seed(9)
    T, E, K, N = 48, 8, 64, 72
    x = torch.randn(T, K, generator=g, device=DEV)
    W = torch.randn(E, N, K, generator=g, device=DEV) / 8
    l = torch.randn(T, E, generator=g, device=DEV).requires_grad_()
    ids, w = mgg.router(l, 2, scoring="sigmoid", scale=1.5)
    assert not ids.requires_grad
    y = mgg.moe(x, W, ids, w)
    dy = torch.randn(T, N, generator=g, device=DEV)
    (y * dy).sum().backward()
    z = R.d(l).requires_grad_()
    rw = R.weights_of(z, ids.cpu().long(), torch.ones(T, 2, dtype=torch.bool), "sigmoid", True, 1.5)
    per = torch.einsum("tn,enk,tk->te", R.d(dy), R.d(W), R.d(x)).gather(1, ids.cpu().long())
    (rw * per).sum().backward()
    err = (R.d(l.grad) - z.grad).norm() / z.grad.norm()
    assert err <= 1e-5, err


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,tg,k", [(128, 8, 4, 8), (256, 8, 2, 16), (256, 32, 16, 8), (512, 16, 8, 12),
                                           (192, 8, 4, 8)])
def test_groups_with_masks(E, groups, tg, k, scoring):
    """Kept groups with fewer than k experts left: the row fills up from all
    experts, lowest first, with weight 0; ties across and within groups."""
    l, g = _logits(40, E, F, E + k, coarse=True)
    gs = E // groups
    low = torch.finfo(F).min
    l[0] = NINF
    l[1, 3:] = low                                     # three experts left
    l[2] = NINF
    l[2, E - 2:] = 1.0                                 # two, at the end
    l[3, gs:] = float("nan")                           # one group left
    for r in range(4, 20):                             # a random few left
        keep = torch.randperm(E, generator=torch.Generator().manual_seed(r))[:r - 3]
        row = torch.full((E,), low, device=DEV)
        row[keep.to(DEV)] = l[r, keep.to(DEV)]
        l[r] = row
    ids, w = _check(l, k, scoring, groups=groups, topk_groups=tg)
    if scoring == "softmax":
        rid = R.select(l, k, scoring, None, groups, tg, True, 1.0)[0]
        assert torch.equal(ids.cpu().long(), rid)
    assert torch.equal(ids[0].cpu(), torch.arange(k, dtype=torch.int32)) and not w[0].any()
