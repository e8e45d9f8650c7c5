"""Cross entropy over a vocabulary and its gradients against float64: one token
to many tiles, vocabularies that divide by nothing, several pieces, ignored and
bad targets, every reduction, penalties, strided rows, T = 0."""
import math

import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R
from tests import step_ref as S
from variable_size_expert_gb300 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32


def _inputs(T, K, V, seed, ignored=0.2, scale=1.0, dtype=torch.int64):
    g = torch.Generator(device=DEV).manual_seed(seed)
    W = (scale * torch.randn(V, K, generator=g, device=DEV) / K ** 0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device=DEV)
    x = (torch.randn(T, K, generator=g, device=DEV)
         + 6 * torch.rand(T, 1, generator=g, device=DEV) * W[t].float()).to(BF)
    off = torch.rand(T, generator=g, device=DEV) < ignored
    return x, W, torch.where(off, S.IGNORE, t).to(dtype), g


def _check(x, W, t, reduction="mean", z_loss=0.0, g=None, want_status=0, sharp=False, **kw):
    st = mgg.new_status(DEV)
    loss, lse, weight = mgg.linear_cross_entropy_forward(x, W, t, reduction=reduction, z_loss=z_loss, status=st, **kw)
    assert mgg.read_status(st) == want_status and loss.dtype == lse.dtype == weight.dtype == F
    losses, rl, tol, t_lse = S.vocab(x, W, t, z_loss)
    T, V = x.shape[0], W.shape[0]
    n = int(((t >= 0) & (t < V)).sum())
    R.within(lse, rl, t_lse, "lse")
    assert abs(weight.item() - (1 / max(n, 1) if reduction == "mean" else 1.0)) <= 2 * R.U * weight.item()
    if reduction == "none":
        R.within(loss, losses, tol, "losses")
        dloss = torch.randn(T, generator=g, device=DEV)
        share = R.d(dloss)
    else:
        w = 1 / max(n, 1) if reduction == "mean" else 1.0
        runs = (R.DEPTH + T / 8192) * R.U
        R.within(loss, losses.sum() * w, (tol.sum() + runs * losses.abs().sum()) * w + 1e-38, "loss")
        dloss = torch.tensor(1.7, device=DEV)
        share = float(dloss) * w
    dx, dW = mgg.linear_cross_entropy_backward(dloss, x, W, t, lse, weight, z_loss=z_loss, status=st, **kw)
    assert mgg.read_status(st) == want_status and dx.dtype == dW.dtype == BF
    rx, rW, tx, tW = S.vocab_grads(share, x, W, t, lse, z_loss)
    R.within(dx, rx, tx + R.rounding(BF, rx) * 1.02, "dx")
    R.within(dW, rW, tW + R.rounding(BF, rW) * 1.02, "dW")
    # two roundings of at most 2^-8, uniformly spread: root mean square 2.4e-3.  (Not
    # of logits near 10^4: f32 numbers lie 2^-10 apart there, so that exp(z - lse) is
    # off by 1e-3 of itself, and where it is close to 1 the difference to 1, which
    # then is the gradient, by any share: only the bounds above, which count it, hold.)
    if sharp:
        return loss, lse, dx, dW
    for got, ref in ((dx, rx), (dW, rW)):
        if ref.numel() > 64 and ref.norm() > 0:
            assert (R.d(got) - ref).norm() <= 3e-3 * ref.norm()
    return loss, lse, dx, dW


SIZES = [(1, 8, 1), (1, 64, 7), (2, 128, 16), (3, 72, 33), (16, 512, 1000), (17, 200, 130), (33, 1024, 257),
         (64, 264, 256), (100, 136, 5003), (129, 64, 8), (255, 320, 515), (256, 256, 256), (257, 192, 2048),
         (600, 64, 2305), (513, 1032, 513)]


@pytest.mark.parametrize("T,K,V", SIZES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_forward_backward(T, K, V, reduction):
    h = T + K + V + len(reduction)
    x, W, t, g = _inputs(T, K, V, h, dtype=(torch.int64, torch.int32)[h % 2])
    _check(x, W, t, reduction, (0.0, 1e-3)[h % 2], g)


# few tiles: groups of 32 tokens, the contraction shared out in a cluster of two, four or
# eight (parts of one length and not; d in f32, in two parts, in one); and sizes of the
# same kind with too many tiles for that
@pytest.mark.parametrize("T,K,V", [(3, 1040, 700), (5, 4096, 300), (31, 2056, 5000), (32, 1032, 128), (100, 1224, 1111),
                                   (129, 576, 130), (640, 520, 1700), (1025, 2600, 7), (32, 520, 20001), (33, 136, 20001),
                                   (100, 72, 9999), (129, 64, 9000), (300, 264, 5003), (1300, 200, 1030),
                                   (4000, 72, 400)])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_few_tiles(T, K, V, reduction):
    x, W, t, g = _inputs(T, K, V, T + K, dtype=(torch.int64, torch.int32)[T % 2])
    a = _check(x, W, t, reduction, 1e-3, g)
    loss, lse, w = mgg.linear_cross_entropy_forward(x, W, t, reduction=reduction, z_loss=1e-3)
    assert torch.equal(loss, a[0]) and torch.equal(lse, a[1])


# pieces of the vocabulary: two to eight, the last one narrow, one slice of dx in it
# or several; few tokens (d in two parts) and many
@pytest.mark.parametrize("T,K,V,piece,reduction", [(300, 64, 1000, 256, "mean"), (1, 40, 2000, 1024, "none"),
                                                   (128, 72, 515, 64, "sum"), (129, 200, 4097, 2048, "mean"),
                                                   (700, 136, 3000, 1500, "none")])
def test_pieces(T, K, V, piece, reduction, monkeypatch):
    monkeypatch.setenv("MGG_VOCAB_PIECE", str(piece))
    x, W, t, g = _inputs(T, K, V, T)
    _check(x, W, t, reduction, 1e-4, g)


# up to 4 tokens the gradients leave one kernel: columns that do not fill its blocks,
# rows that do not fill its chunks, several chunks a block; 5 tokens, the first beyond
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("K,V,reduction", [(1032, 17, "none"), (8, 20000, "mean"), (264, 1999, "sum"),
                                           (2056, 16384, "mean")])
def test_very_few_tokens(T, K, V, reduction, monkeypatch):
    monkeypatch.setenv("MGG_VOCAB_PIECE", "640")
    x, W, t, g = _inputs(T, K, V, T + K, ignored=0.1)
    wide = torch.full((T, K + 16), math.nan, dtype=BF, device=DEV)
    wide[:, 8:-8] = x
    loss, lse, dx, dW = _check(wide[:, 8:-8], W, t, reduction, 1e-3, g)
    if reduction != "none":
        w = 1 / max(int((t >= 0).sum()), 1) if reduction == "mean" else 1.0
        args = (torch.tensor(1.7, device=DEV), x, W, t, lse, torch.tensor(w, device=DEV))
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)
        ax, none = mgg.linear_cross_entropy_backward(*args, z_loss=1e-3, need_dW=False, workspace=ws)
        none2, aW = mgg.linear_cross_entropy_backward(*args, z_loss=1e-3, need_dx=False, workspace=ws)
        assert none is None and none2 is None and torch.equal(dx, ax) and torch.equal(dW, aW)


def test_pieces_of_the_default_size():
    x, W, t, g = _inputs(70000, 8, 2049, 1)
    _check(x, W, t, "mean", 0.0, g)


# rows off 64-byte lines: x is copied from 256 tokens on, W's pieces from 2048 on
@pytest.mark.parametrize("T,K,V", [(256, 72, 500), (2050, 40, 700), (2300, 264, 900)])
def test_rows_off_lines(T, K, V, monkeypatch):
    x, W, t, g = _inputs(T, K, V, T)
    _check(x, W, t, "mean", 0.0, g)
    monkeypatch.setenv("MGG_VOCAB_PIECE", "320")
    _check(x, W, t, "none", 0.0, g)
    wide = torch.zeros(T, K + 8, dtype=BF, device=DEV)
    wide[:, 8:] = x
    _check(wide[:, 8:], W, t, "sum", 0.0, g)


@pytest.mark.parametrize("scale", [0.0, 40.0, 1000.0])
def test_flat_and_sharp_distributions(scale):
    x, W, t, g = _inputs(70, 64, 700, 3, scale=scale)
    if scale == 1000.0:  # the targets' logits decide: hold only that all is finite
        loss, lse, w = mgg.linear_cross_entropy_forward(x, W, t)
        dx, dW = mgg.linear_cross_entropy_backward(loss * 0 + 1, x, W, t, lse, w)
        assert torch.isfinite(loss) and torch.isfinite(lse).all() and torch.isfinite(dx).all() and torch.isfinite(dW).all()
        return
    _check(x, W, t, "mean", 0.0, g, sharp=scale > 1)


def test_ignored_tokens_are_left_out_whatever_they_hold():
    x, W, t, _ = _inputs(300, 64, 500, 4)
    off = t < 0
    a = _check(x, W, t)
    y = x.clone()
    y[off] = math.nan
    loss, lse, w = mgg.linear_cross_entropy_forward(y, W, t)
    dx, dW = mgg.linear_cross_entropy_backward(torch.tensor(1.7, device=DEV), y, W, t, lse, w)
    assert torch.equal(loss, a[0]) and torch.equal(dx[~off], a[2][~off])
    assert torch.equal(dx[off], torch.zeros_like(dx[off]))


def test_all_ignored():
    x, W, t, _ = _inputs(40, 64, 500, 5, ignored=2.0)
    for r in ("mean", "sum"):
        loss, lse, dx, dW = _check(x, W, t, r)
        assert loss.item() == 0 and not dx.any() and not dW.any()


def test_bad_targets_do_not_count_and_are_reported():
    for dtype in (torch.int64, torch.int32):
        x, W, t, g = _inputs(80, 64, 300, 6, dtype=dtype)
        t[3], t[70] = 300, -1
        if dtype == torch.int64:
            t[9] = 1 << 40
        _check(x, W, t, "mean", 0.0, g, want_status=L.MGG_DEV_BAD_TARGET)
    # another ignore_index
    t = torch.where((t < 0) | (t >= 300), 7, t)
    loss, _, w = mgg.linear_cross_entropy_forward(x, W, t, ignore_index=7)
    assert abs(1 / w.item() - int((t != 7).sum())) < 1e-3


def test_no_tokens():
    _, W, _, _ = _inputs(1, 64, 300, 6)
    x, t = torch.zeros(0, 64, dtype=BF, device=DEV), torch.zeros(0, dtype=torch.long, device=DEV)
    for r in ("mean", "sum", "none"):
        loss, lse, w = mgg.linear_cross_entropy_forward(x, W, t, reduction=r)
        assert w.item() == 1 and lse.shape == (0,) and float(loss.sum()) == 0
        dx, dW = mgg.linear_cross_entropy_backward(torch.ones((), device=DEV), x, W, t, lse, w)
        assert dx.shape == (0, 64) and not dW.any()


def test_strided_rows_one_output_and_workspace():
    x, W, t, _ = _inputs(130, 128, 700, 8)
    wide = torch.zeros(130, 200, dtype=BF, device=DEV)
    wide[:, 64:192] = x
    st = mgg.new_status(DEV)
    loss, lse, w = mgg.linear_cross_entropy_forward(x, W, t, status=st)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)
    got = mgg.linear_cross_entropy_forward(wide[:, 64:192], W, t, status=st, workspace=ws)
    assert torch.equal(loss, got[0]) and torch.equal(lse, got[1])
    one = torch.ones((), device=DEV)
    dx, dW = mgg.linear_cross_entropy_backward(one, x, W, t, lse, w)
    ax, none = mgg.linear_cross_entropy_backward(one, wide[:, 64:192], W, t, lse, w, need_dW=False, workspace=ws)
    none2, aW = mgg.linear_cross_entropy_backward(one, x, W, t, lse, w, need_dx=False)
    assert none is None and none2 is None and torch.equal(dx, ax) and torch.equal(dW, aW)
    assert mgg.linear_cross_entropy_backward(one, x, W, t, lse, w, need_dx=False, need_dW=False) == (None, None)


def test_autograd_and_differences():
    T, K, V = 20, 16, 50
    x, W, t, _ = _inputs(T, K, V, 9)
    xr, Wr = x.clone().requires_grad_(), W.clone().requires_grad_()
    (3.0 * mgg.linear_cross_entropy(xr, Wr, t, z_loss=1e-2)).backward()
    n = int((t >= 0).sum())
    e = 1e-5
    for at in ((0, 3), (7, 0), (19, 15)):
        v = []
        for sign in (1, -1):
            xd = R.d(x)
            xd[at] += sign * e
            v.append(3.0 * S.vocab(xd, W, t, 1e-2)[0].sum() / n)
        slope = (v[0] - v[1]) / (2 * e)
        # two bf16 roundings of the terms and of the result, each at most 2^-8
        assert abs(xr.grad[at].item() - slope) <= 2 * R.BF * (abs(slope) + 3.0 / n * float(R.d(W).abs().max()) * 2)
    assert Wr.grad.shape == W.shape
    with pytest.raises(RuntimeError):
        torch.autograd.grad(mgg.linear_cross_entropy(xr, Wr, t), xr, create_graph=True)[0].sum().backward()


def test_captured_and_replayed():
    x, W, t, _ = _inputs(300, 64, 1000, 10)
    xs = x.clone()
    st = mgg.new_status(DEV)

    def both():
        loss, lse, w = mgg.linear_cross_entropy_forward(xs, W, t, status=st)
        return loss, *mgg.linear_cross_entropy_backward(torch.ones_like(loss), xs, W, t, lse, w, status=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in (11, 12):
        xs.copy_(_inputs(300, 64, 1000, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, both()))
    assert mgg.read_status(st) == 0
