"""Layer norm forward and backward against float64: types, widths from 1 to
beyond the register path, ragged row counts, slices, constant rows, T = 0."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, BF, BF), (F, BF, F), (F, F, BF), (BF, F, F)]
# (T, K): one element, one row, around every change of path (16-byte pieces or
# not, 32 / 64 / 128 / 256 / 512 / 1024 threads a row, re-read rows)
SIZES = [(1, 1), (1, 8), (3, 7), (5, 512), (33, 513), (17, 520), (7, 1024), (130, 1032),
         (65, 2048), (9, 2056), (31, 2049), (11, 4096), (6, 4104), (5, 4097), (4, 7168), (3, 8192),
         (3, 8193), (2, 8200), (3, 16384), (2, 16383), (3, 16392), (2, 20001), (700, 72), (1031, 200)]


def _inputs(T, K, xt, wt, seed, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (torch.randn(T, K, generator=g, device=DEV) * 2 + 0.7).to(xt)
    w = (1 + 0.3 * torch.randn(K, generator=g, device=DEV)).to(wt)
    b = torch.randn(K, generator=g, device=DEV).to(wt) if bias else None
    return x, w, b, g


def _check_forward(x, w, b, yt, eps=1e-5):
    y, mean, rstd = mgg.layer_norm_forward(x, w, b, eps=eps, out_dtype=yt)
    assert y.dtype == yt and mean.dtype == rstd.dtype == F
    ry, rm, rr = R.norm_forward(R.d(x), R.d(w), R.d(b), eps)
    ty, tm, tr = R.norm_forward_bounds(R.d(x), R.d(w), R.d(b), eps)
    R.within(mean, rm, tm, "mean")
    R.within(rstd, rr, tr, "rstd")
    R.within(y, ry, ty + R.rounding(yt, ry) * 1.01, "y")
    return y, mean, rstd


def _check_backward(dy, x, w, mean, rstd, bias=True):
    dx, dw, db = mgg.layer_norm_backward(dy, x, w, mean, rstd, bias=bias)
    assert dx.dtype == x.dtype and dw.dtype == w.dtype and (db is None) == (not bias)
    rx, rw, rb, tx, tw, tb = R.norm_backward(R.d(dy), R.d(x), R.d(w), R.d(mean), R.d(rstd))
    R.within(dx, rx, tx + R.rounding(dx.dtype, rx) * 1.01, "dx")
    R.within(dw, rw, tw + R.rounding(dw.dtype, rw) * 1.01, "dweight")
    if bias:
        R.within(db, rb, tb + R.rounding(db.dtype, rb) * 1.01, "dbias")
    return dx, dw, db


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("xt,yt,wt", TYPES)
def test_forward_backward(T, K, xt, yt, wt):
    bias = (T + K) % 3 != 0
    x, w, b, g = _inputs(T, K, xt, wt, T * 31 + K, bias)
    _, mean, rstd = _check_forward(x, w, b, yt)
    dy = torch.randn(T, K, generator=g, device=DEV).to(yt)
    _check_backward(dy, x, w, mean, rstd, bias)


@pytest.mark.parametrize("K", [96, 2048, 7163])
def test_many_rows(K):
    """More rows than one pass of the persistent backward grid holds."""
    x, w, b, g = _inputs(5003, K, BF, F, K)
    _, mean, rstd = _check_forward(x, w, b, BF)
    _check_backward(torch.randn(5003, K, generator=g, device=DEV).to(BF), x, w, mean, rstd)


def test_backward_bits_repeat():
    x, w, _, g = _inputs(3001, 264, F, F, 5)
    dy = torch.randn(3001, 264, generator=g, device=DEV)
    _, mean, rstd = mgg.layer_norm_forward(x, w)
    a = mgg.layer_norm_backward(dy, x, w, mean, rstd)
    b = mgg.layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


@pytest.mark.parametrize("off,ld", [(0, 80), (8, 96), (3, 71), (1, 64 + 8)])
def test_row_slices(off, ld):
    """x as a slice of a wider matrix, aligned and not."""
    g = torch.Generator(device=DEV).manual_seed(ld)
    wide = torch.randn(37, ld, generator=g, device=DEV).to(BF)
    x = wide[:, off:off + 64]
    w, b = torch.rand(64, generator=g, device=DEV), torch.rand(64, generator=g, device=DEV)
    y, mean, rstd = _check_forward(x, w, b, BF)
    z, _, _ = mgg.layer_norm_forward(x.contiguous(), w, b)
    assert torch.equal(y, z)
    _check_backward(torch.randn(37, 64, generator=g, device=DEV).to(BF), x, w, mean, rstd)


def test_unaligned_parameters_and_outputs_of_odd_offset():
    g = torch.Generator(device=DEV).manual_seed(2)
    w = torch.rand(65, generator=g, device=DEV)[1:]
    x = torch.randn(9, 64, generator=g, device=DEV)
    _, mean, rstd = _check_forward(x, w, None, F)
    _check_backward(torch.randn(9, 64, generator=g, device=DEV), x, w, mean, rstd, bias=False)


def test_large_mean_constant_rows_and_nonfinite():
    w, b = torch.ones(256, device=DEV), torch.zeros(256, device=DEV)
    x = torch.randn(4, 256, device=DEV) + 1000.0
    x[1] = 3.0      # constant: y = b, rstd = eps^-1/2
    y, mean, rstd = _check_forward(x, w, b, F)
    assert torch.equal(y[1], b) and mean[1] == 3.0
    assert abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-3
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y, _, _ = mgg.layer_norm_forward(x, w, b)
    assert torch.isfinite(y[:2]).all() and torch.isnan(y[2]).all() and torch.isnan(y[3]).any()


def test_no_rows():
    w = torch.ones(40, device=DEV)
    x = torch.empty(0, 40, device=DEV)
    y, mean, rstd = mgg.layer_norm_forward(x, w, w)
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    dx, dw, db = mgg.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_gradient_against_differences():
    """<dx, v>, <dw, v>, <db, v> against central differences of the float64
    forward: step h leaves h^2 / 6 of the third derivative, below 1e-7 here."""
    x, w, b, g = _inputs(6, 40, F, F, 11)
    r = torch.randn(6, 40, generator=g, device=DEV)
    xs, ws, bs = (t.clone().requires_grad_() for t in (x, w, b))
    (mgg.layer_norm(xs, ws, bs) * r).sum().backward()

    def loss(x_, w_, b_):
        return float((R.norm_forward(x_, w_, b_, 1e-5)[0] * R.d(r)).sum())

    base = [R.d(x), R.d(w), R.d(b)]
    for i, t in enumerate((xs, ws, bs)):
        v = torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).double()
        h = 1e-4
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + h * v, base[i] - h * v
        num = (loss(*hi) - loss(*lo)) / (2 * h)
        got = float((R.d(t.grad) * v).sum())
        assert abs(got - num) <= 1e-4 * (1 + abs(num)), (i, got, num)


def test_other_stream_and_graph():
    x, w, b, _ = _inputs(64, 2048, BF, F, 3)
    ref, _, _ = mgg.layer_norm_forward(x, w, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _, _ = mgg.layer_norm_forward(x, w, b)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = mgg.layer_norm_forward(x, w, b)
        dx, dw, db = mgg.layer_norm_backward(y, x, w, mean, rstd)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref)
    a = mgg.layer_norm_backward(ref, x, w, mean, rstd)
    assert all(torch.equal(i, j) for i, j in zip(a, (dx, dw, db)))
