"""Dense products with their epilogue, forward and backward, against float64:
one token to several tiles, widths that divide by nothing, every activation,
bias and residual types, slices, in-place residual, T = 0."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "silu", "gelu"]
# |act'| is at most 1.13 (GELU, SiLU), the activations add a few U of the value
SLOPE = 1.13


def _inputs(T, K, N, seed, bias=None, residual=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    W = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).to(BF)
    b = torch.randn(N, generator=g, device=DEV).to(bias) if bias else None
    r = torch.randn(T, N, generator=g, device=DEV).to(residual) if residual else None
    return x, W, b, r, g


def _check_forward(x, W, b, r, act, out_dtype, save_pre=True):
    st = mgg.new_status(DEV)
    got = mgg.linear_forward(x, W, b, activation=act, residual=r, out_dtype=out_dtype,
                             save_pre=save_pre, status=st)
    out, pre = got if save_pre else (got, None)
    assert mgg.read_status(st) == 0
    z = R.d(x) @ R.d(W).t()
    tz = R.dot_bound(R.d(x), R.d(W))
    if b is not None:
        z = z + R.d(b)
    tz = tz + 2 * R.U * z.abs()
    ref = R.act(z, act)
    tol = SLOPE * tz + 16 * R.U * z.abs()
    if r is not None:
        ref = ref + R.d(r)
        tol = tol + 2 * R.U * (ref.abs() + R.d(r).abs())
    R.within(out, ref, tol + R.rounding(out.dtype, ref) * 1.01, "out")
    if save_pre:
        assert pre.dtype == BF
        R.within(pre, z, tz + R.rounding(BF, z) * 1.01, "pre")
    return out, pre


def _check_backward(dy, x, W, pre, act, bias_dtype):
    st = mgg.new_status(DEV)
    dx, dW, db = mgg.linear_backward(dy, x, W, pre=pre, activation=act, bias_dtype=bias_dtype,
                                     status=st)
    assert mgg.read_status(st) == 0 and dx.dtype == dW.dtype == BF
    dz = R.d(dy)
    if act != "none":
        dz = dz * R.slope(R.d(pre), act)
    # the products' operand is bf16(dz): half a unit in the last place of each
    # term (f32 arithmetic before it: 16 U), then the accumulation
    tdz = (R.BF * 1.01 + 16 * R.U) * dz.abs() + 16 * R.U * R.d(dy).abs()
    if act == "none" and dy.dtype == BF:
        tdz = torch.zeros_like(dz)
    rx, rW = dz @ R.d(W), dz.t() @ R.d(x)
    tx = tdz @ R.d(W).abs() + 1.01 * R.dot_bound(dz, R.d(W).t())
    tW = tdz.t() @ R.d(x).abs() + 1.01 * R.dot_bound(dz.t(), R.d(x).t())
    R.within(dx, rx, tx + R.rounding(BF, rx) * 1.02, "dx")
    R.within(dW, rW, tW + R.rounding(BF, rW) * 1.02, "dW")
    # these bounds add every rounding up: hold the whole to the roundings'
    # root mean square too (two of at most 2^-8, uniformly spread: 2.4e-3)
    for got, ref in ((dx, rx), (dW, rW)):
        if ref.numel() > 64 and ref.norm() > 0:
            assert (R.d(got) - ref).norm() <= 3e-3 * ref.norm()
    if bias_dtype is not None:
        rb = dz.sum(0)
        tb = (16 + 64 + x.shape[0] / 64) * R.U * (dz.abs() + R.d(dy).abs()).sum(0)
        R.within(db, rb, tb + R.rounding(bias_dtype, rb) * 1.01, "dbias")
    else:
        assert db is None
    return dx, dW, db


SIZES = [(1, 8, 1), (1, 64, 7), (2, 128, 16), (3, 72, 33), (16, 512, 40), (17, 200, 130),
         (33, 1024, 100), (64, 264, 256), (100, 136, 264), (129, 64, 8), (250, 320, 515),
         (256, 256, 256), (300, 192, 2048), (2047, 64, 24), (513, 1032, 513)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_forward_backward(T, K, N, act):
    h = T + K + N + ACTS.index(act)
    bias = (None, F, BF)[h % 3]
    res = (None, F, BF)[(h // 3) % 3]
    out = (BF, F)[h % 2]
    x, W, b, r, g = _inputs(T, K, N, h, bias, res)
    _, pre = _check_forward(x, W, b, r, act, out)
    dy = torch.randn(T, N, generator=g, device=DEV).to(out)
    _check_backward(dy, x, W, pre, act, bias)


@pytest.mark.parametrize("T,K,N,act,bias,res,out", [
    (2304, 128, 2312, "gelu", BF, F, BF),     # tiles of 256 x 256 with ragged edges
    (2050, 192, 2307, "silu", F, BF, BF),     # rows that end off 16-byte boundaries
    (1900, 64, 2560, "none", None, F, F),
    (2560, 72, 2049, "relu", None, None, F),
    (2120, 4096, 2200, "none", BF, None, BF),
])
def test_many_tiles(T, K, N, act, bias, res, out):
    x, W, b, r, g = _inputs(T, K, N, T, bias, res)
    _, pre = _check_forward(x, W, b, r, act, out)
    _check_forward(x, W, b, r, act, out, save_pre=False)
    dy = torch.randn(T, N, generator=g, device=DEV).to(out)
    _check_backward(dy, x, W, pre, act, bias)


@pytest.mark.parametrize("T,K,N", [(2100, 2312, 2056), (1500, 2048, 4104)])
def test_many_tiles_backward(T, K, N):
    """dx and dW both on 256 x 256 tiles, in one launch."""
    x, W, _, _, g = _inputs(T, K, N, 3)
    dy = torch.randn(T, N, generator=g, device=DEV).to(BF)
    _check_backward(dy, x, W, None, "none", F)


@pytest.mark.parametrize("K", [64, 320, 384, 512, 576, 1024, 4096])
def test_long_runs_of_tiles(K):
    """Thirteen tiles per CTA pair, over and over, with contractions shorter and
    longer than the ring of blocks: no wait may run out, and every pass gives
    the same bits, whichever of the copies and the products is ahead."""
    T, N = 8192, 8192
    x, W, b, _, g = _inputs(T, K, N, K, BF)
    st = mgg.new_status(DEV)
    ref = mgg.linear_forward(x, W, b, "gelu", status=st)
    dy = torch.randn(T, N, generator=g, device=DEV).to(BF)
    rdx, rdW, _ = mgg.linear_backward(dy, x, W, status=st)
    for _ in range(12):
        assert torch.equal(mgg.linear_forward(x, W, b, "gelu", status=st), ref)
        dx, dW, _ = mgg.linear_backward(dy, x, W, status=st)
        assert torch.equal(dx, rdx) and torch.equal(dW, rdW)
        mgg.linear_forward(x, W, status=st)
        mgg.linear_forward(x, W, out_dtype=F, status=st)
    assert mgg.read_status(st) == 0
    rows = torch.randint(0, T, (64,), generator=g, device=DEV)
    z = R.d(x[rows]) @ R.d(W).t() + R.d(b)
    tol = SLOPE * R.dot_bound(R.d(x[rows]), R.d(W)) + 16 * R.U * z.abs()
    want = R.act(z, "gelu")
    R.within(ref[rows], want, tol + R.rounding(BF, want) * 1.01, "rows")


@pytest.mark.parametrize("T", [40, 2400])
def test_slices_and_in_place_residual(T):
    K, N = 128, 2304 if T > 2000 else 72
    g = torch.Generator(device=DEV).manual_seed(T)
    wide = torch.randn(T, K + 24, generator=g, device=DEV).to(BF)
    x = wide[:, 8:8 + K]
    W = (torch.randn(N, K, generator=g, device=DEV) / 12).to(BF)
    rw = torch.randn(T, N + 5, generator=g, device=DEV)
    r = rw[:, 2:2 + N]
    out, _ = _check_forward(x, W, None, r, "silu", F)
    acc = r.contiguous()
    got = mgg.linear_forward(x, W, activation="silu", residual=acc, out=acc)
    assert got is acc and torch.equal(acc, out)
    dyw = torch.randn(T, N + 8, generator=g, device=DEV).to(BF)
    for off in (8, 3):                 # readable by the copy engine as it lies, and not
        _check_backward(dyw[:, off:off + N], x, W, None, "none", F)


def test_bits_repeat():
    x, W, b, r, g = _inputs(96, 2048, 512, 1, F, F)
    dy = torch.randn(96, 512, generator=g, device=DEV).to(BF)
    a = [mgg.linear_forward(x, W, b, "gelu", r, F) for _ in range(2)]
    assert torch.equal(a[0], a[1])
    a = [mgg.linear_backward(dy, x, W, bias_dtype=F) for _ in range(2)]
    assert all(torch.equal(i, j) for i, j in zip(*a))


def test_partial_gradients():
    x, W, _, _, g = _inputs(50, 64, 24, 4)
    dy = torch.randn(50, 24, generator=g, device=DEV)
    dx, dW, db = mgg.linear_backward(dy, x, W, bias_dtype=F)
    a = mgg.linear_backward(dy, x, W, need_dW=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    a = mgg.linear_backward(dy, x, W, need_dx=False)
    assert torch.equal(a[1], dW) and a[0] is None
    a = mgg.linear_backward(dy, x, W, need_dx=False, need_dW=False, bias_dtype=F)
    assert torch.equal(a[2], db)


def test_no_rows():
    W = torch.ones(16, 24, device=DEV).to(BF)
    x = torch.empty(0, 24, device=DEV).to(BF)
    out, pre = mgg.linear_forward(x, W, activation="gelu", save_pre=True)
    assert out.shape == pre.shape == (0, 16)
    dx, dW, db = mgg.linear_backward(out, x, W, pre=pre, activation="gelu", bias_dtype=F)
    assert dx.shape == (0, 24) and dW.shape == (16, 24) and not dW.any() and not db.any()


def test_nonfinite_values_stay_in_their_rows():
    x, W, _, _, _ = _inputs(300, 128, 264, 6)
    clean = mgg.linear_forward(x, W)
    x[7, 3], x[290, 5] = float("nan"), float("inf")
    out = mgg.linear_forward(x, W)
    keep = torch.ones(300, dtype=torch.bool, device=DEV)
    keep[7] = keep[290] = False
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[7]).all()
    assert not torch.isfinite(out[290]).all()


def test_extreme_activations():
    """Far ends of the activations: no NaN from overflowing exponentials."""
    x = torch.zeros(4, 8, device=DEV).to(BF)
    x[0, 0], x[1, 0], x[2, 0] = 1.0, -1.0, 1e-3
    W = torch.zeros(8, 8, device=DEV).to(BF)
    W[0, 0], W[1, 0], W[2, 0] = 300.0, 3e38, 90.0
    for act in ACTS:
        out, pre = mgg.linear_forward(x, W, activation=act, out_dtype=F, save_pre=True)
        assert not torch.isnan(out).any()
        ref = R.act(R.d(x) @ R.d(W).t(), act)
        R.within(out, ref, 64 * R.U * ref.abs() + 1e-30, act)
        dy = torch.ones(4, 8, device=DEV)
        _, _, db = mgg.linear_backward(dy, x, W, pre=pre, activation=act, bias_dtype=F)
        assert torch.isfinite(db).all()


def test_gradient_against_differences():
    """Directional derivatives of the float64 layer at the kernel's inputs; the
    kernel's pre and dz are bf16 (2^-8 each, the slope's own change below 1)."""
    x, W, b, r, g = _inputs(12, 32, 24, 8, F, F)
    t = torch.randn(12, 24, generator=g, device=DEV)
    for act in ACTS[2:]:
        xs, Ws, bs, rs = (v.clone().requires_grad_() for v in (x, W, b, r))
        (mgg.linear(xs, Ws, bs, act, rs, F) * t).sum().backward()
        base = [R.d(x), R.d(W), R.d(b), R.d(r)]

        def loss(x_, W_, b_, r_):
            return float(((R.act(x_ @ W_.t() + b_, act) + r_) * R.d(t)).sum())
        for i, v0 in enumerate((xs, Ws, bs, rs)):
            v = torch.randn(v0.shape, generator=torch.Generator().manual_seed(i)).double()
            h = 1e-5
            hi, lo = list(base), list(base)
            hi[i], lo[i] = base[i] + h * v, base[i] - h * v
            num = (loss(*hi) - loss(*lo)) / (2 * h)
            got = float((R.d(v0.grad) * v).sum())
            # three roundings of 2^-8 per term, terms of independent sign
            tol = 4 * R.BF * float((R.d(v0.grad) * v).norm()) + 4 * R.BF * float(
                (R.d(t).norm() * (R.d(W).norm() if i == 0 else R.d(x).norm() if i == 1 else 1)
                 * v.norm() / v.numel() ** 0.5))
            assert abs(got - num) <= tol, (act, i, got, num, tol)


def test_other_stream_and_graph():
    x, W, b, r, g = _inputs(77, 256, 136, 2, F, BF)
    ref = mgg.linear_forward(x, W, b, "gelu", r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = mgg.linear_forward(x, W, b, "gelu", r)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)
    dy = torch.randn(77, 136, generator=g, device=DEV)
    want = mgg.linear_backward(dy, x, W, bias_dtype=F)
    st = mgg.new_status(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mgg.linear_forward(x, W, b, "gelu", r, status=st)
        got = mgg.linear_backward(dy, x, W, bias_dtype=F, status=st)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, ref) and all(torch.equal(i, j) for i, j in zip(got, want))
    assert mgg.read_status(st) == 0


@pytest.mark.parametrize("T,K,N,act,bias,res,out", [
    (2050, 8, 1000, "gelu", BF, F, BF),       # one block of the contraction: half of the accumulators
    (1000, 72, 640, "silu", F, BF, F),        # two blocks, the second ragged
    (1280, 2048, 96, "none", BF, F, F),       # narrow: pieces of the contraction
    (1219, 2168, 360, "relu", F, BF, BF),
    (2720, 5832, 224, "none", None, None, BF),
    (1024, 1096, 1200, "gelu", BF, BF, BF),   # wide single tiles, finished by every warp
    (1030, 1096, 1201, "silu", F, BF, BF),    # the same off 16-byte boundaries
    (1000, 2056, 1208, "none", F, F, F),
    (48, 4096, 2048, "gelu", BF, BF, BF),     # rows along the output's columns, in pieces
    (8, 5000, 3000, "silu", F, F, F),
])
def test_tile_choices(T, K, N, act, bias, res, out):
    x, W, b, r, g = _inputs(T, K, N, T + K, bias, res)
    _, pre = _check_forward(x, W, b, r, act, out)
    again, _ = _check_forward(x, W, b, r, act, out, save_pre=True)
    assert torch.equal(again, _check_forward(x, W, b, r, act, out, save_pre=False)[0])
    dy = torch.randn(T, N, generator=g, device=DEV).to(out)
    dx, dW, _ = _check_backward(dy, x, W, pre, act, bias)
    dx2, dW2, _ = _check_backward(dy, x, W, pre, act, bias)
    assert torch.equal(dx, dx2) and torch.equal(dW, dW2)
