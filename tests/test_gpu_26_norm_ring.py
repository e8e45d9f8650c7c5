"""Layer norm of many rows: the persistent kernels that keep rows on their way
through shared memory, with every pair of types, at both ends of every width of
thread group, aligned and shifted, with more rows per group than the ring has
slots; against float64."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32
TYPES = [(BF, BF, BF), (F, BF, F), (F, F, BF), (BF, F, F)]
# threads a row: 32 up to 512 columns, 64 to 1024, 128 to 2048, 256 to 4096, 512;
# rows that do not start on a piece's boundary count seven columns more
ALIGNED = [264, 512, 520, 1000, 1032, 2048, 2056, 4096, 4104, 8192]
SHIFTED = [267, 505, 507, 1001, 1017, 1019, 2041, 2043, 4089, 4091, 7163, 8185]
EPS = 1e-5


def _rows(K):
    """An odd number of rows, thirteen a group and more (the ring has six slots
    at most), and as many as the choice of the ring asks for."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    width = next(w for w in (512, 1024, 2048, 4096, 1 << 20) if K + (7 if K % 8 else 0) <= w)
    groups = max(1, 8192 // width)
    return (max(13 * sms * groups, 8 * sms * 8192 // K + 1) + 2) | 1


def _within(got, ref, tol, name):
    """As block_ref.within, on the GPU (these matrices are large)."""
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound, the first "
                           f"at {tuple(bad.nonzero()[0].tolist())}")


def _d(t):
    return None if t is None else t.double()


def _check(x, w, b, yt, g):
    y, mean, rstd = mgg.layer_norm_forward(x, w, b, eps=EPS, out_dtype=yt)
    ry, rm, rr = R.norm_forward(_d(x), _d(w), _d(b), EPS)
    ty, tm, tr = R.norm_forward_bounds(_d(x), _d(w), _d(b), EPS)
    _within(mean, rm, tm, "mean")
    _within(rstd, rr, tr, "rstd")
    _within(y, ry, ty + R.rounding(yt, ry) * 1.01, "y")
    del ry, ty
    dy = torch.randn(x.shape, generator=g, device=DEV).to(yt)
    dx, dw, db = mgg.layer_norm_backward(dy, x, w, mean, rstd, bias=b is not None)
    rx, rw, rb, tx, tw, tb = R.norm_backward(_d(dy), _d(x), _d(w), _d(mean), _d(rstd))
    _within(dx, rx, tx + R.rounding(dx.dtype, rx) * 1.01, "dx")
    _within(dw, rw, tw + R.rounding(dw.dtype, rw) * 1.01, "dweight")
    if b is not None:
        _within(db, rb, tb + R.rounding(db.dtype, rb) * 1.01, "dbias")


def _inputs(T, K, xt, wt, bias=True, ld=None):
    g = torch.Generator(device=DEV).manual_seed(T + K)
    x = (torch.randn(T, ld or K, generator=g, device=DEV) * 2 + 0.7).to(xt)[:, :K]
    w = (1 + 0.3 * torch.randn(K, generator=g, device=DEV)).to(wt)
    b = torch.randn(K, generator=g, device=DEV).to(wt) if bias else None
    return x, w, b, g


@pytest.mark.parametrize("K", ALIGNED + SHIFTED)
@pytest.mark.parametrize("xt,yt,wt", TYPES)
def test_every_width(K, xt, yt, wt):
    x, w, b, g = _inputs(_rows(K), K, xt, wt, bias=K % 3 != 0)
    _check(x, w, b, yt, g)


@pytest.mark.parametrize("K,pad", [(512, 8), (1000, 16), (4096, 8), (507, 8), (1001, 16), (8185, 24)])
@pytest.mark.parametrize("xt,yt,wt", TYPES[:2])
def test_rows_of_a_wider_matrix(K, pad, xt, yt, wt):
    """Slices whose rows are aligned, or share the residues of dense rows."""
    x, w, b, g = _inputs(_rows(K), K, xt, wt, ld=K + pad)
    assert not x.is_contiguous()
    _check(x, w, b, yt, g)


@pytest.mark.parametrize("xt,yt,wt", TYPES)
def test_parameters_off_their_boundary(xt, yt, wt):
    K = 1000
    x, _, _, g = _inputs(_rows(K), K, xt, wt)
    p = (1 + 0.3 * torch.randn(2, K + 1, generator=g, device=DEV)).to(wt)
    _check(x, p[0, 1:], p[1, 1:].clone(), yt, g)


@pytest.mark.parametrize("K", [512, 507, 2043, 8185])
@pytest.mark.parametrize("xt,yt", [(BF, BF), (F, BF)])
def test_neighbouring_rows(K, xt, yt):
    """A row of NaN or infinities leaves the rows beside it alone, whose ends
    share its 16-byte pieces."""
    T = _rows(K)
    x, w, b, g = _inputs(T, K, xt, F)
    y, mean, rstd = mgg.layer_norm_forward(x, w, b, out_dtype=yt)
    dy = torch.randn(T, K, generator=g, device=DEV).to(yt)
    dx, _, _ = mgg.layer_norm_backward(dy, x, w, mean, rstd)
    hit = torch.arange(3, T, 5, device=DEV)
    x2, dy2 = x.clone(), dy.clone()
    x2[hit] = float("nan")
    x2[hit[::2]] = float("inf")
    y2, mean2, rstd2 = mgg.layer_norm_forward(x2, w, b, out_dtype=yt)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[hit] = False
    for a, c in ((y, y2), (mean, mean2), (rstd, rstd2)):
        assert torch.equal(a[keep], c[keep])
    assert torch.isnan(y2[~keep]).all()
    dy2[hit] = float("nan")
    dx2, _, _ = mgg.layer_norm_backward(dy2, x2, w, mean2, rstd2)
    assert torch.equal(dx[keep], dx2[keep]) and torch.isnan(dx2[~keep]).all()
