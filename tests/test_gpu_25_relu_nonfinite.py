"""ReLU products where something is infinite or NaN."""
import pytest
import torch

import variable_size_expert_gb300 as mgg

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F = torch.bfloat16, torch.float32

# (T, K, N): pieces of the contraction, single tiles, rows off 16-byte
# boundaries, tiles of 256 x 256
SIZES = [(16, 2048, 512), (300, 128, 264), (130, 64, 77), (2304, 128, 2312)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("out", [BF, F])
def test_forward_keeps_nan(T, K, N, out):
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    W = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).to(BF)
    b = torch.randn(N, generator=g, device=DEV)
    clean = mgg.linear_forward(x, W, b, "relu", out_dtype=out)
    assert (clean >= 0).all() and (clean == 0).any()
    x[3, 5] = float("nan")
    x[T - 1, 0] = float("inf")
    b[N - 2] = float("nan")
    got, pre = mgg.linear_forward(x, W, b, "relu", out_dtype=out, save_pre=True)
    assert torch.isnan(got[3]).all() and torch.isnan(got[:, N - 2]).all()
    rows = torch.ones(T, dtype=torch.bool, device=DEV)
    rows[3] = rows[T - 1] = False
    cols = torch.arange(N, device=DEV) != N - 2
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    z = pre[T - 1][cols].float()        # +inf, -inf (NaN where W is 0)
    want = torch.where(z < 0, torch.zeros_like(z), z)
    assert torch.equal(torch.isnan(got[T - 1][cols]), torch.isnan(want))
    assert torch.equal(got[T - 1][cols].float().nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("T,K,N", SIZES + [(40, 64, 36), (40, 64, 38)])
@pytest.mark.parametrize("dtype", [BF, F])
def test_backward_of_closed_units(T, K, N, dtype):
    """An infinite or NaN dy at a closed unit (pre <= 0) is no part of any
    gradient: the same bits as with dy = 0 there."""
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(T, K, generator=g, device=DEV).to(BF)
    W = (torch.randn(N, K, generator=g, device=DEV) / K ** 0.5).to(BF)
    pre = torch.randn(T, N, generator=g, device=DEV).to(BF)
    pre[:, 0] = -0.0
    dy = torch.randn(T, N, generator=g, device=DEV).to(dtype)
    wild = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV).to(dtype)
    wild = wild[torch.randint(0, 3, (T, N), generator=g, device=DEV)]
    closed = pre <= 0
    want = mgg.linear_backward(torch.where(closed, torch.zeros_like(dy), dy), x, W, pre, "relu", F)
    got = mgg.linear_backward(torch.where(closed, wild, dy), x, W, pre, "relu", F)
    assert all(torch.isfinite(t).all() for t in want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
