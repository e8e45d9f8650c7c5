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
