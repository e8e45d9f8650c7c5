"""The matrix units cut every sum that they add to off, always towards zero.  The
loss of few tokens adds runs of two blocks of the contraction up in f32, whatever
the contraction's length: a loss's error must not grow with it."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from tests import block_ref as R
from tests.test_gpu_29_linear_cross_entropy import _check, _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _lse64(x, W):
    z = torch.cat([x.double() @ w.double().t() for w in W.split(2048)], 1)
    return torch.logsumexp(z, 1), z.mean()


# 153 tiles of 128 rows leave no room for clusters, so that one block adds a logit up
# from end to end; few tiles, whose clusters share it out
@pytest.mark.parametrize("T,K,V", [(32, 16384, 19500), (32, 8192, 19500), (16, 16384, 19500), (17, 4096, 19500),
                                   (32, 16384, 2048)])
def test_no_bias_grows_with_the_contraction(T, K, V):
    g = torch.Generator(device=DEV).manual_seed(K + T)
    # positive terms: what is cut off is one-sided and adds up.  Logits of about 64.
    x = (0.5 + torch.rand(T, K, generator=g, device=DEV)).bfloat16()
    W = ((0.5 + torch.rand(V, K, generator=g, device=DEV)) * (64.0 / K)).bfloat16()
    t = torch.zeros(T, dtype=torch.long, device=DEV)
    _, lse, _ = mgg.linear_cross_entropy_forward(x, W, t)
    ref, z = _lse64(x, W)
    # a run is 128 terms, eight products of 16, of which each may cut off less than a
    # unit in the last place (2^-23) of the run's sum so far; the runs' sums are added
    # with roundings to nearest, which the mean over tokens and vocabulary takes out;
    # then lse's own: its sum, ln 2's product, a few of 1 + log2 of the sum
    tol = 8 * 2.0 ** -23 * z + 3 * R.U * ref.mean() + 8 * R.U
    err = (lse.double() - ref).mean()
    assert err.abs() <= tol, (float(err), float(tol))


# more runs than accumulators (16 up to 16 tokens, else 8), whole rounds of them and not,
# a last run of one block; blocks of their own and clusters
@pytest.mark.parametrize("T,K,V", [(17, 1032, 20001), (32, 1024 + 64, 20001), (20, 2056, 19600), (32, 2048, 19500),
                                   (16, 2056, 20001), (9, 2048 + 128, 19500), (1, 4104, 19500), (32, 8200, 700),
                                   (70, 8200, 300), (16, 16392, 600)])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_accumulators_in_turn(T, K, V, reduction):
    x, W, t, g = _inputs(T, K, V, T + K)
    a = _check(x, W, t, reduction, 1e-3, g)
    b = mgg.linear_cross_entropy_forward(x, W, t, reduction=reduction, z_loss=1e-3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
