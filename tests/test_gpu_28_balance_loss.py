"""Balance loss of a gate, counts and gradient, against float64: one token to
many, expert counts that divide by nothing, both scorings and types, padded
sequences, masked experts, strided logits, bad ids, T = 0."""
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


def _inputs(T, E, k, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = (1.5 * torch.randn(T, E, generator=g, device=DEV)
              + torch.randn(E, generator=g, device=DEV)).to(dtype)
    ids = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].int().contiguous()
    return logits, ids, g


def _check(logits, ids, scoring, mask=None, sequences=1, want_status=0):
    st = mgg.new_status(DEV)
    loss, counts, slope = mgg.balance_loss_forward(logits, ids, scoring, mask, sequences, status=st)
    assert mgg.read_status(st) == want_status
    rl, rc, rs = S.balance(logits, ids, scoring, mask, sequences)
    assert counts.dtype == torch.int32 and torch.equal(counts.cpu().long(), rc)
    R.within(slope, rs, 8 * R.U * rs.abs(), "slope")
    # a sum of positive terms: each relative error, and the longest run of one sum
    T = logits.shape[0]
    rel = S.p_error(logits) + (R.DEPTH + T / 16) * R.U + 16 * R.U
    R.within(loss, rl, rel * rl.abs() + 1e-38, "loss")
    dloss = torch.tensor(0.37, device=DEV)
    got = mgg.balance_loss_backward(dloss, logits, slope, scoring, mask)
    assert got.dtype == logits.dtype and got.is_contiguous()
    rd, tol = S.balance_grad(float(dloss), logits, R.d(slope), scoring, mask)
    R.within(got, rd, tol + 2 * R.U * rd.abs() + R.rounding(got.dtype, rd) * 1.01, "dlogits")
    return loss, counts, got


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (33, 8, 1), (64, 128, 8), (70, 251, 6), (200, 60, 4), (130, 1024, 8),
         (40, 1000, 32), (513, 256, 8), (4096, 64, 2), (1000, 16, 2), (300, 24, 3), (97, 513, 7), (5001, 40, 4)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_sizes(T, E, k, scoring):
    h = T + E + (scoring == "sigmoid")
    logits, ids, g = _inputs(T, E, k, (F, BF)[h % 2], h)
    mask = torch.rand(T, generator=g, device=DEV) < 0.7 if h % 3 else None
    _check(logits, ids, scoring, mask)


@pytest.mark.parametrize("sequences,length,E", [(2, 50, 16), (8, 1, 64), (5, 333, 40), (64, 7, 33), (300, 3, 8)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_sequences(sequences, length, E, scoring):
    T = sequences * length
    logits, ids, g = _inputs(T, E, 2, F, T)
    at = (length * torch.rand(sequences, generator=g, device=DEV)).long()
    at[0] = 0                      # a sequence with no token at all
    mask = (torch.arange(length, device=DEV)[None] < at[:, None]).flatten()
    _check(logits, ids, scoring, mask, sequences)
    _check(logits, ids, scoring, None, sequences)


# one cluster of blocks, two launches: either side of the limit, few blocks' sums to join
# and many, sequences that share a cluster and a number of them that does not, blocks
# without a token
@pytest.mark.parametrize("T,E,sequences", [(1024, 8, 1), (1032, 8, 1), (2048, 64, 1), (2056, 64, 1), (521, 251, 1),
                                           (523, 251, 1), (9, 1024, 1), (17, 1000, 1), (1032, 10, 2), (1032, 10, 4),
                                           (1032, 10, 8), (1032, 10, 3), (16, 600, 8), (20000, 11, 4), (1600, 129, 16)])
def test_blocks_clusters_and_launches(T, E, sequences):
    logits, ids, g = _inputs(T, E, 3, (F, BF)[T % 2], T + E)
    length = T // sequences
    at = (length * torch.rand(sequences, generator=g, device=DEV)).long()
    at[-1] = 0 if sequences > 1 else length // 3
    mask = (torch.arange(length, device=DEV)[None] < at[:, None]).flatten()
    for m in (None, mask):
        a = _check(logits, ids, "softmax", m, sequences)
        b = _check(logits, ids, "softmax", m, sequences)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    _check(logits, ids, "sigmoid", mask, sequences)
    ids[T // 3, 1], ids[T - 1, 2] = -(1 << 31), E
    _check(logits, ids, "softmax", None, sequences, want_status=L.MGG_DEV_BAD_EXPERT_ID)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F, BF])
def test_masked_experts_and_padding(scoring, dtype):
    logits, ids, g = _inputs(96, 24, 2, dtype, 5)
    low = torch.finfo(dtype).min
    for row, bad in enumerate((-math.inf, math.nan, low)):
        logits[row, 3:9] = bad
        logits[8 + row] = bad                     # a token with no expert left
    logits[5, 2] = math.inf
    logits[6, 2] = 300.0
    logits[7] = -300.0
    mask = torch.ones(96, dtype=torch.bool, device=DEV)
    mask[40:] = False
    logits[50] = math.nan                         # what a padded token holds does not matter
    logits[51] = math.inf
    ids[52] = 1 << 20
    _, _, got = _check(logits, ids, scoring, mask)
    assert torch.equal(got[40:], torch.zeros_like(got[40:]))
    assert torch.isfinite(got.float()).all()


def test_even_load_is_one():
    T, E, k = 64, 16, 2
    logits = torch.zeros(T, E, device=DEV)
    ids = (torch.arange(T * k, device=DEV) % E).view(T, k).int()
    loss, counts, _ = mgg.balance_loss_forward(logits, ids)
    assert loss.item() == 1.0 and (counts == T * k // E).all()


def test_bad_ids_are_reported_and_not_counted():
    logits, ids, _ = _inputs(50, 12, 3, F, 1)
    ids[4, 1], ids[9, 0] = -1, 12
    _check(logits, ids, "softmax", want_status=L.MGG_DEV_BAD_EXPERT_ID)


def test_no_token_counts_and_no_tokens():
    logits, ids, _ = _inputs(10, 12, 3, F, 1)
    off = torch.zeros(10, dtype=torch.bool, device=DEV)
    loss, counts, slope = mgg.balance_loss_forward(logits, ids, mask=off)
    assert loss.item() == 0 and not counts.any() and not slope.any()
    loss, counts, slope = mgg.balance_loss_forward(logits[:0], ids[:0], sequences=4)
    assert loss.item() == 0 and counts.shape == slope.shape == (4, 12) and not counts.any() and not slope.any()
    assert mgg.balance_loss_backward(loss, logits[:0], slope).shape == (0, 12)


def test_strided_and_unaligned_logits():
    wide = torch.randn(70, 100, device=DEV)
    ids = torch.randint(0, 64, (70, 2), device=DEV, dtype=torch.int32)
    for at in (0, 1, 4):
        _check(wide[:, at:at + 64], ids, "softmax")
        _check(wide.bfloat16()[:, at:at + 64], ids, "sigmoid")


def test_same_bits_again_and_on_a_side_stream():
    logits, ids, _ = _inputs(3000, 96, 4, F, 2)
    a = mgg.balance_loss_forward(logits, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = mgg.balance_loss_forward(logits, ids)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences():
    logits, ids, _ = _inputs(24, 10, 2, F, 3)
    z = logits.clone().requires_grad_()
    loss, counts = mgg.balance_loss(z, ids, "sigmoid", sequences=2)
    (2.5 * loss).backward()
    # the loss as a function of the logits in float64, its counts held fixed
    e = 1e-5
    for t, j in ((0, 0), (3, 7), (23, 9), (12, 4)):
        up, down = (logits.double().cpu().clone() for _ in range(2))
        up[t, j] += e
        down[t, j] -= e
        slope = 2.5 * (S.balance(up, ids, "sigmoid", None, 2)[0] - S.balance(down, ids, "sigmoid", None, 2)[0]) / (2 * e)
        # differences: third derivatives of a few 1e-2 times e^2, cancellation 1e-16 / e
        assert abs(z.grad[t, j].item() - slope) <= 1e-8 + 1e-4 * abs(slope)
    assert not counts.requires_grad
