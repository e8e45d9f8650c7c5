"""Workspace sizes of the losses at the largest sides: finite up to the longest one
that the calls take, 0 beyond, where the call itself says what is wrong."""
import pytest

from tests.test_step_host import FAKE, lib  # noqa: F401
from variable_size_expert_gb300 import _lib as L

MOST = 1 << 30


@pytest.mark.parametrize("op", [L.MGG_OP_VOCAB_FORWARD, L.MGG_OP_VOCAB_BACKWARD])
@pytest.mark.parametrize("T", [1, 4, 5, 128, 200, 1000])
def test_vocabulary(lib, op, T):  # noqa: F811
    def ws(T, V, K):
        return lib.mgg_workspace_bytes(op, T, 0, 0, V, K, 0)
    # (one token's statistics; pieces that hold a token's share of 256 MB at least)
    assert 0 < ws(T, MOST, 8) < 1 << 47 and 0 < ws(T, 1000, MOST) < 1 << 50
    for side in (MOST + 8, (1 << 31) - 8, (1 << 31) - 1):
        assert ws(T, side, 8) == ws(T, 1000, side) == ws(side, 1000, 8) == 0
    call = lib.mgg_linear_cross_entropy
    for V in (MOST + 8, (1 << 31) - 1):
        assert call(FAKE, 8, FAKE, FAKE, 1, -100, T, 8, V, 2, 0.0, FAKE, FAKE, FAKE, FAKE, FAKE, 256,
                    None) == L.MGG_ERR_INVALID_ARG


def test_balance(lib):  # noqa: F811
    def ws(T, B, E):
        return lib.mgg_workspace_bytes(L.MGG_OP_BALANCE, T, B, E, 0, 0, 1)
    assert 0 < ws(MOST, 1, 1024) < 1 << 30 and ws(MOST, MOST, 8) >= MOST * 8 * 8
    assert ws(MOST + 8, 1, 8) == ws((1 << 31) - 1, 1, 8) == 0
