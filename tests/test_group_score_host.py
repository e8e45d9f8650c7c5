"""The group score's values at the C ABI and the torch API, before the device
is touched."""
import os

import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import _lib as L, build

FAKE = 0x10000      # never dereferenced: the checks fail first


def test_values():
    import __graft_entry__ as g
    if not (os.path.exists(L.LIB_PATH) and os.path.exists(build.HOST)):
        g.build()
    lib = L.load()

    def select(scoring, T=0):
        return lib.mgg_select_experts(FAKE, L.MGG_F32, 16, T, 16, 2, scoring, None, 4, 2, 1, 1.0, FAKE, FAKE, None)
    for base in (L.MGG_SCORE_SOFTMAX, L.MGG_SCORE_SIGMOID):
        for group in (0, L.MGG_GROUP_BEST, L.MGG_GROUP_TWO_BEST):
            assert select(base | group) == L.MGG_OK
        assert select(base | L.MGG_GROUP_BEST | L.MGG_GROUP_TWO_BEST, T=4) == L.MGG_ERR_INVALID_ARG
        assert select(base | 0x400, T=4) == L.MGG_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="group_score"):
        mgg.select_experts(torch.zeros(4, 16), 2, groups=4, topk_groups=2, group_score="three best")
