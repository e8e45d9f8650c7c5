"""Operands on different GPUs are refused before anything else, by name.  The
tensors here only claim a device: they have no memory that could be read."""
import os

import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import _lib, build


class Claim(torch.Tensor):
    @staticmethod
    def __new__(cls, shape, dtype, device):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=device)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"{func} ran on a tensor without memory")


BF, F, I = torch.bfloat16, torch.float32, torch.int32
T, K, N, E, k = 4, 64, 24, 16, 2

CALLS = {
    "layer_norm_forward": (lambda x, weight, bias: mgg.layer_norm_forward(x, weight, bias),
                           dict(x=((T, K), F), weight=((K,), F), bias=((K,), F))),
    "layer_norm_backward": (lambda dy, x, weight, mean, rstd, workspace:
                            mgg.layer_norm_backward(dy, x, weight, mean, rstd, workspace=workspace),
                            dict(dy=((T, K), F), x=((T, K), F), weight=((K,), F), mean=((T,), F),
                                 rstd=((T,), F), workspace=((1 << 20,), torch.uint8))),
    "select_experts": (lambda logits, bias: mgg.select_experts(logits, k, bias=bias),
                       dict(logits=((T, E), F), bias=((E,), F))),
    "select_experts_backward": (lambda dtopk, logits, expert_ids, topk_weights, status:
                                mgg.select_experts_backward(dtopk, logits, expert_ids, topk_weights,
                                                            status=status),
                                dict(dtopk=((T, k), F), logits=((T, E), F), expert_ids=((T, k), I),
                                     topk_weights=((T, k), F), status=((1,), I))),
    "linear_forward": (lambda x, W, bias, residual, status, out:
                       mgg.linear_forward(x, W, bias, residual=residual, status=status, out=out),
                       dict(x=((T, K), BF), W=((N, K), BF), bias=((N,), F), residual=((T, N), F),
                            status=((1,), I), out=((T, N), BF))),
    "linear_backward": (lambda dy, x, W, pre, status, workspace:
                        mgg.linear_backward(dy, x, W, pre, "gelu", status=status, workspace=workspace),
                        dict(dy=((T, N), BF), x=((T, K), BF), W=((N, K), BF), pre=((T, N), BF),
                             status=((1,), I), workspace=((1 << 20,), torch.uint8))),
}
CASES = [(c, a) for c, (_, args) in CALLS.items() for a in list(args)[1:]]


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(build.HOST)):
        g.build()


@pytest.mark.parametrize("call,arg", CASES, ids=[f"{c}-{a}" for c, a in CASES])
@pytest.mark.parametrize("where", ["cuda:1", "cpu"])
def test_operand_elsewhere(call, arg, where):
    f, args = CALLS[call]
    ts = {n: Claim(s, d, where if n == arg else "cuda:0") for n, (s, d) in args.items()}
    with pytest.raises(ValueError, match=f"^{arg} must be on the first argument's device"):
        f(**ts)
