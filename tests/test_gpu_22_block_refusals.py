"""Refusals of the torch API that need CUDA tensors: shapes, dtypes, strides,
and the library's own errors as MggError."""
import pytest
import torch

import variable_size_expert_gb300 as mgg
from variable_size_expert_gb300 import _lib as L

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def test_shapes_dtypes_strides():
    x, w, xb, Wb = _t(4, 64), _t(64), _t(4, 64, dtype=BF), _t(24, 64, dtype=BF)
    m, k2 = _t(4), _t(4, 2)
    ids = _t(4, 2, dtype=torch.int32)
    cases = [
        (ValueError, lambda: mgg.layer_norm_forward(x, _t(63))),
        (ValueError, lambda: mgg.layer_norm_forward(x[0], w)),
        (ValueError, lambda: mgg.layer_norm_forward(x.t(), _t(4))),
        (ValueError, lambda: mgg.layer_norm_forward(x[:1].expand(4, 64), w)),
        (TypeError, lambda: mgg.layer_norm_forward(x, w, w.bfloat16())),
        (TypeError, lambda: mgg.layer_norm_forward(x.half(), w)),
        (TypeError, lambda: mgg.layer_norm_forward(x, w, out_dtype=torch.float16)),
        (TypeError, lambda: mgg.layer_norm_forward(x, w, out_dtype="bf16")),
        (ValueError, lambda: mgg.layer_norm_forward(x, w, w.cpu())),
        (ValueError, lambda: mgg.layer_norm_backward(x[:, :32], x, w, m, m)),
        (ValueError, lambda: mgg.layer_norm_backward(x, x, w, m[:3], m)),
        (ValueError, lambda: mgg.layer_norm_backward(x, x, w, m.bfloat16(), m)),
        (ValueError, lambda: mgg.layer_norm_backward(_t(64, 4).t(), x, w, m, m)),
        (ValueError, lambda: mgg.select_experts(x, 2, bias=_t(63))),
        (ValueError, lambda: mgg.select_experts(x, 2, bias=w.bfloat16())),
        (ValueError, lambda: mgg.select_experts(x, -1)),
        (TypeError, lambda: mgg.select_experts(x.double(), 2)),
        (TypeError, lambda: mgg.select_experts(x, 2.5)),
        (ValueError, lambda: mgg.select_experts_backward(k2[:, :1], x, ids, k2)),
        (ValueError, lambda: mgg.select_experts_backward(k2, x, ids, k2.bfloat16())),
        (ValueError, lambda: mgg.linear_forward(xb, Wb[:, :32])),
        (ValueError, lambda: mgg.linear_forward(xb, Wb.t())),
        (TypeError, lambda: mgg.linear_forward(xb, Wb.float())),
        (ValueError, lambda: mgg.linear_forward(xb, Wb, _t(23))),
        (TypeError, lambda: mgg.linear_forward(xb, Wb, _t(24, dtype=torch.float16))),
        (ValueError, lambda: mgg.linear_forward(xb, Wb, residual=_t(4, 23))),
        (TypeError, lambda: mgg.linear_forward(xb, Wb, out_dtype=torch.float16)),
        (ValueError, lambda: mgg.linear_forward(xb, Wb, out=_t(3, 24))),
        (TypeError, lambda: mgg.linear_forward(xb, Wb, out=_t(4, 24), out_dtype=BF)),
        (ValueError, lambda: mgg.linear_forward(xb, Wb, status=_t(1))),
        (ValueError, lambda: mgg.linear_backward(_t(4, 23), xb, Wb)),
        (ValueError, lambda: mgg.linear_backward(_t(4, 24), xb, Wb, activation="gelu")),
        (TypeError, lambda: mgg.linear_backward(_t(4, 24), xb, Wb, pre=_t(4, 24), activation="gelu")),
    ]
    for i, (want, f) in enumerate(cases):
        with pytest.raises(want):
            f()
            pytest.fail(f"case {i} was not refused")


def test_library_errors():
    x, xb = _t(4, 64), _t(4, 60, dtype=BF)
    for code, f in (
            (L.MGG_ERR_INVALID_ARG, lambda: mgg.layer_norm_forward(x, _t(64), eps=-1.0)),
            (L.MGG_ERR_INVALID_ARG, lambda: mgg.select_experts(x, 65)),
            (L.MGG_ERR_INVALID_ARG, lambda: mgg.select_experts(x, 2, groups=5)),
            (L.MGG_ERR_INVALID_ARG, lambda: mgg.select_experts(x, 2, scale=0.0)),
            (L.MGG_ERR_ALIGNMENT, lambda: mgg.linear_forward(xb, _t(8, 60, dtype=BF))),
            (L.MGG_ERR_ALIGNMENT, lambda: mgg.linear_forward(_t(4, 72, dtype=BF)[:, 4:68],
                                                             _t(8, 64, dtype=BF)))):
        with pytest.raises(L.MggError) as e:
            f()
        assert e.value.status == code
