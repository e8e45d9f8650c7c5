"""torch-facing API of the layers around the experts in a MoE transformer
block: layer norm, the choice of the experts from the gate's logits, and
dense products with their epilogue (the gate, a shared expert, the residual
stream).

As in ops.py every step runs in libmgg.so's kernels on the current stream;
inputs are CUDA tensors.  Row inputs may be slices of wider matrices (their
last dimension contiguous); everything else is contiguous.

  layer_norm(x, weight, bias)              differentiable
  router(logits, k, ...)                   differentiable expert choice
  linear(x, W, bias, activation, residual) differentiable
plus the *_forward / *_backward calls under them.  The gradients have no
gradients of their own: asking for them (create_graph) is an error.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from .ops import _ids_i32, new_status

__all__ = [
    "layer_norm_forward", "layer_norm_backward", "layer_norm", "select_experts",
    "select_experts_backward", "router", "linear_forward", "linear_backward", "linear",
]

_SCORING = {"softmax": L.MGG_SCORE_SOFTMAX, "sigmoid": L.MGG_SCORE_SIGMOID}
_GROUP_SCORE = {None: 0, "best": L.MGG_GROUP_BEST, "two best": L.MGG_GROUP_TWO_BEST}
_ACTIVATION = {"none": L.MGG_ACT_NONE, "relu": L.MGG_ACT_RELU, "silu": L.MGG_ACT_SILU,
               "gelu": L.MGG_ACT_GELU}


class _Host:
    """The compiled entry (csrc/host.cpp: argument checks, output allocation,
    the C-ABI call), loaded at the first call; fails loudly if not built."""

    def __getattr__(self, name):
        global _host
        L.load()
        from . import _host as module
        _host = module
        return getattr(module, name)


_host = _Host()


# ---------------------------------------------------------------- layer norm
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                       eps: float = 1e-5, out_dtype: torch.dtype | None = None):
    """Layer norm of the rows of x [T, K].  Returns (y [T, K] in ``out_dtype``
    (default: x's), mean [T], rstd [T] float32) (mgg_layer_norm_forward)."""
    return _host.layer_norm_forward(x, weight, bias, eps, out_dtype)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        workspace: torch.Tensor | None = None):
    """Gradients of layer_norm_forward from its saved statistics.  Returns
    (dx in x's dtype, dweight and dbias in weight's; dbias None without
    ``bias``)."""
    return _host.layer_norm_backward(dy, x, weight, mean, rstd, bias, workspace)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, ctx.bias)
        return dx, dw, db, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Layer norm of the rows of x [T, K], differentiable to x, weight and bias."""
    return _LayerNorm.apply(x, weight, bias, eps, out_dtype)


# ---------------------------------------------------------------- expert choice
def _scoring(name: str) -> int:
    if name not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}")
    return _SCORING[name]


def select_experts(logits: torch.Tensor, k: int, scoring: str = "softmax",
                   bias: torch.Tensor | None = None, groups: int = 1, topk_groups: int = 1,
                   renormalize: bool = True, scale: float = 1.0, group_score: str | None = None):
    """The k experts of every token and their weights, from the gate's logits
    [T, E].  Returns (expert_ids [T, k] int32, topk_weights [T, k] float32),
    best first, equal keys to the lowest expert; ``bias`` [E] float32 moves
    the choice, not the weights.  -inf, NaN or the dtype's lowest value mask
    an expert.  ``group_score``: a group counts by its "best" key or the sum
    of its "two best" (with softmax of the scores, not the logits); None:
    two best with sigmoid, best with softmax (mgg_select_experts)."""
    if group_score not in _GROUP_SCORE:
        raise ValueError("group_score must be 'best', 'two best' or None")
    return _host.select_experts(logits, k, _scoring(scoring) | _GROUP_SCORE[group_score], bias, groups,
                                topk_groups, renormalize, scale)


def select_experts_backward(dtopk: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                            topk_weights: torch.Tensor, scoring: str = "softmax",
                            renormalize: bool = True, scale: float = 1.0,
                            status: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of topk_weights to the logits (their dtype), the choice held
    fixed, from what select_experts returned with the same options."""
    st = status if status is not None else new_status(logits.device)
    return _host.select_experts_backward(dtopk, logits, _ids_i32(expert_ids), topk_weights,
                                         _scoring(scoring), renormalize, scale, st)


class _Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, scoring, bias, groups, topk_groups, renormalize, scale, status,
                group_score):
        ids, w = select_experts(logits, k, scoring, bias, groups, topk_groups, renormalize, scale,
                                group_score)
        ctx.save_for_backward(logits, ids, w)
        ctx.opts = (scoring, renormalize, scale, status)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    @once_differentiable
    def backward(ctx, _, dw):
        logits, ids, w = ctx.saved_tensors
        d = select_experts_backward(dw.contiguous(), logits, ids, w, *ctx.opts)
        return d, None, None, None, None, None, None, None, None, None


def router(logits: torch.Tensor, k: int, scoring: str = "softmax",
           bias: torch.Tensor | None = None, groups: int = 1, topk_groups: int = 1,
           renormalize: bool = True, scale: float = 1.0, status: torch.Tensor | None = None,
           group_score: str | None = None):
    """select_experts, its weights differentiable to the logits: the
    expert_ids and topk_weights that ``moe`` takes.  ``status``: the word the
    backward reports errors in (without one they are dropped, and each
    backward zeroes a word of its own)."""
    return _Router.apply(logits, k, scoring, bias, groups, topk_groups, renormalize, scale, status,
                         group_score)


# ---------------------------------------------------------------- dense products
def _activation(name: str) -> int:
    if name not in _ACTIVATION:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATION)}")
    return _ACTIVATION[name]


def linear_forward(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
                   activation: str = "none", residual: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, save_pre: bool = False,
                   status: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """act(x W^T + bias) + residual for x [T, K], W [N, K] bfloat16.  Returns
    out [T, N] in ``out_dtype`` (default bfloat16), or with ``save_pre``
    (out, pre): pre = x W^T + bias in bfloat16, which the backward of an
    activation needs (mgg_linear_forward)."""
    st = status if status is not None else new_status(x.device)
    return _host.linear_forward(x, W, bias, _activation(activation), residual, out_dtype, save_pre, st,
                                out)


def linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor,
                    pre: torch.Tensor | None = None, activation: str = "none",
                    bias_dtype: torch.dtype | None = None, need_dx: bool = True,
                    need_dW: bool = True, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """Gradients of linear_forward: (dx [T, K], dW [N, K] bfloat16, dbias [N]
    in ``bias_dtype``, None without one).  dy bfloat16 or float32; ``pre`` from
    the forward, needed with an activation.  The residual's gradient is dy."""
    st = status if status is not None else new_status(x.device)
    return _host.linear_backward(dy, x, W, pre, _activation(activation), bias_dtype, need_dx, need_dW,
                                 st, workspace)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, activation, residual, out_dtype, status):
        keep = activation != "none" and any(ctx.needs_input_grad[:3])
        out = linear_forward(x, W, bias, activation, residual, out_dtype, save_pre=keep,
                             status=status)
        out, pre = out if keep else (out, None)
        ctx.save_for_backward(x, W, pre)
        ctx.activation, ctx.status = activation, status
        ctx.bias_dtype = bias.dtype if bias is not None and ctx.needs_input_grad[2] else None
        ctx.residual_dtype = residual.dtype if residual is not None else None
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, W, pre = ctx.saved_tensors
        nx, nw, nb = ctx.needs_input_grad[:3]
        dx = dW = db = None
        if nx or nw or nb:
            dx, dW, db = linear_backward(dy.contiguous(), x, W, pre, ctx.activation,
                                         ctx.bias_dtype, need_dx=nx, need_dW=nw,
                                         status=ctx.status)
        dr = dy.to(ctx.residual_dtype) if ctx.needs_input_grad[4] else None
        return dx, dW, db, None, dr, None, None


def linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None,
           out_dtype: torch.dtype | None = None,
           status: torch.Tensor | None = None) -> torch.Tensor:
    """act(x W^T + bias) + residual, differentiable to x, W, bias and residual.
    ``status``: the word that forward and backward report errors in (without
    one they are dropped, and each call zeroes a word of its own)."""
    return _Linear.apply(x, W, bias, activation, residual, out_dtype, status)
