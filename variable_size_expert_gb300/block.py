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
plus the *_forward / *_backward calls under them.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .ops import _dtype_code, _ids_i32, _ptr, _stream, _workspace, new_status

__all__ = [
    "layer_norm_forward", "layer_norm_backward", "layer_norm", "select_experts",
    "select_experts_backward", "router", "linear_forward", "linear_backward", "linear",
]

_SCORING = {"softmax": L.MGG_SCORE_SOFTMAX, "sigmoid": L.MGG_SCORE_SIGMOID}
_ACTIVATION = {"none": L.MGG_ACT_NONE, "relu": L.MGG_ACT_RELU, "silu": L.MGG_ACT_SILU,
               "gelu": L.MGG_ACT_GELU}


def _rows(t: torch.Tensor, what: str) -> tuple[int, int]:
    """Pointer and row stride (elements) of a 2-D tensor with contiguous rows."""
    if t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}: rows must not overlap")
    return t.data_ptr(), ld


def _expect(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _opt(t: torch.Tensor | None) -> int | None:
    return None if t is None else _ptr(t)


# ---------------------------------------------------------------- layer norm
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                       eps: float = 1e-5, out_dtype: torch.dtype | None = None):
    """Layer norm of the rows of x [T, K].  Returns (y [T, K] in ``out_dtype``
    (default: x's), mean [T], rstd [T] float32) (mgg_layer_norm_forward)."""
    xp, ldx = _rows(x, "x")
    T, K = x.shape
    y = torch.empty(T, K, dtype=out_dtype or x.dtype, device=x.device)
    _expect(weight.shape == (K,) and (bias is None or bias.shape == (K,)),
            "weight and bias must be [K] with the K of x")
    if bias is not None and bias.dtype != weight.dtype:
        raise TypeError("weight and bias must share a dtype")
    mean = torch.empty(T, dtype=torch.float32, device=x.device)
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    L.check(L.load().mgg_layer_norm_forward(xp, _dtype_code(x), ldx, _ptr(weight), _opt(bias),
                                            _dtype_code(weight), T, K, eps, _ptr(y),
                                            _dtype_code(y), _ptr(mean), _ptr(rstd), _stream()),
            "mgg_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        workspace: torch.Tensor | None = None):
    """Gradients of layer_norm_forward from its saved statistics.  Returns
    (dx in x's dtype, dweight and dbias in weight's; dbias None without
    ``bias``)."""
    lib = L.load()
    xp, ldx = _rows(x, "x")
    T, K = x.shape
    _expect(dy.shape == (T, K) and weight.shape == (K,), "dy [T, K] and weight [K] must match x")
    _expect(mean.shape == (T,) and rstd.shape == (T,) and mean.dtype == torch.float32
            and rstd.dtype == torch.float32, "mean and rstd must be float32 [T]")
    dx = torch.empty(T, K, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(weight)
    db = torch.empty_like(weight) if bias else None
    nbytes = lib.mgg_workspace_bytes(L.MGG_OP_LAYER_NORM_BACKWARD, T, 0, 0, 0, K, L.MGG_F32)
    ws = workspace if workspace is not None and workspace.numel() >= nbytes else _workspace(nbytes, x.device)
    L.check(lib.mgg_layer_norm_backward(_ptr(dy), _dtype_code(dy), xp, _dtype_code(x), ldx,
                                        _ptr(weight), _dtype_code(weight), _ptr(mean), _ptr(rstd),
                                        T, K, _ptr(dx), _ptr(dw), _opt(db), _ptr(ws), ws.numel(),
                                        _stream()), "mgg_layer_norm_backward")
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps, out_dtype)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias = bias is not None
        return y

    @staticmethod
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
                   renormalize: bool = True, scale: float = 1.0):
    """The k experts of every token and their weights, from the gate's logits
    [T, E].  Returns (expert_ids [T, k] int32, topk_weights [T, k] float32),
    best first, equal keys to the lowest expert; ``bias`` [E] float32 moves
    the choice, not the weights.  -inf, NaN or the dtype's lowest value mask
    an expert (mgg_select_experts)."""
    lp, ldl = _rows(logits, "logits")
    T, E = logits.shape
    _expect(bias is None or (bias.shape == (E,) and bias.dtype == torch.float32),
            "bias must be float32 [E]")
    ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    L.check(L.load().mgg_select_experts(lp, _dtype_code(logits), ldl, T, E, k, _scoring(scoring),
                                        _opt(bias), groups, topk_groups, int(renormalize), scale,
                                        _ptr(ids), _ptr(w), _stream()), "mgg_select_experts")
    return ids, w


def select_experts_backward(dtopk: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                            topk_weights: torch.Tensor, scoring: str = "softmax",
                            renormalize: bool = True, scale: float = 1.0,
                            status: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of topk_weights to the logits (their dtype), the choice held
    fixed, from what select_experts returned with the same options."""
    lp, ldl = _rows(logits, "logits")
    T, E = logits.shape
    k = expert_ids.shape[1]
    _expect(expert_ids.shape == (T, k) and topk_weights.shape == (T, k) and dtopk.shape == (T, k),
            "dtopk, expert_ids and topk_weights must be [T, k] with the T of logits")
    _expect(dtopk.dtype == torch.float32 and topk_weights.dtype == torch.float32,
            "dtopk and topk_weights must be float32")
    st = status if status is not None else new_status(logits.device)
    d = torch.empty(T, E, dtype=logits.dtype, device=logits.device)
    L.check(L.load().mgg_select_experts_backward(
        _ptr(dtopk), lp, _dtype_code(logits), ldl, _ptr(_ids_i32(expert_ids)), _ptr(topk_weights),
        T, E, k, _scoring(scoring), int(renormalize), scale, _ptr(d), _ptr(st), _stream()),
        "mgg_select_experts_backward")
    return d


class _Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, scoring, bias, groups, topk_groups, renormalize, scale):
        ids, w = select_experts(logits, k, scoring, bias, groups, topk_groups, renormalize, scale)
        ctx.save_for_backward(logits, ids, w)
        ctx.opts = (scoring, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return ids, w

    @staticmethod
    def backward(ctx, _, dw):
        logits, ids, w = ctx.saved_tensors
        d = select_experts_backward(dw.contiguous(), logits, ids, w, *ctx.opts)
        return d, None, None, None, None, None, None, None


def router(logits: torch.Tensor, k: int, scoring: str = "softmax",
           bias: torch.Tensor | None = None, groups: int = 1, topk_groups: int = 1,
           renormalize: bool = True, scale: float = 1.0):
    """select_experts, its weights differentiable to the logits: the
    expert_ids and topk_weights that ``moe`` takes."""
    return _Router.apply(logits, k, scoring, bias, groups, topk_groups, renormalize, scale)


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
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("x and W must be bfloat16")
    xp, ldx = _rows(x, "x")
    T, K = x.shape
    _expect(W.dim() == 2 and W.shape[1] == K, "W must be [N, K] with the K of x")
    N = W.shape[0]
    _expect(bias is None or bias.shape == (N,), "bias must be [N]")
    rp, ldr, rcode = None, N, L.MGG_F32
    if residual is not None:
        _expect(residual.shape == (T, N), "residual must be [T, N]")
        rp, ldr = _rows(residual, "residual")
        rcode = _dtype_code(residual)
    dev = x.device
    if out is None:
        out = torch.empty(T, N, dtype=out_dtype or torch.bfloat16, device=dev)
    else:
        _expect(out.shape == (T, N) and (out_dtype is None or out.dtype == out_dtype),
                "out must be [T, N] in out_dtype")
    pre = torch.empty(T, N, dtype=torch.bfloat16, device=dev) if save_pre else None
    st = status if status is not None else new_status(dev)
    L.check(L.load().mgg_linear_forward(
        xp, ldx, _ptr(W), _opt(bias), _dtype_code(bias) if bias is not None else L.MGG_F32, rp,
        rcode, ldr, T, K, N, _activation(activation), _ptr(out), _dtype_code(out), _opt(pre),
        _ptr(st), _stream()), "mgg_linear_forward")
    return (out, pre) if save_pre else out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor,
                    pre: torch.Tensor | None = None, activation: str = "none",
                    bias_dtype: torch.dtype | None = None, need_dx: bool = True,
                    need_dW: bool = True, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """Gradients of linear_forward: (dx [T, K], dW [N, K] bfloat16, dbias [N]
    in ``bias_dtype``, None without one).  dy bfloat16 or float32; ``pre`` from
    the forward, needed with an activation.  The residual's gradient is dy."""
    lib = L.load()
    if x.dtype != torch.bfloat16 or W.dtype != torch.bfloat16:
        raise TypeError("x and W must be bfloat16")
    xp, ldx = _rows(x, "x")
    T, K = x.shape
    _expect(W.dim() == 2 and W.shape[1] == K, "W must be [N, K] with the K of x")
    N = W.shape[0]
    _expect(dy.shape == (T, N), "dy must be [T, N]")
    dyp, lddy = _rows(dy, "dy")
    _expect(pre is None or (pre.shape == (T, N) and pre.dtype == torch.bfloat16),
            "pre must be bfloat16 [T, N]")
    _expect(activation == "none" or pre is not None, "an activation's backward needs pre")
    dev = x.device
    dx = torch.empty(T, K, dtype=torch.bfloat16, device=dev) if need_dx else None
    dW = torch.empty(N, K, dtype=torch.bfloat16, device=dev) if need_dW else None
    db = torch.empty(N, dtype=bias_dtype, device=dev) if bias_dtype is not None else None
    st = status if status is not None else new_status(dev)
    nbytes = lib.mgg_workspace_bytes(L.MGG_OP_LINEAR_BACKWARD, T, 0, 0, N, K, L.MGG_BF16)
    ws = workspace if workspace is not None and workspace.numel() >= nbytes else _workspace(nbytes, dev)
    L.check(lib.mgg_linear_backward(
        dyp, _dtype_code(dy), lddy, xp, ldx, _ptr(W), _opt(pre), _activation(activation), T, K, N,
        _opt(dx), _opt(dW), _opt(db), _dtype_code(db) if db is not None else L.MGG_F32, _ptr(st),
        _ptr(ws), ws.numel(), _stream()), "mgg_linear_backward")
    return dx, dW, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, activation, residual, out_dtype):
        keep = activation != "none" and any(ctx.needs_input_grad[:3])
        out = linear_forward(x, W, bias, activation, residual, out_dtype, save_pre=keep)
        out, pre = out if keep else (out, None)
        ctx.save_for_backward(x, W, pre)
        ctx.activation = activation
        ctx.bias_dtype = bias.dtype if bias is not None and ctx.needs_input_grad[2] else None
        ctx.residual_dtype = residual.dtype if residual is not None else None
        return out

    @staticmethod
    def backward(ctx, dy):
        x, W, pre = ctx.saved_tensors
        nx, nw, nb = ctx.needs_input_grad[:3]
        dx = dW = db = None
        if nx or nw or nb:
            dx, dW, db = linear_backward(dy.contiguous(), x, W, pre, ctx.activation,
                                         ctx.bias_dtype, need_dx=nx, need_dW=nw)
        dr = dy.to(ctx.residual_dtype) if ctx.needs_input_grad[4] else None
        return dx, dW, db, None, dr, None


def linear(x: torch.Tensor, W: torch.Tensor, bias: torch.Tensor | None = None,
           activation: str = "none", residual: torch.Tensor | None = None,
           out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """act(x W^T + bias) + residual, differentiable to x, W, bias and residual."""
    return _Linear.apply(x, W, bias, activation, residual, out_dtype)
