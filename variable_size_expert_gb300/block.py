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
from .ops import _ids_i32, _ptr, _stream, _workspace, new_status

__all__ = [
    "layer_norm_forward", "layer_norm_backward", "layer_norm", "select_experts",
    "select_experts_backward", "router", "linear_forward", "linear_backward", "linear",
]

_SCORING = {"softmax": L.MGG_SCORE_SOFTMAX, "sigmoid": L.MGG_SCORE_SIGMOID}
_ACTIVATION = {"none": L.MGG_ACT_NONE, "relu": L.MGG_ACT_RELU, "silu": L.MGG_ACT_SILU,
               "gelu": L.MGG_ACT_GELU}


# The host's share of a small call is most of its time, so the checks below
# read each attribute of a tensor once, and tensors made here are not checked.
_CODE = {torch.bfloat16: L.MGG_BF16, torch.float32: L.MGG_F32}
_empty = torch.empty


def _code(dtype: torch.dtype) -> int:
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: bfloat16 or float32")
    return code


def _rows(t: torch.Tensor, what: str) -> tuple[int, int, int, int]:
    """Pointer, rows, columns and row stride (elements) of a 2-D tensor with
    contiguous rows."""
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    rows, cols = shape
    if t.is_contiguous():
        return t.data_ptr(), rows, cols, cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    if ld < cols:
        raise ValueError(f"{what}: rows must not overlap")
    return t.data_ptr(), rows, cols, ld


def _dense(t: torch.Tensor, shape: tuple, what: str) -> int:
    """Pointer of a contiguous tensor of the given shape."""
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _f32(t: torch.Tensor, shape: tuple, what: str) -> int:
    if t.dtype != torch.float32:
        raise ValueError(f"{what} must be float32")
    return _dense(t, shape, what)


def _room(workspace: torch.Tensor | None, nbytes: int, device) -> torch.Tensor:
    if workspace is not None:
        n = workspace.numel() * workspace.element_size()
        if n >= nbytes and workspace.is_cuda and workspace.is_contiguous():
            return workspace
    return _workspace(nbytes, device)


# ---------------------------------------------------------------- layer norm
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                       eps: float = 1e-5, out_dtype: torch.dtype | None = None):
    """Layer norm of the rows of x [T, K].  Returns (y [T, K] in ``out_dtype``
    (default: x's), mean [T], rstd [T] float32) (mgg_layer_norm_forward)."""
    xp, T, K, ldx = _rows(x, "x")
    dt = x.dtype
    yt = dt if out_dtype is None else out_dtype
    wt = weight.dtype
    shape = (K,)
    wp = _dense(weight, shape, "weight")
    bp = None
    if bias is not None:
        bp = _dense(bias, shape, "bias")
        if bias.dtype != wt:
            raise TypeError("weight and bias must share a dtype")
    xc, yc, wc = _code(dt), _code(yt), _code(wt)
    dev = x.device
    y = _empty((T, K), dtype=yt, device=dev)
    mean = _empty(T, dtype=torch.float32, device=dev)
    rstd = _empty(T, dtype=torch.float32, device=dev)
    r = L.load().mgg_layer_norm_forward(xp, xc, ldx, wp, bp, wc, T, K, eps, y.data_ptr(), yc,
                                        mean.data_ptr(), rstd.data_ptr(), _stream())
    if r:
        L.check(r, "mgg_layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                        mean: torch.Tensor, rstd: torch.Tensor, bias: bool = True,
                        workspace: torch.Tensor | None = None):
    """Gradients of layer_norm_forward from its saved statistics.  Returns
    (dx in x's dtype, dweight and dbias in weight's; dbias None without
    ``bias``)."""
    xp, T, K, ldx = _rows(x, "x")
    dyp = _dense(dy, (T, K), "dy")
    wp = _dense(weight, (K,), "weight")
    mp, rp = _f32(mean, (T,), "mean"), _f32(rstd, (T,), "rstd")
    dt, wt, dev = x.dtype, weight.dtype, x.device
    xc, wc, yc = _code(dt), _code(wt), _code(dy.dtype)
    lib = L.load()
    dx = _empty((T, K), dtype=dt, device=dev)
    dw = _empty(K, dtype=wt, device=dev)
    db = _empty(K, dtype=wt, device=dev) if bias else None
    ws = _room(workspace, lib.mgg_workspace_bytes(L.MGG_OP_LAYER_NORM_BACKWARD, T, 0, 0, 0, K,
                                                  L.MGG_F32), dev)
    r = lib.mgg_layer_norm_backward(dyp, yc, xp, xc, ldx, wp, wc, mp, rp, T, K, dx.data_ptr(),
                                    dw.data_ptr(), db.data_ptr() if bias else None, ws.data_ptr(),
                                    ws.numel() * ws.element_size(), _stream())
    if r:
        L.check(r, "mgg_layer_norm_backward")
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
    lp, T, E, ldl = _rows(logits, "logits")
    bp = None if bias is None else _f32(bias, (E,), "bias")
    lc, sc = _code(logits.dtype), _scoring(scoring)
    dev = logits.device
    ids = _empty((T, k), dtype=torch.int32, device=dev)
    w = _empty((T, k), dtype=torch.float32, device=dev)
    r = L.load().mgg_select_experts(lp, lc, ldl, T, E, k, sc, bp, groups, topk_groups,
                                    renormalize, scale, ids.data_ptr(), w.data_ptr(), _stream())
    if r:
        L.check(r, "mgg_select_experts")
    return ids, w


def select_experts_backward(dtopk: torch.Tensor, logits: torch.Tensor, expert_ids: torch.Tensor,
                            topk_weights: torch.Tensor, scoring: str = "softmax",
                            renormalize: bool = True, scale: float = 1.0,
                            status: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of topk_weights to the logits (their dtype), the choice held
    fixed, from what select_experts returned with the same options."""
    lp, T, E, ldl = _rows(logits, "logits")
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [T, k]")
    k = expert_ids.shape[1]
    shape = (T, k)
    ids = _ids_i32(expert_ids)
    ip = _dense(ids, shape, "expert_ids")
    gp, wp = _f32(dtopk, shape, "dtopk"), _f32(topk_weights, shape, "topk_weights")
    dt, dev = logits.dtype, logits.device
    lc, sc = _code(dt), _scoring(scoring)
    st = status if status is not None else new_status(dev)
    d = _empty((T, E), dtype=dt, device=dev)
    r = L.load().mgg_select_experts_backward(gp, lp, lc, ldl, ip, wp, T, E, k, sc, renormalize,
                                             scale, d.data_ptr(), _ptr(st), _stream())
    if r:
        L.check(r, "mgg_select_experts_backward")
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
    bf16 = torch.bfloat16
    if x.dtype != bf16 or W.dtype != bf16:
        raise TypeError("x and W must be bfloat16")
    xp, T, K, ldx = _rows(x, "x")
    N = W.shape[0] if W.dim() else 0
    Wp = _dense(W, (N, K), "W")
    bp, bc, rp, rc, ldr = None, L.MGG_F32, None, L.MGG_F32, N
    if bias is not None:
        bp, bc = _dense(bias, (N,), "bias"), _code(bias.dtype)
    if residual is not None:
        rp, rT, rN, ldr = _rows(residual, "residual")
        rc = _code(residual.dtype)
        if rT != T or rN != N:
            raise ValueError(f"residual must be {[T, N]}, got {[rT, rN]}")
    ac = _activation(activation)
    dev = x.device
    if out is None:
        out = _empty((T, N), dtype=bf16 if out_dtype is None else out_dtype, device=dev)
        op = out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out must have out_dtype")
        op = _dense(out, (T, N), "out")
    oc = _code(out.dtype)
    pre = _empty((T, N), dtype=bf16, device=dev) if save_pre else None
    st = status if status is not None else new_status(dev)
    r = L.load().mgg_linear_forward(xp, ldx, Wp, bp, bc, rp, rc, ldr, T, K, N, ac, op, oc,
                                    pre.data_ptr() if save_pre else None, _ptr(st), _stream())
    if r:
        L.check(r, "mgg_linear_forward")
    return (out, pre) if save_pre else out


def linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor,
                    pre: torch.Tensor | None = None, activation: str = "none",
                    bias_dtype: torch.dtype | None = None, need_dx: bool = True,
                    need_dW: bool = True, status: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None):
    """Gradients of linear_forward: (dx [T, K], dW [N, K] bfloat16, dbias [N]
    in ``bias_dtype``, None without one).  dy bfloat16 or float32; ``pre`` from
    the forward, needed with an activation.  The residual's gradient is dy."""
    bf16 = torch.bfloat16
    if x.dtype != bf16 or W.dtype != bf16:
        raise TypeError("x and W must be bfloat16")
    xp, T, K, ldx = _rows(x, "x")
    N = W.shape[0] if W.dim() else 0
    Wp = _dense(W, (N, K), "W")
    dyp, dT, dN, lddy = _rows(dy, "dy")
    if dT != T or dN != N:
        raise ValueError(f"dy must be {[T, N]}, got {[dT, dN]}")
    ac, dc = _activation(activation), _code(dy.dtype)
    pp = None
    if pre is not None:
        if pre.dtype != bf16:
            raise TypeError("pre must be bfloat16")
        pp = _dense(pre, (T, N), "pre")
    elif ac != L.MGG_ACT_NONE:
        raise ValueError("an activation's backward needs pre")
    dev = x.device
    dx = _empty((T, K), dtype=bf16, device=dev) if need_dx else None
    dW = _empty((N, K), dtype=bf16, device=dev) if need_dW else None
    db, bc = None, L.MGG_F32
    if bias_dtype is not None:
        bc = _code(bias_dtype)
        db = _empty(N, dtype=bias_dtype, device=dev)
    st = status if status is not None else new_status(dev)
    lib = L.load()
    ws = _room(workspace, lib.mgg_workspace_bytes(L.MGG_OP_LINEAR_BACKWARD, T, 0, 0, N, K,
                                                  L.MGG_BF16), dev)
    r = lib.mgg_linear_backward(
        dyp, dc, lddy, xp, ldx, Wp, pp, ac, T, K, N, dx.data_ptr() if need_dx else None,
        dW.data_ptr() if need_dW else None, db.data_ptr() if db is not None else None, bc, _ptr(st),
        ws.data_ptr(), ws.numel() * ws.element_size(), _stream())
    if r:
        L.check(r, "mgg_linear_backward")
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
