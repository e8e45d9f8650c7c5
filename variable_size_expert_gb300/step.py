"""torch-facing API of what a training step needs around the blocks: the
balance loss of a gate, the cross entropy over a vocabulary straight from the
hidden states, and the AdamW step over all of a model's tensors.

  balance_loss(logits, expert_ids, ...)    differentiable, with the experts' counts
  linear_cross_entropy(x, W, targets, ...) differentiable
  adamw_step(params, grads, ...)           in place; AdamW keeps its state
plus the *_forward / *_backward calls under them.  As in block.py every step
runs in libmgg.so's kernels on the current stream, the tensors of a call live
on one GPU and it runs there, and gradients of gradients are an error.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _lib as L
from . import block
from .block import _scoring
from .ops import _ids_i32, new_status

__all__ = [
    "balance_loss_forward", "balance_loss_backward", "balance_loss",
    "linear_cross_entropy_forward", "linear_cross_entropy_backward", "linear_cross_entropy",
    "adamw_state", "adamw_step", "AdamW",
]

_REDUCTION = {"none": L.MGG_REDUCE_NONE, "sum": L.MGG_REDUCE_SUM, "mean": L.MGG_REDUCE_MEAN}


# ---------------------------------------------------------------- balance loss
def balance_loss_forward(logits: torch.Tensor, expert_ids: torch.Tensor, scoring: str = "softmax",
                         mask: torch.Tensor | None = None, sequences: int = 1,
                         status: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Balance loss of a gate from its logits [T, E] and the chosen experts
    [T, k]: the mean over the ``sequences`` equal runs of tokens of
    sum_e (E counts_e / (k n)) (mean probability of e); 1 where the load is
    even.  ``mask`` [T] bool: the tokens that count.  Returns (loss [] float32,
    counts [sequences, E] int32, slope [sequences, E] float32, what the
    backward needs) (mgg_balance_loss)."""
    st = status if status is not None else new_status(logits.device)
    return block._host.balance_loss_forward(logits, _ids_i32(expert_ids), _scoring(scoring), mask, sequences,
                                            st, workspace)


def balance_loss_backward(dloss: torch.Tensor, logits: torch.Tensor, slope: torch.Tensor,
                          scoring: str = "softmax", mask: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of the loss to the logits (their dtype), the counts held
    fixed; dloss a float32 scalar on the GPU."""
    return block._host.balance_loss_backward(dloss, logits, slope, _scoring(scoring), mask)


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, scoring, mask, sequences, status):
        loss, counts, slope = balance_loss_forward(logits, ids, scoring, mask, sequences, status)
        ctx.save_for_backward(logits, slope, mask)
        ctx.scoring = scoring
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _):
        logits, slope, mask = ctx.saved_tensors
        return balance_loss_backward(dloss, logits, slope, ctx.scoring, mask), None, None, None, None, None


def balance_loss(logits: torch.Tensor, expert_ids: torch.Tensor, scoring: str = "softmax",
                 mask: torch.Tensor | None = None, sequences: int = 1, status: torch.Tensor | None = None):
    """(loss, counts) of balance_loss_forward, the loss differentiable to the
    logits: the auxiliary loss beside ``router``'s choice, and the load."""
    return _BalanceLoss.apply(logits, expert_ids, scoring, mask, sequences, status)


# ---------------------------------------------------------------- cross entropy
def _reduction(name: str) -> int:
    if name not in _REDUCTION:
        raise ValueError(f"reduction must be one of {sorted(_REDUCTION)}")
    return _REDUCTION[name]


def linear_cross_entropy_forward(x: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                                 ignore_index: int = -100, reduction: str = "mean", z_loss: float = 0.0,
                                 status: torch.Tensor | None = None,
                                 workspace: torch.Tensor | None = None):
    """Cross entropy of the logits x W^T [T, V], which are never kept, for x
    [T, K], W [V, K] bfloat16 and targets [T] int64 or int32: lse - logit of
    the target + z_loss lse^2 a token, 0 where the target is ``ignore_index``.
    Returns (loss: [T] with reduction "none", else [], the sum or the mean over
    the tokens that count, 0 if none does; lse [T]; weight [1], a token's
    weight in the loss), float32.  A target outside the vocabulary does not
    count and is reported in ``status`` (mgg_linear_cross_entropy)."""
    st = status if status is not None else new_status(x.device)
    return block._host.linear_cross_entropy_forward(x, W, targets, ignore_index, _reduction(reduction), z_loss,
                                                    st, workspace)


def linear_cross_entropy_backward(dloss: torch.Tensor, x: torch.Tensor, W: torch.Tensor,
                                  targets: torch.Tensor, lse: torch.Tensor, weight: torch.Tensor,
                                  ignore_index: int = -100, z_loss: float = 0.0, need_dx: bool = True,
                                  need_dW: bool = True, status: torch.Tensor | None = None,
                                  workspace: torch.Tensor | None = None):
    """Gradients of linear_cross_entropy_forward from its lse and weight: (dx
    [T, K], dW [V, K]) bfloat16.  dloss float32 on the GPU: a scalar, or [T]
    after reduction "none".  Whatever x holds of tokens that do not count
    reaches neither."""
    st = status if status is not None else new_status(x.device)
    return block._host.linear_cross_entropy_backward(dloss, x, W, targets, lse, weight, ignore_index, z_loss,
                                                     need_dx, need_dW, st, workspace)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, targets, ignore_index, reduction, z_loss, status):
        loss, lse, weight = linear_cross_entropy_forward(x, W, targets, ignore_index, reduction, z_loss, status)
        ctx.save_for_backward(x, W, targets, lse, weight)
        ctx.opts = (ignore_index, z_loss)
        ctx.status = status
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        nx, nw = ctx.needs_input_grad[:2]
        dx, dW = linear_cross_entropy_backward(dloss.contiguous(), *ctx.saved_tensors, *ctx.opts, need_dx=nx,
                                               need_dW=nw, status=ctx.status)
        return dx, dW, None, None, None, None, None


def linear_cross_entropy(x: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean", z_loss: float = 0.0,
                         status: torch.Tensor | None = None) -> torch.Tensor:
    """The loss of linear_cross_entropy_forward, differentiable to x and W.
    ``status``: the word that forward and backward report errors in (without
    one they are dropped, and each call zeroes a word of its own)."""
    return _LinearCrossEntropy.apply(x, W, targets, ignore_index, reduction, z_loss, status)


# ---------------------------------------------------------------- AdamW
def adamw_state(params, bits: int = 32):
    """Moments of ``params`` before the first step: (exp_avg, exp_avg_sq,
    exp_avg_scale, exp_avg_sq_scale), lists as adamw_step takes them; with
    ``bits`` 8 float8_e4m3fn codes (of the second moment's root) and a float32
    scale for each 256 elements, else float32 and None for the scales."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    params = list(params)
    dtype = torch.float32 if bits == 32 else torch.float8_e4m3fn
    m, v = ([torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(dtype) if bits == 8
             else torch.zeros(p.shape, dtype=dtype, device=p.device) for p in params] for _ in range(2))
    if bits == 32:
        return m, v, None, None
    ms, vs = ([torch.zeros(-(-p.numel() // L.MGG_ADAMW_BLOCK), device=p.device) for p in params]
              for _ in range(2))
    return m, v, ms, vs


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 1e-2, masters=None, exp_avg_scale=None, exp_avg_sq_scale=None,
               grad_scale: torch.Tensor | None = None) -> None:
    """One AdamW step over lists of dense tensors, in place: params (bfloat16 or
    float32), grads (either), moments from adamw_state; with ``masters``
    (float32 copies of bfloat16 params) those are updated and the params
    receive them rounded.  ``step`` counts from 1; it and ``lr`` may be GPU
    tensors of one element (int32, float32), which a captured call reads anew.
    ``grad_scale`` (float32 [1] on the GPU) multiplies the gradients
    (mgg_adamw_step)."""
    block._host.adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr, betas[0], betas[1], eps, weight_decay,
                           masters, exp_avg_scale, exp_avg_sq_scale, grad_scale)


def _versions(tensors) -> list:
    """How often each was written in place (a tensor of inference mode does not count)."""
    try:
        return [t._version for t in tensors]
    except RuntimeError:
        return [0 if t.is_inference() else t._version for t in tensors]


class AdamW:
    """AdamW over ``params`` with their state: step() updates those that have a
    gradient, in one launch for each mix of dtypes among them; a step that is
    refused has updated and counted nothing.  ``bits`` 8 holds the moments in 8
    bits.  ``master`` keeps float32 copies of bfloat16 params; they take over
    what was written into their params since the last step (weights that were
    loaded), found by the tensors' versions: see sync_masters.  One count of
    steps holds for all of them: a gradient that first comes later is corrected
    as one that was zero until then.  ``capturable``: the count lives on the
    GPU, so that a captured step() counts its replays; ``lr`` may then be a
    float32 tensor."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
                 bits: int = 32, master: bool = True, capturable: bool = False):
        self.params = list(params)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale = adamw_state(self.params, bits)
        self.masters = [p.detach().float() if master and p.dtype == torch.bfloat16 else None
                        for p in self.params]
        self._seen = _versions(self.params)     # the params' versions that their masters stand for
        self.capturable = capturable
        device = self.params[0].device if self.params else "cpu"
        self.count = torch.zeros(1, dtype=torch.int32, device=device) if capturable else 0

    @torch.no_grad()
    def step(self, grad_scale: torch.Tensor | None = None) -> None:
        grads = [p.grad for p in self.params]
        mixes: dict = {}
        for i, (p, g, w) in enumerate(zip(self.params, grads, self.masters)):
            if g is not None:
                mixes.setdefault((p.dtype, g.dtype, w is None), []).append(i)
        seen = _versions(self.params)
        late = [] if seen == self._seen else [i for i, (a, b) in enumerate(zip(seen, self._seen)) if a != b]
        for i in late:
            if grads[i] is not None and self.masters[i] is not None:
                self._take_over(i)
        count = self.count if self.capturable else self.count + 1
        calls = []
        for (_, _, alone), at in mixes.items():
            def pick(t):
                return t if t is None or len(at) == len(t) else [t[i] for i in at]
            calls.append((pick(self.params), pick(grads), pick(self.exp_avg), pick(self.exp_avg_sq), count, self.lr,
                          self.betas, self.eps, self.weight_decay, None if alone else pick(self.masters),
                          pick(self.exp_avg_scale), pick(self.exp_avg_sq_scale), grad_scale))
        # One call refuses before it updates anything.  Where something precedes a call
        # (another mix, the count on the GPU), all are checked first.  (Without a GPU
        # the first call refuses.)
        if (self.capturable or len(calls) > 1) and any(c[0][0].is_cuda for c in calls):
            for c in calls:
                block._host.adamw_check(*c[:6], c[6][0], c[6][1], *c[7:])
        if self.capturable:
            self.count += 1
        for c in calls:
            adamw_step(*c)
        self.count = count
        seen = _versions(self.params)
        for i in late:
            if grads[i] is None:        # (to be taken over when one comes)
                seen[i] = self._seen[i]
        self._seen = seen

    def _take_over(self, i: int) -> None:
        p, w = self.params[i].detach(), self.masters[i]
        # (what a param holds unchanged is its master rounded: that keeps its bits)
        w.copy_(torch.where(w.to(p.dtype) == p, w, p.to(w.dtype)))

    @torch.no_grad()
    def sync_masters(self) -> None:
        """Masters take over every element of their params that is not the
        master's own, rounded.  step() does so for params whose version has
        changed; to be called after writes that count no version (through
        ``.data``, by a captured graph) and after writes that replays of a
        captured step are to see."""
        for i, w in enumerate(self.masters):
            if w is not None:
                self._take_over(i)
        self._seen = _versions(self.params)

    def zero_grad(self) -> None:
        for p in self.params:
            p.grad = None
