"""Plain float64 forms (CPU torch) of a training step's losses and optimiser,
written from their definitions, and the error bounds their kernels are held to
(first order, as in block_ref.py: U is the f32 unit roundoff, BF half a unit in
the last place of bfloat16, DEPTH the longest run of one thread's sum)."""
import math

import torch

from tests.block_ref import BF, DEPTH, U, d, dot_bound, scores

IGNORE = -100


# ---------------------------------------------------------------- balance loss
def probabilities(logits, scoring):
    """(p, a): a is the sigmoid of each logit, None with softmax."""
    if logits.dtype == torch.double:  # (`scores` takes the kernels' types, by way of f32)
        a = torch.sigmoid(logits)
        return (torch.softmax(logits, 1), None) if scoring == "softmax" else (a / a.sum(1, keepdim=True), a)
    p, open_, _ = scores(logits, scoring)
    if scoring == "softmax":
        return p, None
    a = torch.where(open_, p, torch.zeros_like(p))
    s = a.sum(1, keepdim=True)
    return a / torch.where(s > 0, s, torch.ones_like(s)), a


def balance(logits, ids, scoring, mask=None, sequences=1):
    """(loss, counts, slope)"""
    T, E = logits.shape
    k, B = ids.shape[1], sequences
    p, _ = probabilities(logits, scoring)
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu()
    counts, slope = torch.zeros(B, E, dtype=torch.long), torch.zeros(B, E, dtype=torch.double)
    n = on.view(B, -1).sum(1)
    live = int((n > 0).sum())
    i = ids.cpu().long()
    for b in range(B):
        at = slice(b * (T // B), (b + 1) * (T // B))
        chosen = i[at][on[at]].flatten()
        chosen = chosen[(chosen >= 0) & (chosen < E)]
        counts[b] = torch.bincount(chosen, minlength=E)
        if n[b] > 0:
            slope[b] = E * counts[b].double() / (k * float(n[b]) ** 2 * live)
    loss = (slope * (p * on.double()[:, None]).view(B, -1, E).sum(1)).sum()
    return loss, counts, slope


def p_error(logits):
    """Relative error of a probability: the exponential's argument (up to twice
    the largest finite logit) and a sum over the experts."""
    z = logits.float()
    z = z[torch.isfinite(z) & (z.abs() < 1e30)]
    return (4 * (float(z.abs().max()) if z.numel() else 0.0) + DEPTH) * U


def balance_grad(dloss, logits, slope, scoring, mask=None):
    """(dlogits, bound)"""
    T = logits.shape[0]
    p, a = probabilities(logits, scoring)
    g = slope.repeat_interleave(T // slope.shape[0], 0)
    dz = p * (g - (p * g).sum(1, keepdim=True))
    tol = p * (g.abs() + (p * g.abs()).sum(1, keepdim=True)) * 4 * p_error(logits)
    if a is not None:
        dz, tol = dz * (1 - a), tol * (1 - a) + U * dz.abs()
    on = dloss * (torch.ones(T) if mask is None else mask.cpu()).double()[:, None]
    return dz * on, tol * on.abs()


# ---------------------------------------------------------------- cross entropy
def vocab(x, W, targets, z_loss=0.0):
    """(losses [T], lse, bounds of both); targets outside [0, V) do not count."""
    z, t = d(x) @ d(W).t(), targets.cpu().long()
    V = z.shape[1]
    tz = dot_bound(d(x), d(W))
    lse = torch.logsumexp(z, 1)
    # every logit off by its bound moves lse by the largest; the sum's terms are
    # off by a few U each, in runs of 16 a thread, 6 steps and a tile in eight
    t_lse = tz.max(1).values + (DEPTH + V / 2048) * U + 4 * U * lse.abs()
    on = (t >= 0) & (t < V)
    at = torch.where(on, t, 0)[:, None]
    losses = lse - z.gather(1, at)[:, 0] + z_loss * lse * lse
    tol = t_lse * (1 + 2 * z_loss * lse.abs()) + tz.gather(1, at)[:, 0] + 8 * U * (lse.abs() + losses.abs())
    zero = torch.zeros_like(lse)
    return torch.where(on, losses, zero), lse, torch.where(on, tol, zero), t_lse


def vocab_grads(dloss, x, W, targets, lse, z_loss=0.0):
    """dx, dW and their bounds; dloss [T] or a number, a token's weight in it."""
    xd, Wd, t, l = d(x), d(W), targets.cpu().long(), d(lse)
    V = Wd.shape[0]
    on = ((t >= 0) & (t < V)).double()
    z = xd @ Wd.t()
    # p = exp(z - lse): the logit's error, the argument's roundings, ex2's 2 ulp
    rel = dot_bound(xd, Wd) + 4 * U * (z.abs() + l.abs()[:, None]) + 8 * U
    p = torch.exp(z - l[:, None]) * (1 + 2 * z_loss * l)[:, None]
    dz = p.clone()
    rows = torch.arange(len(t))[on > 0]
    dz[rows, t[rows]] -= 1.0
    g = torch.as_tensor(dloss, dtype=torch.double).expand(len(t))
    w = (on * g)[:, None]
    # the operand of both products is bf16(dz)
    tdz = (p.abs() * rel + dz.abs() * (BF * 1.01 + 4 * U)) * w.abs()
    dz = dz * w
    tx = tdz @ Wd.abs() + 1.01 * dot_bound(dz, Wd.t()) + 8 * U * (dz @ Wd).abs()
    tW = tdz.t() @ xd.abs() + 1.01 * dot_bound(dz.t(), xd.t()) + 8 * U * (dz.t() @ xd).abs()
    return dz @ Wd, dz.t() @ xd, tx, tW


# ---------------------------------------------------------------- AdamW
def adamw(p, g, m, v, t, lr, betas, eps, decay, scale=1.0):
    """(p, m, v) after the step and the bound of p; v the second moment."""
    b1, b2 = betas
    g = g * scale
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    den = (v1 / (1 - b2 ** t)).sqrt() + eps
    u = lr / (1 - b1 ** t) / den
    p1 = p * (1 - lr * decay) - u * m1
    # m's terms and coefficients are rounded (4 U of either, they may cancel); the
    # corrections, the root, its reciprocal and the products 24 U; p's own 3 U
    tol = u * 4 * U * (b1 * m.abs() + (1 - b1) * g.abs()) + 24 * U * (u * m1).abs() + 3 * U * p.abs()
    return p1, m1, v1, tol


def grid8(x, t, second):
    """x [n] in blocks of 256 on the 8-bit grid at step t: (values in units of the
    scale, scale, fractional distance of each to the next decision)."""
    n = x.numel()
    b = torch.zeros(-(-n // 256) * 256, dtype=torch.double)
    b[:n] = x
    finite = torch.where(torch.isfinite(b), b, torch.zeros_like(b)).view(-1, 256)
    scale = finite.abs().max(1).values / 448
    q = (b.view(-1, 256).abs() / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).flatten()[:n]
    salt = 1 << 31 if second else 0
    walk = torch.tensor([((i * 0x9E3779B1 + t * 0xC13FA9A9 + salt) % 2 ** 32) >> 12 for i in range(n)],
                        dtype=torch.double) / 2 ** 20
    step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
    steps = q / step + walk
    val = (torch.floor(steps) * step).clamp(max=448.0)
    if second:
        val = torch.where(q > 0, val.clamp(min=2.0 ** -9), val)
    near = (steps - torch.round(steps)).abs()
    return torch.copysign(torch.where(torch.isfinite(x), val, torch.full_like(val, math.nan)), x), scale, near
