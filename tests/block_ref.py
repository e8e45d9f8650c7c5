"""Plain float64 forms (CPU torch) of the layers around the experts, written
from their definitions, and the error bounds their kernels are held to.

Bounds are first-order rounding bounds.  U = 2^-24 is the f32 unit roundoff;
a sum of n terms formed by a tree over per-thread runs has depth at most
DEPTH here (16 terms per thread, 5 levels in a warp, 32 warps; the long-row
path runs K / 512 terms per thread), so its error is within DEPTH * U times
the sum of the magnitudes.  A bf16 result (8 significant bits) adds 2^-8 of its
magnitude (half a unit in the last place)."""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
DEPTH = 128


def d(t):
    return None if t is None else t.detach().cpu().double()


def within(got, ref, tol, name):
    g = d(got)
    assert g.shape == ref.shape, f"{name}: shape {tuple(g.shape)}"
    bad = ~((g - ref).abs() <= tol)
    if bad.any():
        i = int(((g - ref).abs() - tol).flatten().nan_to_num(math.inf).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {g.numel()} outside their bound; worst "
                             f"got {g.flatten()[i]} ref {ref.flatten()[i]} "
                             f"bound {torch.as_tensor(tol).expand_as(ref).flatten()[i]}")


def rounding(dtype, ref):
    """What storing ref in dtype may change (bf16: half a unit in the last place)."""
    return (BF if dtype == torch.bfloat16 else U) * ref.abs() + 1e-38


# ---------------------------------------------------------------- layer norm
def norm_forward(x, w, b, eps):
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = (xc.square().mean(1) + eps) ** -0.5
    y = xc * rstd[:, None] * w
    return (y if b is None else y + b), mean, rstd


def norm_forward_bounds(x, w, b, eps):
    y, mean, rstd = norm_forward(x, w, b, eps)
    mag = x.abs().mean(1)
    t_mean = DEPTH * U * mag
    xc = (x - mean[:, None]).abs()
    # an error e of the mean moves every x - mean by e, the variance by e^2
    # and (through the rounding of x - mean) rstd by 2 U + DEPTH U
    t_rstd = 2 * DEPTH * U * rstd + rstd * (t_mean * rstd) ** 2
    wr = w.abs() * rstd[:, None]
    t_y = wr * t_mean[:, None] + wr * xc * (3 * DEPTH * U + (t_mean * rstd)[:, None] ** 2)
    t_y = t_y + 4 * U * (y.abs() + (0 if b is None else b.abs()))
    return t_y, t_mean, t_rstd


def norm_backward(dy, x, w, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    c1 = g.mean(1, keepdim=True)
    c2 = (g * xh).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - c1 - xh * c2)
    mag = g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    t_dx = 2 * DEPTH * U * rstd[:, None] * mag
    # column sums: a run of T / (groups of rows) terms, then the groups, then the blocks
    n = DEPTH + x.shape[0] / 16
    return (dx, (dy * xh).sum(0), dy.sum(0),
            t_dx, n * U * (dy * xh).abs().sum(0), n * U * dy.abs().sum(0))


# ---------------------------------------------------------------- expert choice
def scores(logits, scoring):
    """(p float64, open mask): p is 0 where masked."""
    low = torch.finfo(logits.dtype).min
    open_ = logits.float() > low
    z = d(logits.float().clamp(max=torch.finfo(torch.float32).max))
    z = torch.where(open_.cpu(), z, torch.full_like(z, -math.inf))
    if scoring == "softmax":
        top = z.max(1, keepdim=True).values
        e = torch.where(z > -math.inf, torch.exp(z - torch.where(top > -math.inf, top, 0.0)),
                        torch.zeros_like(z))
        s = e.sum(1, keepdim=True)
        return e / torch.where(s > 0, s, torch.ones_like(s)), open_.cpu(), z
    return torch.sigmoid(z), open_.cpu(), z


def select(logits, k, scoring, bias, groups, topk_groups, renorm, scale):
    """ids, weights and keys of the definition in float64, ties to the lowest index."""
    p, open_, z = scores(logits, scoring)
    T, E = p.shape
    key = z if scoring == "softmax" and bias is None else p + (0 if bias is None else d(bias))
    key = torch.where(open_, key, torch.full_like(key, -math.inf))
    if groups > 1:
        per = key.view(T, groups, E // groups)
        srt = per.sort(dim=2, descending=True).values
        sc = srt[:, :, 0].clone()
        if scoring == "sigmoid" and E // groups > 1:
            sc += torch.where(srt[:, :, 1] > -math.inf, srt[:, :, 1], torch.zeros_like(sc))
        pick = torch.sort(sc, dim=1, descending=True, stable=True).indices[:, :topk_groups]
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, pick, True)
        key = torch.where(keep.repeat_interleave(E // groups, 1), key,
                          torch.full_like(key, -math.inf))
    srt, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = ids[:, :k]
    w = torch.where(srt[:, :k] > -math.inf, p.gather(1, ids), torch.zeros(T, k).double())
    return ids, weigh(w, renorm, scale), key


def weigh(w, renorm, scale):
    if renorm:
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s > 0, s, torch.ones_like(s))
    return w * scale


def weights_of(z, ids, live, scoring, renorm, scale):
    """topk_weights as a differentiable function of float64 logits z, the
    choice held fixed; ``live``: which choices carry weight."""
    p = torch.softmax(z, 1) if scoring == "softmax" else torch.sigmoid(z)
    w = torch.where(live, p.gather(1, ids), torch.zeros_like(live, dtype=torch.float64))
    return weigh(w, renorm, scale)


# ---------------------------------------------------------------- dense products
def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.special.erf(z / math.sqrt(2)))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.special.erf(z / math.sqrt(2))) \
            + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def dot_bound(a, b):
    """Bound of sum_k a b on the tensor cores: bf16 products are exact in f32,
    one addition per 16 of the contraction and up to 16 within it, each within
    one f32 unit in the last place (2 U, truncation) of the magnitudes."""
    K = a.shape[1]
    return 2 * U * (K / 16 + 16 + 8) * (a.abs() @ b.abs().t())
