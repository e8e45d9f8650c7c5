"""Cases of the operators around the expert products, as a MoE transformer
block calls them: the layer norm before the layer, the choice of the experts
from the gate's logits, and the dense products beside the experts (gate,
shared expert, residual), each forward and backward.

``own`` False computes them in plain torch operations in float32, rounded
once at the end; ``own`` True makes the library's calls.
"""
import math
import random

import torch

own = False

NORM_EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # norm of a decode batch's rows at a wide hidden size: latency
        _ln("norm_decode", T=16, K=7168, x="bf16", y="bf16", w="bf16"),
        # norm of a float32 residual stream into the bf16 operands of the experts
        _ln("norm_stream", T=16384, K=2048, x="f32", y="bf16", w="f32"),
        # its gradient at the step's usual token count
        _ln("norm_backward", T=4096, K=2048, x="f32", y="bf16", w="f32", back=True),
        # ragged: a token count and a width that divide by nothing
        _ln("norm_backward_odd", T=8191, K=7163, x="bf16", y="bf16", w="bf16", back=True),
        # a decode step's choice: softmax over bf16 logits (many equal values)
        _sel("select_decode", T=64, E=128, k=8, scoring="softmax", logits="bf16"),
        # a prefill's choice: sigmoid scores, balance bias, 4 of 8 groups
        _sel("select_groups", T=16384, E=256, k=8, scoring="sigmoid", bias=True, groups=8,
             topk_groups=4, scale=2.5),
        # gradients: renormalised (zero off the chosen experts), and not (dense)
        _sel("select_backward", T=4096, E=64, k=8, scoring="softmax", back=True),
        _sel("select_backward_dense", T=16384, E=256, k=8, scoring="softmax", renorm=False,
             back=True),
        # a decode step's projection onto the residual stream: reads the weight once
        _lin("linear_decode", T=16, K=7168, N=2048, residual="f32", out="f32"),
        # the shared expert's up projection in training: bias, GELU, z kept
        _lin("linear_up", T=8192, K=2048, N=8192, act="gelu", bias="bf16", pre=True),
        # gradients of the gate product: a few columns, float32 dy
        _lin("linear_backward_gate", T=4096, K=2048, N=64, out="f32", back=True),
        # gradients of the up projection
        _lin("linear_backward_up", T=8192, K=2048, N=8192, act="gelu", bias="bf16", back=True),
    ]


def _ln(name, T, K, x, y, w, bias=True, back=False):
    return dict(name=name, op="norm", T=T, K=K, x=x, y=y, w=w, bias=bias, back=back)


def _sel(name, T, E, k, scoring, logits="f32", bias=False, groups=1, topk_groups=1, renorm=True,
         scale=1.0, back=False):
    return dict(name=name, op="select", T=T, E=E, k=k, scoring=scoring, logits=logits, bias=bias,
                groups=groups, topk_groups=topk_groups, renorm=renorm, scale=scale, back=back)


def _lin(name, T, K, N, act="none", bias=None, residual=None, out="bf16", pre=False, back=False):
    return dict(name=name, op="linear", T=T, K=K, N=N, act=act, bias=bias, residual=residual,
                out=out, pre=pre, back=back)


# most work of a drawn dense product (that of the largest listed one)
_MOST = 8192 * 2048 * 8192


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "select", "linear"])
    back = rng.random() < 0.5
    T = _log(rng, 1, 16384)
    if kind == "norm":
        # widths: multiples of 8 as hidden sizes are, and any
        K = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            K = max(64, K // 8 * 8)
        while T * K > 8191 * 7163:
            T = _log(rng, 1, 16384)
        x, y = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
        c = _ln("", T, K, x, y, rng.choice(["f32", "bf16"]), bias=rng.random() < 0.7, back=back)
    elif kind == "select":
        E = _log(rng, 8, 1024)
        groups = topk_groups = 1
        if rng.random() < 0.4:
            E = max(16, E // 16 * 16)
            groups = rng.choice([2, 4, 8])
            topk_groups = rng.randint(1, groups)
        k = min(_log(rng, 1, 16), topk_groups * (E // groups))
        while T * E > 16384 * 256:
            T = _log(rng, 1, 16384)
        scoring = rng.choice(["softmax", "sigmoid"])
        # a bias goes with sigmoid scores: with softmax ones the last bit of a
        # sum would decide near ties, and no order of that sum is the right one
        # one expert's weight, renormalised, is a constant
        renorm = k > 1 and rng.random() < 0.6
        c = _sel("", T, E, k, scoring, logits=rng.choice(["f32", "bf16"]),
                 bias=scoring == "sigmoid" and rng.random() < 0.7, groups=groups,
                 topk_groups=topk_groups, renorm=renorm,
                 scale=rng.choice([1.0, 2.5]), back=back)
    else:
        K = max(64, _log(rng, 64, 8192) // 8 * 8)
        N = _log(rng, 4, 8192)
        if rng.random() < 0.7:
            N = max(8, N // 8 * 8)
        while T * K * N > _MOST:
            T = _log(rng, 1, 16384)
        c = _lin("", T, K, N, act=rng.choice(["none", "relu", "silu", "gelu"]),
                 bias=rng.choice([None, "f32", "bf16"]),
                 residual=None if back else rng.choice([None, "f32", "bf16"]),
                 out=rng.choice(["bf16", "f32"]), pre=not back and rng.random() < 0.4, back=back)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(_DT[dtype])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    T = c["T"]
    if c["op"] == "norm":
        K = c["K"]
        # a residual stream: channels of unequal scale and a common offset
        chan = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
        s["x"] = (torch.randn(T, K, generator=g, device="cuda") * chan + 0.3 * chan).to(_DT[c["x"]])
        s["w"] = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(_DT[c["w"]])
        s["b"] = _randn(g, K, dtype=c["w"], std=0.1) if c["bias"] else None
        if c["back"]:
            s["dy"] = _randn(g, T, K, dtype=c["y"])
            x = s["x"].float()
            mean = x.mean(1)
            s["mean"] = mean
            s["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + NORM_EPS)
    elif c["op"] == "select":
        E, k = c["E"], c["k"]
        # logits of a trained gate: some experts liked more than others
        s["logits"] = (1.5 * torch.randn(T, E, generator=g, device="cuda")
                       + 0.5 * torch.randn(E, generator=g, device="cuda")).to(_DT[c["logits"]])
        s["bias"] = _randn(g, E, std=0.05) if c["bias"] else None
        if c["back"]:
            s["ids"], s["weights"] = _select_plain(c, s)
            s["dw"] = _randn(g, T, k)
    else:
        K, N = c["K"], c["N"]
        s["x"] = _randn(g, T, K, dtype="bf16")
        s["W"] = _randn(g, N, K, dtype="bf16", std=1.0 / math.sqrt(K))
        if c["back"]:
            s["dy"] = _randn(g, T, N, dtype=c["out"])
            s["pre"] = _randn(g, T, N, dtype="bf16") if c["act"] != "none" else None
        else:
            s["b"] = _randn(g, N, dtype=c["bias"], std=0.1) if c["bias"] else None
            s["residual"] = _randn(g, T, N, dtype=c["residual"]) if c["residual"] else None
    # the word that the library's kernels report errors in, kept by the program
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _OWN[c["op"], c["back"]](c, state)
    return _PLAIN[c["op"], c["back"]](c, state)


def _norm_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.layer_norm_forward(s["x"], s["w"], s["b"], eps=NORM_EPS, out_dtype=_DT[c["y"]])


def _norm_back_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], bias=c["bias"])


def _select_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.select_experts(s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"],
                              groups=c["groups"], topk_groups=c["topk_groups"],
                              renormalize=c["renorm"], scale=c["scale"])


def _select_back_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.select_experts_backward(s["dw"], s["logits"], s["ids"], s["weights"],
                                       scoring=c["scoring"], renormalize=c["renorm"],
                                       scale=c["scale"], status=s["status"])


def _linear_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.linear_forward(s["x"], s["W"], s["b"], activation=c["act"], residual=s["residual"],
                              out_dtype=_DT[c["out"]], save_pre=c["pre"], status=s["status"])


def _linear_back_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.linear_backward(s["dy"], s["x"], s["W"], pre=s["pre"], activation=c["act"],
                               bias_dtype=_DT[c["bias"]] if c["bias"] else None,
                               status=s["status"])


# ------------------------------------------------------------------ plain forms
def _norm_plain(c, s):
    K = c["K"]
    x = s["x"].float()
    mean = x.sum(1) / K
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).sum(1) / K + NORM_EPS)
    y = xc * rstd[:, None] * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    return y.to(_DT[c["y"]]), mean, rstd


def _norm_back_plain(c, s):
    K = c["K"]
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    c1 = g.sum(1, keepdim=True) / K
    c2 = (g * xh).sum(1, keepdim=True) / K
    dx = s["rstd"][:, None] * (g - c1 - xh * c2)
    dw = (dy * xh).sum(0).to(s["w"].dtype)
    return dx.to(s["x"].dtype), dw, dy.sum(0).to(s["w"].dtype) if c["bias"] else None


def _select_plain(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    raw = s["logits"]
    # masked: NaN, -inf and the type's lowest value; +inf counts as the largest
    open_ = raw > torch.finfo(raw.dtype).min
    z = raw.float().clamp(max=torch.finfo(torch.float32).max)
    ninf = torch.full_like(z, -math.inf)
    if c["scoring"] == "softmax":
        zm = torch.where(open_, z, ninf)
        top = zm.max(1, keepdim=True).values
        e = torch.where(open_, torch.exp(z - torch.where(top > -math.inf, top, 0.0)), 0.0)
        tot = e.sum(1, keepdim=True)
        p = e / torch.where(tot > 0, tot, 1.0)
        key = z  # the scores grow with the logits: the same order, without their rounding
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
        key = p if s["bias"] is None else p + s["bias"]
    key = torch.where(open_, key, ninf)
    if c["groups"] > 1:
        G = c["groups"]
        best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        score = best[:, :, 0]
        if c["scoring"] == "sigmoid" and E // G > 1:
            second = best[:, :, 1]
            score = score + torch.where(second > -math.inf, second, 0.0)
        pick = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, pick, True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, ninf)
    key, ids = torch.sort(key, dim=1, descending=True, stable=True)
    key, ids = key[:, :k], ids[:, :k]
    w = torch.where(key > -math.inf, p.gather(1, ids), 0.0)
    if c["renorm"]:
        tot = w.sum(1, keepdim=True)
        w = w / torch.where(tot > 0, tot, 1.0)
    return ids.to(torch.int32), w * c["scale"]


def _select_back_plain(c, s):
    z = s["logits"].float()
    ids, w, g = s["ids"].long(), s["weights"], s["dw"]
    dot = (g * w).sum(1, keepdim=True)
    if c["scoring"] == "softmax":
        if c["renorm"]:
            d = torch.zeros_like(z).scatter_(1, ids, w * (g - dot / c["scale"]))
        else:
            e = torch.exp(z - z.max(1, keepdim=True).values)
            d = (e / e.sum(1, keepdim=True)) * -dot
            d = d.scatter_add(1, ids, w * g)
    else:
        p = 1.0 / (1.0 + torch.exp(-z.gather(1, ids)))
        d = w * (1.0 - p) * ((g - dot / c["scale"]) if c["renorm"] else g)
        d = torch.zeros_like(z).scatter_(1, ids, d)
    return d.to(s["logits"].dtype)


def _linear_plain(c, s):
    z = s["x"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    if c["act"] == "relu":
        out = torch.where(z > 0, z, 0.0)
    elif c["act"] == "silu":
        out = z / (1.0 + torch.exp(-z))
    elif c["act"] == "gelu":
        out = 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    else:
        out = z
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(_DT[c["out"]])
    return (out, z.to(torch.bfloat16)) if c["pre"] else out


def _linear_back_plain(c, s):
    dz = s["dy"].float()
    if c["act"] != "none":
        z = s["pre"].float()
        if c["act"] == "relu":
            dz = torch.where(z > 0, dz, 0.0)
        elif c["act"] == "silu":
            sg = 1.0 / (1.0 + torch.exp(-z))
            dz = dz * (sg * (1.0 + z * (1.0 - sg)))
        else:
            cdf = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
            dz = dz * (cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    dx = (dz @ s["W"].float()).to(torch.bfloat16)
    dW = (dz.t() @ s["x"].float()).to(torch.bfloat16)
    return dx, dW, dz.sum(0).to(_DT[c["bias"]]) if c["bias"] else None


_PLAIN = {("norm", False): _norm_plain, ("norm", True): _norm_back_plain,
          ("select", False): _select_plain, ("select", True): _select_back_plain,
          ("linear", False): _linear_plain, ("linear", True): _linear_back_plain}
_OWN = {("norm", False): _norm_own, ("norm", True): _norm_back_own,
        ("select", False): _select_own, ("select", True): _select_back_own,
        ("linear", False): _linear_own, ("linear", True): _linear_back_own}


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "norm":
        K = c["K"]
        xb, yb, wb = (4 if c[n] == "f32" else 2 for n in ("x", "y", "w"))
        par = K * wb * (2 if c["bias"] else 1)
        if c["back"]:
            # dy, x, the statistics and w in; dx and the two gradients out
            return {"bytes": T * K * (2 * xb + yb) + 8 * T + K * wb + par, "flops": 14 * T * K}
        return {"bytes": T * K * (xb + yb) + 8 * T + par, "flops": 8 * T * K}
    if c["op"] == "select":
        E, k = c["E"], c["k"]
        lb = 4 if c["logits"] == "f32" else 2
        if c["back"]:
            # ids, weights and their gradient in, the whole gradient out; the
            # logits whole, of the chosen only, or not at all
            if c["scoring"] == "softmax":
                seen = 0 if c["renorm"] else E
            else:
                seen = k
            return {"bytes": T * (E * lb + seen * lb + 12 * k), "flops": T * (6 * k + 4 * E)}
        return {"bytes": T * (E * lb + 8 * k) + (4 * E if c["bias"] else 0),
                "flops": T * E * (6 + k)}
    K, N = c["K"], c["N"]
    yb = 4 if c["out"] == "f32" else 2
    if c["back"]:
        b = T * N * (yb + (2 if c["act"] != "none" else 0)) + 2 * (T * K + N * K) * 2
        b += N * (4 if c["bias"] == "f32" else 2) if c["bias"] else 0
        return {"bytes": b, "flops": 4 * T * N * K}
    b = T * N * (yb + (2 if c["pre"] else 0)) + (T * K + N * K) * 2
    b += T * N * (4 if c["residual"] == "f32" else 2) if c["residual"] else 0
    b += N * (4 if c["bias"] == "f32" else 2) if c["bias"] else 0
    return {"bytes": b, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in float64, laid out as run()'s outputs."""
    c = case
    s = prepare(c, seed)
    d = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor)}
    if c["op"] == "norm":
        if not c["back"]:
            var, mean = torch.var_mean(d["x"], 1, correction=0)
            rstd = (var + NORM_EPS).pow(-0.5)
            y = torch.einsum("tk,t,k->tk", d["x"] - mean.unsqueeze(1), rstd, d["w"])
            return (y + d["b"] if "b" in d else y), mean, rstd
        # the gradient of <dy, y> through xh = (x - mean) rstd, where mean and
        # rstd are the given statistics of the row
        K = c["K"]
        xh = (d["x"] - d["mean"].unsqueeze(1)).mul_(d["rstd"].unsqueeze(1))
        dw, db = torch.einsum("tk,tk->k", d["dy"], xh), d["dy"].sum(0)
        g = d["dy"].mul_(d["w"])
        dot = torch.einsum("tk,tk->t", g, xh) / K
        dx = g.sub(g.mean(1, keepdim=True)).sub_(xh.mul_(dot.unsqueeze(1)))
        return dx.mul_(d["rstd"].unsqueeze(1)), dw, db if c["bias"] else None
    if c["op"] == "select":
        return _select_exact(c, s, d)
    x, W = d["x"], d["W"]
    if not c["back"]:
        z = torch.addmm(d["b"], x, W.mT) if "b" in d else torch.mm(x, W.mT)
        out = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
               "gelu": lambda v: v * torch.special.ndtr(v)}[c["act"]](z)
        out = out + d["residual"] if "residual" in d else out
        return (out, z) if c["pre"] else out
    dz = d["dy"]
    if c["act"] != "none":
        z = d["pre"]
        if c["act"] == "relu":
            slope = (z > 0).double()
        elif c["act"] == "silu":
            slope = torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
        else:
            slope = torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
        dz = dz * slope
    return torch.mm(dz, W), torch.mm(dz.mT, x), dz.sum(0) if c["bias"] else None


def _select_exact(c, s, d):
    # the cases' logits are finite: no masks here
    z = d["logits"]
    p = torch.softmax(z, 1) if c["scoring"] == "softmax" else torch.sigmoid(z)
    if not c["back"]:
        key = p + d["bias"] if "bias" in d else p
        if c["groups"] > 1:
            per = key.unflatten(1, (c["groups"], -1))
            n = min(2, per.shape[2]) if c["scoring"] == "sigmoid" else 1
            low = per.topk(n, 2).values.sum(2).topk(c["topk_groups"], 1).values[:, -1:]
            per = per.masked_fill((per.topk(n, 2).values.sum(2) < low).unsqueeze(2), -math.inf)
            key = per.flatten(1)
        w = p.gather(1, key.topk(c["k"], 1).indices)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return None, w * c["scale"]  # the ids are whole numbers, held against the plain form's
    # the weights as a function of the logits, the choice held fixed, and its
    # gradient by the chain rule from the scores
    ids, g = s["ids"].long(), d["dw"]
    chosen = p.gather(1, ids)
    tot = chosen.sum(1, keepdim=True)
    w = chosen / tot if c["renorm"] else chosen
    dp = c["scale"] * g
    if c["renorm"]:
        dp = (dp - (dp * w).sum(1, keepdim=True)) / tot
    full = torch.zeros_like(p).scatter_(1, ids, dp)
    if c["scoring"] == "sigmoid":
        return full * p * (1 - p)
    return p * (full - (full * p).sum(1, keepdim=True))


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(case, work(case))
