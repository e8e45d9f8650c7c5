"""Cases of the operators that a training step needs around the block: the
balance loss of the gate with the experts' counts, the cross entropy over a
large vocabulary straight from the last hidden states, and the AdamW step over
all of a model's tensors.  Losses forward and backward.

``own`` False computes them in plain torch operations in float32, rounded
once at the end; ``own`` True makes the library's calls.
"""
import math
import random

import torch

own = False

IGNORE = -100  # the target of a token that does not count
LR, BETAS, EPS, DECAY = 3e-4, (0.9, 0.95), 1e-8, 0.1
BLOCK = 256    # elements that share a scale of the 8-bit states


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a small gate of a short batch: latency
        _bal("balance_small", T=512, E=8, k=2),
        # a long batch of padded sequences, sigmoid scores, a loss for each sequence
        _bal("balance_sequences", T=16384, E=256, k=8, scoring="sigmoid", sequences=8, mask=True),
        # gradient at the step's usual token count
        _bal("balance_backward", T=4096, E=64, k=8, logits="bf16", back=True),
        # ragged: token and expert counts that divide by nothing, padded
        _bal("balance_backward_odd", T=16381, E=251, k=6, scoring="sigmoid", mask=True, back=True),
        # the loss of a few tokens: reads the vocabulary's weights once
        _ce("vocab_few", T=16, K=2048, V=32768),
        # the loss of a training batch, a tenth of its tokens ignored
        _ce("vocab_train", T=8192, K=2048, V=32768, ignored=0.1),
        # its gradients at the step's usual token count
        _ce("vocab_backward", T=4096, K=2048, V=32768, ignored=0.1, back=True),
        # ragged: per-token losses with a penalty on the normaliser, odd vocabulary
        _ce("vocab_backward_odd", T=1111, K=1160, V=50257, reduction="none", z_loss=1e-4, back=True),
        # the norms and biases of a block: a few small tensors, latency
        _adam("adamw_small", tensors=12, n=30_000, p="f32", g="f32"),
        # a block's weights in bfloat16 with float32 masters, gradients clipped
        _adam("adamw_master", tensors=16, n=60_000_000, p="bf16", g="bf16", master=True, scale=True),
        # the largest: 8-bit states
        _adam("adamw_8bit", tensors=16, n=120_000_000, p="f32", g="bf16", bits=8),
        # many ragged tensors, 8-bit states, bfloat16 weights alone
        _adam("adamw_8bit_ragged", tensors=200, n=3_000_000, p="bf16", g="f32", bits=8),
    ]


def _bal(name, T, E, k, scoring="softmax", logits="f32", sequences=1, mask=False, back=False):
    return dict(name=name, op="balance", T=T, E=E, k=k, scoring=scoring, logits=logits,
                sequences=sequences, mask=mask, back=back)


def _ce(name, T, K, V, ignored=0.0, reduction="mean", z_loss=0.0, back=False):
    return dict(name=name, op="vocab", T=T, K=K, V=V, ignored=ignored, reduction=reduction,
                z_loss=z_loss, back=back)


def _adam(name, tensors, n, p, g, master=False, bits=32, scale=False):
    return dict(name=name, op="adamw", tensors=tensors, n=n, p=p, g=g, master=master, bits=bits,
                scale=scale, back=False)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "vocab", "adamw"])
    back = rng.random() < 0.5
    if kind == "balance":
        T, E = _log(rng, 1, 16384), _log(rng, 4, 1024)
        while T * E > 16384 * 256:
            T = _log(rng, 1, 16384)
        sequences = rng.choice([1, 1, 2, 4])
        T = max(1, T // sequences) * sequences
        c = _bal("", T, E, rng.randint(1, min(8, E)), rng.choice(["softmax", "sigmoid"]),
                 rng.choice(["f32", "bf16"]), sequences, rng.random() < 0.5, back)
    elif kind == "vocab":
        K = max(64, _log(rng, 64, 4096) // 8 * 8)
        V = _log(rng, 512, 131072)
        if rng.random() < 0.5:
            V = max(512, V // 128 * 128)
        T = _log(rng, 1, 8192)
        while T * K * V * (3 if back else 1) > 8192 * 2048 * 32768 or T * V > 8192 * 32768:
            T = _log(rng, 1, 8192)
        # at least one token of a mean counts
        c = _ce("", T, K, V, rng.choice([0.0, 0.1, 0.5]) if T > 16 else 0.0,
                rng.choice(["mean", "mean", "sum", "none"]), rng.choice([0.0, 0.0, 1e-4]), back)
    else:
        tensors = _log(rng, 1, 300)
        n = max(tensors, _log(rng, 1000, 60_000_000))
        p = rng.choice(["f32", "bf16"])
        c = _adam("", tensors, n, p, rng.choice(["f32", "bf16"]), p == "bf16" and rng.random() < 0.5,
                  rng.choice([8, 32]), rng.random() < 0.5)
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
    # the word that the library's kernels report errors in, kept by the program
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    {"balance": _prepare_balance, "vocab": _prepare_vocab, "adamw": _prepare_adamw}[c["op"]](c, g, s)
    return s


def _prepare_balance(c, g, s):
    T, E, k, B = c["T"], c["E"], c["k"], c["sequences"]
    # logits of a trained gate: some experts liked more than others
    s["logits"] = (1.5 * torch.randn(T, E, generator=g, device="cuda")
                   + 0.5 * torch.randn(E, generator=g, device="cuda")).to(_DT[c["logits"]])
    s["ids"] = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
    s["mask"] = None
    if c["mask"]:  # sequences padded at their end, each to a length of its own
        length = (T // B * (0.5 + 0.5 * torch.rand(B, generator=g, device="cuda"))).ceil()
        s["mask"] = (torch.arange(T // B, device="cuda")[None, :] < length[:, None]).flatten()
    if c["back"]:
        s["dloss"] = torch.full((), 0.01, device="cuda")
        s["slope"] = _balance_plain(c, s)[2]


def _prepare_vocab(c, g, s):
    T, K, V = c["T"], c["K"], c["V"]
    s["W"] = _randn(g, V, K, dtype="bf16", std=1.0 / math.sqrt(K))
    # tokens of a text: the frequent ones most of the time
    s["targets"] = (torch.exp(torch.rand(T, generator=g, device="cuda") * math.log(V)) - 1.0).long().clamp(0, V - 1)
    # hidden states that point to their target's row, some more than others
    sure = 12.0 * torch.rand(T, 1, generator=g, device="cuda")
    s["x"] = (torch.randn(T, K, generator=g, device="cuda") + sure * s["W"][s["targets"]].float()).to(torch.bfloat16)
    if c["ignored"]:
        off = torch.rand(T, generator=g, device="cuda") < c["ignored"]
        off[0] = False
        s["targets"] = torch.where(off, IGNORE, s["targets"])
    if c["back"]:
        s["dloss"] = _randn(g, T) if c["reduction"] == "none" else torch.ones((), device="cuda")
        _, s["lse"], s["weight"] = _vocab_plain(c, s)


def _sizes(c):
    """The tensors' sizes: matrices, and vectors beside them."""
    r = random.Random(c["n"])
    w = [r.uniform(0.5, 1.5) * (1.0 if i % 3 else 0.02) for i in range(c["tensors"])]
    return [max(1, int(c["n"] * x / sum(w))) for x in w]


def _prepare_adamw(c, g, s):
    # one buffer of each kind, every tensor at a boundary of 256 elements; the
    # elements between two tensors are zeros
    sizes = _sizes(c)
    room = [-(-m // BLOCK) * BLOCK for m in sizes]
    starts, n = [sum(room[:i]) for i in range(len(room))], sum(room)
    s["index"] = torch.cat([torch.arange(r, device="cuda") for r in room])
    inside = s["index"] < torch.cat([torch.full((r,), m, device="cuda") for m, r in zip(sizes, room)])

    def flat(std, dtype="f32"):
        return torch.where(inside, _randn(g, n, std=std), 0.0).to(_DT[dtype])

    def split(t, per=1):
        return [t[a // per:a // per + -(-m // per)] for a, m in zip(starts, sizes)]

    w = flat(0.02)
    # gradients of unequal size, and the moments of earlier ones
    size = 1e-3 * torch.exp(torch.randn(n, generator=g, device="cuda"))
    m = flat(0.3) * size
    v = torch.where(inside, (size * (0.7 + 0.6 * torch.rand(n, generator=g, device="cuda"))).square(), 0.0)
    f = s["flat"] = {"p": w.to(_DT[c["p"]]), "g": (flat(1.0) * size).to(_DT[c["g"]])}
    f["master"] = w if c["master"] else None
    if c["bits"] == 8:
        f["m"], f["ms"] = _state8(m)
        f["v"], f["vs"] = _state8(v.sqrt())
    else:
        f["m"], f["v"], f["ms"], f["vs"] = m, v, None, None
    s["lists"] = {k: None if t is None else split(t, BLOCK if k in ("ms", "vs") else 1) for k, t in f.items()}
    s["scale"] = torch.full((1,), 0.37, device="cuda") if c["scale"] else None
    s["step"] = 100


def _state8(x):
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1) / 448.0
    return (b / torch.where(scale > 0, scale, 1.0)[:, None]).to(torch.float8_e4m3fn).view(-1), scale


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["case"]
    if own:
        return _OWN[c["op"], c["back"]](c, state)
    return _PLAIN[c["op"], c["back"]](c, state)


def _balance_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.balance_loss_forward(s["logits"], s["ids"], scoring=c["scoring"], mask=s["mask"],
                                    sequences=c["sequences"], status=s["status"])


def _balance_back_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.balance_loss_backward(s["dloss"], s["logits"], s["slope"], scoring=c["scoring"], mask=s["mask"])


def _vocab_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.linear_cross_entropy_forward(s["x"], s["W"], s["targets"], ignore_index=IGNORE,
                                            reduction=c["reduction"], z_loss=c["z_loss"], status=s["status"])


def _vocab_back_own(c, s):
    import variable_size_expert_gb300 as mgg
    return mgg.linear_cross_entropy_backward(s["dloss"], s["x"], s["W"], s["targets"], s["lse"], s["weight"],
                                             ignore_index=IGNORE, z_loss=c["z_loss"], status=s["status"])


def _adamw_own(c, s):
    import variable_size_expert_gb300 as mgg
    s["step"] += 1
    t = s["lists"]
    mgg.adamw_step(t["p"], t["g"], t["m"], t["v"], s["step"], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY,
                   masters=t["master"], exp_avg_scale=t["ms"], exp_avg_sq_scale=t["vs"], grad_scale=s["scale"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    f = s["flat"]
    return f["p"], f["master"], f["m"], f["v"], f["ms"], f["vs"]


# ------------------------------------------------------------------ plain forms
def _scores(c, z):
    """The probabilities, and for sigmoid scores the scores themselves."""
    if c["scoring"] == "softmax":
        e = torch.exp(z - z.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), None
    a = 1.0 / (1.0 + torch.exp(-z))
    return a / a.sum(1, keepdim=True), a


def _counted(c, s):
    """[T] float: 1 for a token that counts."""
    T = c["T"]
    return torch.ones(T, device=s["logits"].device) if s["mask"] is None else s["mask"].float()


def _balance_plain(c, s):
    T, E, k, B = c["T"], c["E"], c["k"], c["sequences"]
    p, _ = _scores(c, s["logits"].float())
    on = _counted(c, s)
    seq = torch.arange(T, device=p.device) // (T // B)
    slot = (seq[:, None] * E + s["ids"].long()).flatten()
    counts = torch.zeros(B * E, dtype=torch.int32, device=p.device)
    counts.index_add_(0, slot, on.int()[:, None].expand(T, k).reshape(-1))
    counts = counts.view(B, E)
    n = on.view(B, -1).sum(1)
    used = (n > 0).float().sum()
    some = torch.where(n > 0, n, 1.0)
    slope = counts.float() * (E / k) / (some * some)[:, None] / torch.where(used > 0, used, 1.0)
    loss = (slope * (p * on[:, None]).view(B, -1, E).sum(1)).sum()
    return loss, counts, slope


def _balance_back_plain(c, s):
    T, E, B = c["T"], c["E"], c["sequences"]
    p, a = _scores(c, s["logits"].float())
    g = s["slope"].repeat_interleave(T // B, 0)
    d = p * (g - (p * g).sum(1, keepdim=True))
    if a is not None:
        d = d * (1.0 - a)
    return (d * (s["dloss"] * _counted(c, s))[:, None]).to(s["logits"].dtype)


def _vocab_plain(c, s):
    t = s["targets"]
    z = s["x"].float() @ s["W"].float().t()
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    on = t != IGNORE
    losses = lse - z.gather(1, torch.where(on, t, 0)[:, None])[:, 0] + c["z_loss"] * lse * lse
    losses = torch.where(on, losses, 0.0)
    weight = torch.ones(1, device=z.device)
    if c["reduction"] == "none":
        return losses, lse, weight
    if c["reduction"] == "mean":
        weight = 1.0 / on.float().sum().clamp(min=1.0).view(1)
    return losses.sum() * weight[0], lse, weight


def _vocab_back_plain(c, s):
    t, lse = s["targets"], s["lse"]
    x, W = s["x"].float(), s["W"].float()
    p = torch.exp(x @ W.t() - lse[:, None])
    on = t != IGNORE
    d = p * (1.0 + 2.0 * c["z_loss"] * lse)[:, None]
    d = d.scatter_add(1, torch.where(on, t, 0)[:, None], torch.full_like(lse, -1.0)[:, None])
    d = d * torch.where(on, s["dloss"] * s["weight"], 0.0)[:, None]
    return (d @ W).to(torch.bfloat16), (d.t() @ x).to(torch.bfloat16)


def _adamw_plain(c, s):
    s["step"] += 1
    f, t = s["flat"], s["step"]
    b1, b2 = BETAS
    g = f["g"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    if c["bits"] == 8:
        m = (f["m"].float().view(-1, BLOCK) * f["ms"][:, None]).view(-1)
        r = (f["v"].float().view(-1, BLOCK) * f["vs"][:, None]).view(-1)
        m = m * b1 + g * (1.0 - b1)
        r = torch.sqrt((r * r) * b2 + (g * g) * (1.0 - b2))
        f["m"].copy_(_encode8(m, f["ms"], s["index"], t, 0, False))
        f["v"].copy_(_encode8(r, f["vs"], s["index"], t, 1 << 31, True))
    else:
        m = f["m"].mul_(b1).add_(g * (1.0 - b1))
        r = torch.sqrt(f["v"].mul_(b2).add_((g * g) * (1.0 - b2)))
    p = f["p"] if f["master"] is None else f["master"]
    u = (m / (1.0 - b1 ** t)) / (r / math.sqrt(1.0 - b2 ** t) + EPS)
    p.copy_(p.float() * (1.0 - LR * DECAY) - u * LR)
    if f["master"] is not None:
        f["p"].copy_(p)
    return _adamw_outputs(s)


# Rounding to 8 bits: an element's threshold walks a Weyl sequence over the
# steps, so that changes of less than a step of the code add up over them.
_WALK_I, _WALK_T = 0x9E3779B1, 0xC13FA9A9


def _encode8(x, scale, index, t, salt, floor):
    """x in blocks to e4m3 values; ``scale`` receives the blocks' factors.
    ``floor``: what is not zero does not become zero."""
    top = x.view(-1, BLOCK).abs().amax(1)
    full = torch.full_like(top, 448.0)
    scale.copy_(top / full)
    inv = torch.where(top > 2.0 ** -110, full / top, 0.0)
    # the bits of |x| / scale as a float of 4 exponent and 3 mantissa bits, and 20 below them
    y = (x.abs().view(-1, BLOCK) * inv[:, None]).view(-1) * 2.0 ** -120
    u = (index * _WALK_I + (t * _WALK_T + salt)) & 0xFFFFFFFF
    code = ((y.view(torch.int32) + (u >> 12).int()) >> 20).clamp(max=0x7E)
    if floor:
        code = torch.where(y > 0, code.clamp(min=1), code)
    return (code.to(torch.uint8) | torch.where(x < 0, 0x80, 0).to(torch.uint8)).view(torch.float8_e4m3fn)


_PLAIN = {("balance", False): _balance_plain, ("balance", True): _balance_back_plain,
          ("vocab", False): _vocab_plain, ("vocab", True): _vocab_back_plain, ("adamw", False): _adamw_plain}
_OWN = {("balance", False): _balance_own, ("balance", True): _balance_back_own,
        ("vocab", False): _vocab_own, ("vocab", True): _vocab_back_own, ("adamw", False): _adamw_own}


# ------------------------------------------------------------------ the work
def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k, B = c["T"], c["E"], c["k"], c["sequences"]
        lb = 4 if c["logits"] == "f32" else 2
        mask = T if c["mask"] else 0
        if c["back"]:
            return {"bytes": 2 * T * E * lb + mask + 4 * B * E, "flops": 8 * T * E}
        return {"bytes": T * (E * lb + 4 * k) + mask + 8 * B * E, "flops": 5 * T * E}
    if c["op"] == "vocab":
        T, K, V = c["T"], c["K"], c["V"]
        one = 2 * (T * K + V * K)
        if c["back"]:
            # the logits, not kept, are computed again; then the two products
            return {"bytes": 2 * one + 12 * T, "flops": 6 * T * K * V}
        return {"bytes": one + 12 * T, "flops": 2 * T * K * V}
    n = c["n"]
    pb, gb = (4 if c[k] == "f32" else 2 for k in ("p", "g"))
    weights = (8 + pb) if c["master"] else 2 * pb
    states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (weights + gb + states), "flops": 15 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in float64, laid out as run()'s outputs."""
    c = case
    s = prepare(c, seed)
    if c["op"] == "balance":
        return _balance_exact(c, s)
    if c["op"] == "vocab":
        return _vocab_exact(c, s)
    return _adamw_exact(c, s)


def _balance_exact(c, s):
    B, E, k = c["sequences"], c["E"], c["k"]
    z = s["logits"].double()
    a = torch.sigmoid(z)
    p = torch.softmax(z, 1) if c["scoring"] == "softmax" else a / a.sum(1, keepdim=True)
    on = torch.ones_like(z[:, 0]) if s["mask"] is None else s["mask"].double()
    if c["back"]:
        g = s["slope"].double()[torch.arange(c["T"], device=z.device).div(c["T"] // B, rounding_mode="floor")]
        inner = torch.einsum("te,te->t", p, g).unsqueeze(1)
        slope = (p - p * a) if c["scoring"] == "sigmoid" else p
        return torch.einsum("te,t->te", slope * (g - inner), on * s["dloss"].double())
    hits = torch.nn.functional.one_hot(s["ids"].long(), E).sum(1).double() * on.unsqueeze(1)
    counts = hits.unflatten(0, (B, -1)).sum(1)
    n = on.unflatten(0, (B, -1)).sum(1)
    live = max(1, int((n > 0).sum()))
    n = n.clamp(min=1.0).unsqueeze(1)
    share = counts * E / (k * n)
    mean = (p * on.unsqueeze(1)).unflatten(0, (B, -1)).sum(1) / n
    return (share * mean).sum() / live, None, share / n / live


def _vocab_exact(c, s):
    x, W, t = s["x"].double(), s["W"].double(), s["targets"]
    z = torch.mm(x, W.mT)
    on = (t >= 0).double()
    if not c["back"]:
        lse = torch.logsumexp(z, 1)
        rows = torch.arange(len(t), device=z.device)
        losses = on * (lse - z[rows, t.clamp(min=0)] + c["z_loss"] * lse.square())
        one = torch.ones(1, dtype=torch.float64, device=z.device)
        if c["reduction"] == "none":
            return losses, lse, one
        w = one / on.sum() if c["reduction"] == "mean" else one
        return losses.sum() * w.squeeze(0), lse, w
    # the given statistics define the probabilities
    lse = s["lse"].double()
    p = z.sub_(lse.unsqueeze(1)).exp_()
    p.mul_((1.0 + 2.0 * c["z_loss"] * lse).unsqueeze(1))
    p[torch.arange(len(t), device=p.device), t.clamp(min=0)] -= 1.0
    p.mul_((on * s["dloss"].double() * s["weight"].double()).unsqueeze(1))
    return torch.mm(p, W), torch.mm(p.mT, x)


def _adamw_exact(c, s):
    f, t = s["flat"], s["step"] + 1
    b1, b2 = BETAS
    g = f["g"].double() * (1.0 if s["scale"] is None else s["scale"].double())
    if c["bits"] == 8:
        m = (f["m"].double().unflatten(0, (-1, BLOCK)) * f["ms"].double().unsqueeze(1)).flatten()
        v = (f["v"].double().unflatten(0, (-1, BLOCK)) * f["vs"].double().unsqueeze(1)).flatten().square()
    else:
        m, v = f["m"].double(), f["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g.square()
    p = (f["p"] if f["master"] is None else f["master"]).double()
    p = p - LR * DECAY * p - LR * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
    master = None if f["master"] is None else p
    if c["bits"] == 32:
        return p, master, m, v, None, None
    m, ms = _grid8(m, s["index"], t, 0, False)
    r, rs = _grid8(v.sqrt(), s["index"], t, 0x80000000, True)
    return p, master, m, r, ms, rs


def _grid8(x, index, t, salt, floor):
    """x onto the e4m3 values of its blocks: down to the grid after adding the
    element's share of a step (2^-9 below 2^-6, else 2^-3 of the power of two)."""
    b = x.unflatten(0, (-1, BLOCK))
    scale = b.abs().amax(1) / 448
    q = (b.abs() / torch.where(scale > 0, scale, 1.0).unsqueeze(1)).flatten()
    step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
    share = (((index * _WALK_I + t * _WALK_T + salt) % 2 ** 32) // 4096).double() / 2 ** 20
    q = (torch.floor(q / step + share) * step).clamp(max=448.0)
    if floor:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
    return torch.copysign(q, x), scale


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(case, work(case))
