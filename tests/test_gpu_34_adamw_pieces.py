"""The 8-bit AdamW step of a large model: from some ten million elements a launch on
a warp takes eight blocks of 256 at a time, their scales a lane each.  The same
tensors one call each (a block a warp) must give the same bits."""
import pytest
import torch

import variable_size_expert_gb300 as mgg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _case(sizes, pt, gt, master, seed, offset):
    """Lists as adamw_step takes them; every third tensor starts off its boundaries."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(n, i, dtype, std):
        o = offset if i % 3 == 1 else 0
        return (torch.randn(n + o, generator=g, device=DEV) * std).to(dtype)[o:]
    p = [rand(n, i, pt, 1.0) for i, n in enumerate(sizes)]
    grads = [rand(n, i, gt, 1e-2) for i, n in enumerate(sizes)]
    m, v, ms, vs = mgg.adamw_state(p, 8)
    for t, s, top in ((m, ms, 255), (v, vs, 127)):
        for i, n in enumerate(sizes):
            o = offset if i % 3 == 1 else 0
            codes = torch.randint(0, top, (n + o,), generator=g, device=DEV, dtype=torch.uint8)
            codes[codes & 0x7F == 0x7F] = 0x7E  # (0x7F is NaN)
            t[i] = codes[o:].view(torch.float8_e4m3fn)
            s[i].copy_(1e-5 * (0.5 + torch.rand(s[i].shape, generator=g, device=DEV)))
    masters = [x.float() for x in p] if master else None
    return p, grads, m, v, ms, vs, masters


def _clone(case):
    return [None if l is None else [t.clone() for t in l] for l in case]


def _step(case, at):
    p, g, m, v, ms, vs, w = ([None if l is None else l[i] for i in at] if l is not None else None for l in case)
    mgg.adamw_step(p, g, m, v, 7, lr=1e-2, betas=(0.9, 0.99), weight_decay=0.1, masters=w, exp_avg_scale=ms,
                   exp_avg_sq_scale=vs)


# more than 8 * 32 blocks an SM: one large tensor among ragged ones; tensors of a launch
# with the small table (24) and with the large one; last pieces of one to eight blocks,
# last blocks of one to 256 elements
SIZES = {
    "few": [9_000_001, 2048 * 400, 2048 * 400 + 1, 256 * 1027, 300_007, 2047, 2049, 5, 256],
    "many": [290_000 + 311 * i for i in range(44)] + [1, 255, 257, 1792, 1793],
}


@pytest.mark.parametrize("sizes", sorted(SIZES))
@pytest.mark.parametrize("pt,gt,master", [(torch.float32, torch.bfloat16, False),
                                          (torch.bfloat16, torch.float32, True)])
def test_pieces_of_eight_blocks(sizes, pt, gt, master):
    sizes = SIZES[sizes]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-n // 256) for n in sizes) >= 8 * 32 * sms > max(-(-n // 256) for n in sizes)
    case = _case(sizes, pt, gt, master, len(sizes), 3)
    alone = _clone(case)
    # (a copy starts on its boundary: the elements' order in a lane is another, their
    # arithmetic is not)
    for i in range(len(sizes)):
        _step(alone, [i])
    _step(case, range(len(sizes)))
    for name, a, b in zip(("p", "g", "m", "v", "ms", "vs", "master"), case, alone):
        for i, n in enumerate(sizes if a is not None else []):
            x, y = a[i], b[i]
            if x.dtype == torch.float8_e4m3fn:
                x, y = x.view(torch.uint8), y.view(torch.uint8)
            assert torch.equal(x, y), (name, i, n)
