"""Refusals of the layers around the experts, checked before the device is
touched: the C ABI's status codes, and the exceptions of the torch API on CPU
tensors."""
import ctypes
import math
import os

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    from variable_size_expert_gb300 import _lib, build
    if not (os.path.exists(_lib.LIB_PATH) and os.path.exists(build.HOST)):
        g.build()
    return _lib.load()


FAKE = 0x10000      # never dereferenced: the checks fail first


def _norm(lib, x=FAKE, xd=0, ldx=64, w=FAKE, b=None, wd=0, T=4, K=64, eps=1e-5, y=FAKE, yd=0, mean=FAKE,
          rstd=FAKE):
    return lib.mgg_layer_norm_forward(x, xd, ldx, w, b, wd, T, K, eps, y, yd, mean, rstd, None)


def test_layer_norm_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al, dt = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT, L.MGG_ERR_DTYPE
    for kw, want in ((dict(x=None), inv), (dict(w=None), inv), (dict(y=None), inv), (dict(mean=None), inv),
                     (dict(rstd=None), inv), (dict(T=-1), inv), (dict(K=0), inv), (dict(ldx=63), inv),
                     (dict(eps=-1.0), inv), (dict(eps=math.nan), inv), (dict(eps=math.inf), inv),
                     (dict(xd=2), dt), (dict(wd=9), dt), (dict(yd=2), dt), (dict(x=FAKE + 1), al),
                     (dict(xd=1, x=FAKE + 2), al), (dict(b=FAKE + 1), al), (dict(yd=1, y=FAKE + 2), al)):
        assert _norm(lib, **kw) == want, kw
    assert _norm(lib, T=0, x=None, y=None) == L.MGG_OK

    def back(dy=FAKE, x=FAKE, w=FAKE, mean=FAKE, T=4, K=64, ldx=64, dx=FAKE, dw=FAKE, db=None):
        return lib.mgg_layer_norm_backward(dy, 0, x, 0, ldx, w, 0, mean, FAKE, T, K, dx, dw, db, FAKE, 1 << 30,
                                           None)
    for kw, want in ((dict(dy=None), inv), (dict(dx=None), inv), (dict(dw=None), inv), (dict(mean=None), inv),
                     (dict(T=-1), inv), (dict(K=0), inv), (dict(ldx=8), inv), (dict(dx=FAKE + 1), al),
                     (dict(db=FAKE + 1), al)):
        assert back(**kw) == want, kw
    assert lib.mgg_workspace_bytes(L.MGG_OP_LAYER_NORM_BACKWARD, 0, 0, 0, 0, 64, 0) == 0


def _select(lib, l=FAKE, d=1, ldl=16, T=4, E=16, k=2, sc=0, bias=None, G=1, tg=1, scale=1.0, ids=FAKE, w=FAKE):
    return lib.mgg_select_experts(l, d, ldl, T, E, k, sc, bias, G, tg, 1, scale, ids, w, None)


def test_select_experts_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al, dt = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT, L.MGG_ERR_DTYPE
    for kw, want in ((dict(l=None), inv), (dict(ids=None), inv), (dict(w=None), inv), (dict(T=-1), inv),
                     (dict(E=0), inv), (dict(E=1025, ldl=1025), inv), (dict(k=0), inv), (dict(k=17), inv),
                     (dict(E=64, ldl=64, k=33), inv), (dict(ldl=15), inv), (dict(sc=2), inv),
                     (dict(G=3), inv), (dict(G=0), inv), (dict(G=4, tg=0), inv), (dict(G=4, tg=5), inv),
                     (dict(G=4, tg=1, k=5), inv), (dict(E=64, ldl=64, G=64), inv),
                     (dict(scale=0.0), inv), (dict(scale=-1.0), inv), (dict(scale=math.nan), inv),
                     (dict(scale=math.inf), inv), (dict(d=2), dt), (dict(l=FAKE + 2), al),
                     (dict(bias=FAKE + 2), al), (dict(ids=FAKE + 1), al)):
        assert _select(lib, **kw) == want, kw
    assert _select(lib, T=0, l=None, ids=None, w=None) == L.MGG_OK

    def back(g=FAKE, l=FAKE, ids=FAKE, k=2, sc=0, scale=1.0, d=FAKE, st=FAKE):
        return lib.mgg_select_experts_backward(g, l, 1, 16, ids, FAKE, 4, 16, k, sc, 1, scale, d, st, None)
    for kw, want in ((dict(g=None), inv), (dict(l=None), inv), (dict(ids=None), inv), (dict(d=None), inv),
                     (dict(st=None), inv), (dict(k=0), inv), (dict(sc=7), inv), (dict(scale=0.0), inv),
                     (dict(d=FAKE + 2), al)):
        assert back(**kw) == want, kw


def _linear(lib, x=FAKE, ldx=64, W=FAKE, b=None, bd=0, r=None, rd=0, ldr=24, T=4, K=64, N=24, act=0, out=FAKE,
            od=0, pre=None, st=FAKE):
    return lib.mgg_linear_forward(x, ldx, W, b, bd, r, rd, ldr, T, K, N, act, out, od, pre, st, None)


def test_linear_refusals(lib):
    from variable_size_expert_gb300 import _lib as L
    inv, al, dt = L.MGG_ERR_INVALID_ARG, L.MGG_ERR_ALIGNMENT, L.MGG_ERR_DTYPE
    for kw, want in ((dict(x=None), inv), (dict(W=None), inv), (dict(out=None), inv), (dict(st=None), inv),
                     (dict(T=-1), inv), (dict(K=0), inv), (dict(N=0), inv), (dict(ldx=56), inv),
                     (dict(r=FAKE, ldr=23), inv), (dict(act=4), inv), (dict(act=-1), inv),
                     (dict(od=2), dt), (dict(b=FAKE, bd=2), dt), (dict(r=FAKE, rd=2), dt),
                     (dict(K=60), al), (dict(ldx=68), al), (dict(x=FAKE + 8), al), (dict(W=FAKE + 8), al),
                     (dict(out=FAKE + 1), al), (dict(od=1, out=FAKE + 2), al), (dict(b=FAKE + 1), al),
                     (dict(r=FAKE + 1), al), (dict(pre=FAKE + 1), al)):
        assert _linear(lib, **kw) == want, kw
    assert _linear(lib, T=0, x=None, out=None) == L.MGG_OK

    def back(dy=FAKE, dyd=0, lddy=24, x=FAKE, W=FAKE, pre=None, act=0, T=4, K=64, N=24, dx=FAKE, dW=FAKE,
             db=None, st=FAKE):
        return lib.mgg_linear_backward(dy, dyd, lddy, x, K, W, pre, act, T, K, N, dx, dW, db, 0, st, FAKE,
                                       1 << 30, None)
    for kw, want in ((dict(dy=None), inv), (dict(x=None), inv), (dict(W=None), inv), (dict(st=None), inv),
                     (dict(act=3), inv), (dict(act=9), inv), (dict(T=-1), inv), (dict(lddy=23), inv),
                     (dict(dyd=2), dt), (dict(K=60), al), (dict(dx=FAKE + 8), al), (dict(dW=FAKE + 8), al),
                     (dict(dy=FAKE + 1), al), (dict(db=FAKE + 1), al)):
        assert back(**kw) == want, kw
    assert lib.mgg_workspace_bytes(L.MGG_OP_LINEAR_BACKWARD, 0, 0, 0, 64, 0, 0) == 0
    # dz and at least one partial row of the bias gradient
    assert lib.mgg_workspace_bytes(L.MGG_OP_LINEAR_BACKWARD, 100, 0, 0, 60, 0, 0) >= 100 * 64 * 2 + 60 * 4


def test_torch_api_refusals(lib):
    import variable_size_expert_gb300 as mgg
    x, b = torch.zeros(4, 64), torch.zeros(4, 64).bfloat16()
    st = torch.zeros(1, dtype=torch.int32)
    cases = [
        (ValueError, lambda: mgg.layer_norm_forward(x, x[0])),                       # not on a GPU
        (TypeError, lambda: mgg.layer_norm_forward([1.0], x[0])),
        (ValueError, lambda: mgg.select_experts(x, 2)),
        (ValueError, lambda: mgg.select_experts(x, 2, scoring="tanh")),
        (ValueError, lambda: mgg.linear_forward(b, b, activation="tanh", status=st)),
        (TypeError, lambda: mgg.linear_forward(x, b, status=st)),                    # not bfloat16
        (ValueError, lambda: mgg.linear_forward(b, b, status=st)),
        (TypeError, lambda: mgg.linear_backward(x, x, x, status=st)),
        (ValueError, lambda: mgg.select_experts_backward(x[:, :2], x, torch.zeros(4, 2), x[:, :2], status=st)),
    ]
    for want, f in cases:
        with pytest.raises(want):
            f()
