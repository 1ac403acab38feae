"""The linear layer with bias, function and residual, layer norm and the balance loss:
what the C entry points refuse on the host, before any launch (no GPU needed), the empty
calls that are no-ops, and what the binding refuses."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
P = vp(4096)          # a pointer of good alignment; never read: every call here returns before a launch
NULL = None
ODD = vp(4096 + 8)    # not 16-byte aligned
ODD4 = vp(4096 + 2)   # not 4-byte aligned


@pytest.fixture(scope="module")
def lmoe():
    from top_routing_mxfp4_gb300 import build
    build.build()
    from top_routing_mxfp4_gb300 import lmoe
    return lmoe


BAD_SIZES = (dict(rows=-1), dict(rows=(1 << 29) + 1), dict(K=0), dict(K=-8), dict(K=12), dict(N=0), dict(N=-4),
             dict(rows=1 << 29, K=4096), dict(rows=1 << 29, N=4096), dict(K=1 << 22, N=1 << 22))


def test_linear_act_refusals(lmoe):
    size = lambda rows=64, K=256, N=96: lmoe.linear_act_workspace_size(rows, K, N)
    need = size()
    assert need >= 256 and size(rows=0) > 0 and size(rows=1, N=1) > 0
    assert all(size(**b) == 0 for b in BAD_SIZES)

    def call(x=P, W=P, bias=None, bias_fmt=0, fn=1, res=None, res_fmt=0, rows=64, K=256, N=96, fmt=0, out=P, pre=NULL, ws=P,
             n=need, act=True):
        A = lmoe.LinearAct(bias, bias_fmt, fn, res, res_fmt)
        return lmoe._linear_act(x, W, ctypes.byref(A) if act else None, rows, K, N, fmt, out, pre, ws, n, NULL)

    for bad in BAD_SIZES + (dict(x=NULL), dict(W=NULL), dict(out=NULL), dict(x=ODD), dict(W=ODD), dict(out=ODD), dict(pre=ODD),
                            dict(bias=4104), dict(res=4104), dict(fn=-1), dict(fn=5), dict(fmt=2), dict(fmt=-1),
                            dict(bias_fmt=2), dict(res_fmt=-1), dict(res=4096, res_fmt=1), dict(pre=P),
                            dict(pre=vp(8192), res=8192)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 64))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
        assert call(act=False, **bad) == lmoe.ERR_WORKSPACE, bad
    assert call(rows=0, x=NULL, W=NULL, out=NULL, ws=NULL, n=0) == lmoe.OK


def test_linear_act_backward_refusals(lmoe):
    size = lambda rows=64, K=256, N=96: lmoe.linear_act_backward_workspace_size(rows, K, N)
    need = size()
    assert need > 256 and all(size(**b) == 0 for b in BAD_SIZES)

    def call(dout=P, dfmt=0, x=P, W=P, pre=P, fn=1, rows=64, K=256, N=96, dx=P, dW=P, wfmt=0, db=P, ws=P, n=need):
        return lmoe._linear_act_back(dout, dfmt, x, W, pre, fn, rows, K, N, dx, dW, wfmt, db, ws, n, NULL)

    for bad in BAD_SIZES + (dict(dout=NULL), dict(dout=ODD), dict(x=NULL), dict(x=ODD), dict(W=NULL), dict(W=ODD), dict(pre=NULL),
                            dict(pre=ODD), dict(fn=0), dict(fn=7), dict(dfmt=2), dict(wfmt=-1), dict(dx=ODD), dict(dW=ODD),
                            dict(db=ODD)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 128))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
    assert call(dx=NULL, dW=NULL, db=NULL, ws=NULL, n=0) == lmoe.OK
    assert call(rows=0, dout=NULL, x=NULL, W=NULL, pre=NULL, dx=P, dW=NULL, db=NULL, ws=NULL, n=0) == lmoe.OK


NORM_BAD = (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=12), dict(H=32776), dict(fmt=2), dict(fmt=-1))


def test_layer_norm_refusals(lmoe):
    def call(x=P, fmt=0, w=P, b=P, eps=1e-5, T=4, H=64, out=P, mean=P, rstd=P):
        return lmoe._layer_norm(x, fmt, w, b, eps, T, H, out, mean, rstd, NULL)

    for bad in NORM_BAD + (dict(x=NULL), dict(out=NULL), dict(x=ODD), dict(w=ODD), dict(b=ODD), dict(out=ODD), dict(mean=NULL),
                           dict(rstd=NULL), dict(mean=ODD4), dict(rstd=ODD4), dict(eps=-1e-6), dict(eps=float("nan")),
                           dict(eps=float("inf"))):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    assert call(T=0, x=NULL, out=NULL) == lmoe.OK


def test_layer_norm_backward_refusals(lmoe):
    need = lmoe.layer_norm_backward_workspace_size(4, 64)
    assert need > 256 and lmoe.layer_norm_backward_workspace_size(0, 64) > 0
    assert all(lmoe.layer_norm_backward_workspace_size(b.get("T", 4), b.get("H", 64)) == 0 for b in NORM_BAD if "fmt" not in b)

    def call(dy=P, x=P, fmt=0, mean=P, rstd=P, w=P, add=P, T=4, H=64, dx=P, dw=P, db=P, ws=P, n=need):
        return lmoe._layer_norm_back(dy, x, fmt, mean, rstd, w, add, T, H, dx, dw, db, ws, n, NULL)

    for bad in NORM_BAD + (dict(dy=NULL), dict(x=NULL), dict(mean=NULL), dict(rstd=NULL), dict(dx=NULL), dict(dy=ODD), dict(x=ODD),
                           dict(w=ODD), dict(add=ODD), dict(dx=ODD), dict(mean=ODD4), dict(rstd=ODD4), dict(dw=ODD4),
                           dict(db=ODD4)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 128))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
        assert call(db=NULL, **bad) == lmoe.ERR_WORKSPACE, bad
    assert call(T=0, dy=NULL, x=NULL, mean=NULL, rstd=NULL, dx=NULL, dw=NULL, db=NULL, ws=NULL, n=0) == lmoe.OK


def test_balance_loss_refusals(lmoe):
    need = lmoe.balance_loss_workspace_size(64, 96, 4)
    assert need > 256 and lmoe.balance_loss_workspace_size(0, 1, 1) > 0
    sizes = (dict(T=-1), dict(E=0), dict(E=2049), dict(k=0), dict(k=33), dict(E=3, k=4), dict(T=1 << 29))
    assert all(lmoe.balance_loss_workspace_size(b.get("T", 64), b.get("E", 96), b.get("k", 4)) == 0 for b in sizes)

    def call(logits=P, idx=P, mask=NULL, T=64, E=96, k=4, loss=P, counts=P, probs=P, d=4096, cb=1.0, cz=1.0, scale=None,
             w=None, dw=None, ws=P, n=need, grad=True):
        G = lmoe.BalanceGrad(d, cb, cz, scale, w, dw)
        return lmoe._balance(logits, idx, mask, T, E, k, loss, counts, probs, ctypes.byref(G) if grad else None, ws, n, NULL)

    for bad in sizes + (dict(logits=NULL), dict(idx=NULL), dict(loss=NULL), dict(counts=NULL), dict(probs=NULL), dict(d=None),
                        dict(logits=ODD), dict(idx=ODD), dict(loss=ODD), dict(counts=ODD), dict(probs=ODD), dict(d=4104),
                        dict(scale=4098), dict(w=4096), dict(dw=4096), dict(w=4104, dw=4096), dict(w=4096, dw=4104),
                        dict(cb=float("nan")), dict(cz=float("inf")), dict(T=0, loss=NULL)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 128))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
        assert call(grad=False, **bad) == lmoe.ERR_WORKSPACE, bad


def test_the_binding_refuses_host_tensors_and_unknown_functions(lmoe):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    f = torch.zeros(4, 64)
    for call in (lambda: lmoe.linear_act_bf16(x, w), lambda: lmoe.linear_act_bf16(x, w, act="swish"),
                 lambda: lmoe.linear_act_bf16_backward(x, x, w), lambda: lmoe.linear_act_bf16_backward(x, x, w, act=None),
                 lambda: lmoe.layer_norm(x), lambda: lmoe.layer_norm(x[0]), lambda: lmoe.layer_norm_backward(x, x, f, f),
                 lambda: lmoe.balance_loss(f, torch.zeros(4, 2, dtype=torch.int32)), lambda: lmoe.balance_loss(f, None)):
        with pytest.raises(ValueError):
            call()
