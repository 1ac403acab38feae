"""The norms, the MXFP4 linear and the grouped bf16 products: what the C entry
points refuse on the host, before any launch (no GPU needed), and the empty
calls that are no-ops."""
import ctypes

import pytest

vp = ctypes.c_void_p
P = vp(4096)          # a pointer of good alignment; never read: every call here returns before a launch
NULL = None
ODD = vp(4096 + 4)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lmoe():
    from top_routing_mxfp4_gb300 import build
    build.build()
    from top_routing_mxfp4_gb300 import lmoe
    return lmoe


def test_rms_norm_refusals(lmoe):
    def call(x=P, fmt=0, w=P, eps=1e-5, T=4, H=64, out=P):
        return lmoe._rms_norm(x, fmt, w, eps, T, H, out, NULL)

    for bad in (dict(x=NULL), dict(w=NULL), dict(out=NULL), dict(x=ODD), dict(w=ODD), dict(out=ODD), dict(fmt=2),
                dict(fmt=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(T=-1), dict(H=0),
                dict(H=12), dict(H=32776), dict(T=1 << 31)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    assert call(T=0, x=NULL, w=NULL, out=NULL) == lmoe.OK


def test_residual_norm_refusals(lmoe):
    def call(y=P, res=P, fmt=0, post=P, gate=NULL, kind=0, scale=1.0, eps=1e-5, nw=P, T=4, H=64, ro=P, no=P):
        return lmoe._residual_norm(y, res, fmt, post, gate, kind, scale, eps, nw, T, H, ro, no, NULL)

    for bad in (dict(y=NULL), dict(res=NULL), dict(ro=NULL), dict(no=NULL), dict(y=ODD), dict(res=ODD), dict(ro=ODD),
                dict(no=ODD), dict(post=ODD), dict(nw=ODD), dict(kind=4, gate=P), dict(kind=-1, gate=P),
                dict(kind=1), dict(kind=2), dict(kind=3), dict(kind=0, gate=P), dict(kind=3, gate=ODD),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(eps=-1.0), dict(H=20), dict(fmt=7)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    assert call(T=0) == lmoe.OK


def test_linear_mxfp4_refusals(lmoe):
    need = lmoe.linear_mxfp4_workspace_size(64, 256, 96)
    assert need >= 256
    for bad in ((-1, 256, 96), (1, 48, 96), (1, 0, 96), (1, 256, 0), (1 << 31, 256, 96)):
        assert lmoe.linear_mxfp4_workspace_size(*bad) == 0

    def call(x=P, q=P, s=P, rows=64, K=256, N=96, out=P, ws=P, n=need):
        return lmoe._linear_mx(x, q, s, rows, K, N, out, ws, n, NULL)

    for bad in (dict(x=NULL), dict(q=NULL), dict(s=NULL), dict(out=NULL), dict(x=ODD), dict(s=ODD), dict(out=ODD),
                dict(q=vp(4096 + 16)), dict(K=40), dict(K=-32), dict(N=0), dict(rows=-1), dict(rows=1 << 31)):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 64))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
    assert call(rows=0, x=NULL, out=NULL, ws=NULL, n=0) == lmoe.OK


def test_grouped_refusals(lmoe):
    need = lmoe.grouped_workspace_size()

    def groups(offsets=4096, perm=4096, n=64, E=8, k=2):
        return lmoe.Groups(offsets, perm, n, E, k)

    def call(x=P, x_rows=32, W=P, g=None, gather=1, row_w=NULL, K=64, N=40, fmt=0, out=P, ws=P, n=need, swiglu=False):
        g = groups() if g is None else g
        if swiglu:
            return lmoe._grouped_swiglu(x, x_rows, W, W, ctypes.byref(g), gather, K, N, out, ws, n, NULL)
        return lmoe._grouped_linear(x, x_rows, W, ctypes.byref(g), gather, row_w, K, N, fmt, out, ws, n, NULL)

    for sw in (False, True):
        for bad in (dict(x=NULL), dict(W=NULL), dict(out=NULL), dict(x=ODD), dict(W=ODD), dict(out=ODD), dict(K=60),
                    dict(K=0), dict(N=0), dict(x_rows=-1), dict(x_rows=0), dict(g=groups(offsets=None)),
                    dict(g=groups(perm=None)), dict(g=groups(n=-1)), dict(g=groups(E=0)), dict(g=groups(E=2049)),
                    dict(g=groups(k=0)), dict(g=groups(n=1 << 31)), dict(gather=0, x_rows=63),
                    dict(N=1 << 29), dict(x_rows=1 << 31), dict(g=groups(offsets=4098))):
            assert call(swiglu=sw, **bad) == lmoe.ERR_INVALID_ARG, (sw, bad)
        for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 64))):
            assert call(swiglu=sw, **bad) == lmoe.ERR_WORKSPACE, bad
        assert call(swiglu=sw, g=groups(n=0, offsets=None), x=NULL, out=NULL, ws=NULL) == lmoe.OK
    assert call(fmt=2) == lmoe.ERR_INVALID_ARG
    assert lmoe._grouped_linear(P, 32, P, None, 1, NULL, 64, 40, 0, P, P, need, NULL) == lmoe.ERR_INVALID_ARG


def test_residual_block_refusals(lmoe):
    size = lambda D, hidden: lmoe._res_block_ws(ctypes.byref(D), hidden)
    D = lmoe.dims(8, 512, 896, 16, 64)
    need = size(D, 1024)
    assert need > lmoe.workspace_size(8, 512, 896, 16, 64)
    assert size(lmoe.dims(8, 500, 896, 16, 64), 1024) == 0
    for hidden in (0, 1000, -64, 32768 + 64):
        assert size(D, hidden) == 0
    W = lmoe.ExpertWeights(256, 256, 256, 256, 256, 256, lmoe.LAYOUT_TC)
    bf, mx = lmoe.Projection(4096, None, None), lmoe.Projection(None, 4096, 4096)

    def block(inp=bf, out=mx, pre=4096, post=4096, gate=None, kind=0, scale=1.0, eps=1e-5, nw=4096):
        return lmoe.ResidualBlockStruct(inp, out, pre, post, gate, kind, scale, eps, nw)

    def call(res=P, fmt=0, x_n=NULL, b=None, dims=D, hidden=1024, ro=P, no=P, ws=P, n=need, Wr3=P, weights=W):
        b = block() if b is None else b
        return lmoe._res_block(res, fmt, x_n, ctypes.byref(b), Wr3, NULL, ctypes.byref(weights), ctypes.byref(dims), hidden,
                               ro, no, ws, n, NULL)

    for bad in (dict(res=NULL), dict(res=ODD), dict(ro=NULL), dict(ro=ODD), dict(no=NULL), dict(fmt=2), dict(x_n=ODD),
                dict(Wr3=NULL), dict(hidden=1000), dict(hidden=65536), dict(dims=lmoe.dims(8, 500, 896, 16, 64)),
                dict(b=block(pre=None)), dict(b=block(kind=1)), dict(b=block(gate=4096)), dict(b=block(kind=5, gate=4096)),
                dict(b=block(scale=float("nan"))), dict(b=block(eps=-1.0)), dict(b=block(inp=lmoe.Projection(None, 4096, None))),
                dict(b=block(out=lmoe.Projection(None, 4096 + 16, 4096))), dict(b=block(inp=lmoe.Projection(4100, None, None))),
                dict(b=block(post=4100)),
                dict(weights=lmoe.ExpertWeights(256, 256, 256, 256, 256, 256, lmoe.LAYOUT_CANONICAL))):
        assert call(**bad) == lmoe.ERR_INVALID_ARG, bad
    for bad in (dict(ws=NULL), dict(n=need - 1), dict(ws=vp(4096 + 16))):
        assert call(**bad) == lmoe.ERR_WORKSPACE, bad
    assert call(dims=lmoe.dims(8, 512, 896, 16, 64, 2)) == lmoe.ERR_UNSUPPORTED
    assert call(dims=lmoe.dims(0, 512, 896, 16, 64), res=NULL, ro=NULL, ws=NULL) == lmoe.OK


def test_binding_refuses_tensors_off_the_gpu(lmoe):
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.ones(64)
    with pytest.raises(ValueError):
        lmoe.rms_norm(x, w)
    with pytest.raises(ValueError):
        lmoe.residual_norm(x, x)
    with pytest.raises(ValueError):
        lmoe.linear_mxfp4(x, torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8), 4)
    with pytest.raises(ValueError):
        lmoe.grouped_linear_bf16(x, torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32))


def test_linear_workspace_never_shrinks(lmoe):
    # a workspace for the most rows serves every smaller call, whichever tiles it takes
    for K, N in ((96, 512), (1536, 8192), (2048, 8192), (7168, 14336)):
        need = [lmoe.linear_mxfp4_workspace_size(rows, K, N) for rows in range(1, 1200)]
        assert need == sorted(need), (K, N)
