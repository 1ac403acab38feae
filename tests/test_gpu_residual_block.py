"""The operators run together: the block on a residual stream (norm, MXFP4 or
bf16 projections, the layer, norm with gate and residual add), and the bf16
experts between router, permute and combine."""
import numpy as np
import pytest
import torch

import lmoe_inputs as gen
from _util import device_bank, to_dev_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D = torch.float64
U, HALF = 2.0 ** -24, 2.0 ** -8


def _layer(lmoe):
    wl = gen.WORKLOADS["tiny"]
    return lmoe.Layer(torch.from_numpy(gen.router_f32(wl)).to(DEV), device_bank(wl, DEV), k=wl.k), wl


def _block(lmoe, layer, wl, hidden, mx, g):
    W_in = torch.randn(wl.d, hidden, device=DEV, generator=g) * hidden ** -0.5
    W_out = torch.randn(hidden, wl.d, device=DEV, generator=g) * wl.d ** -0.5
    vec = lambda: 1 + 0.1 * torch.randn(hidden, device=DEV, generator=g)
    conv = lmoe.LinearMxfp4 if mx else (lambda W: W.to(torch.bfloat16))
    return lmoe.ResidualBlock(layer, conv(W_in), conv(W_out), pre_w=vec(), post_w=vec(), gate=vec(), scale=0.4)


def _by_hand(lmoe, b, res, x_n, gate, next_w):
    """The block, call by call."""
    lin = lambda W, x: W.forward(x) if isinstance(W, lmoe.LinearMxfp4) else lmoe.linear_bf16(x, W)
    n = lmoe.rms_norm(res, b.pre_w, b.eps) if x_n is None else x_n
    o = lin(b.W_out, b.layer.forward(lin(b.W_in, n)))
    return lmoe.residual_norm(o, res, post_w=b.post_w, gate=b.gate if gate is None else gate, scale=b.scale,
                              next_w=next_w, eps=b.eps)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T", [1, 8, 70])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_block_is_its_calls(cuda_lib, mx, T, dt):
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    layer, wl = _layer(lmoe)
    b = _block(lmoe, layer, wl, 1088, mx, g)
    res = torch.randn(T, 1088, device=DEV, generator=g).to(dt)
    nw = torch.rand(1088, device=DEV, generator=g) + 0.5
    tok = torch.rand(T, 1, device=DEV, generator=g)
    for x_n, gate, next_w in ((None, None, nw), (None, tok, None), (torch.randn(T, 1088, device=DEV, generator=g).bfloat16(), None, nw)):
        r, n = b.forward(res, x_n=x_n, gate=gate, next_w=next_w)
        r2, n2 = _by_hand(lmoe, b, res, x_n, gate, next_w)
        assert b.device_status() == lmoe.OK
        assert torch.equal(r, r2)
        assert (n is None and n2 is None) or torch.equal(n, n2)


def test_two_blocks_in_place_and_captured(cuda_lib):
    """Two blocks after one another on one stream tensor, the first handing its normalised rows to the second; the
    same two captured into a graph and replayed on fresh rows."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    layer, wl = _layer(lmoe)
    a, b = (_block(lmoe, layer, wl, 1024, True, g) for _ in range(2))
    start = torch.randn(16, 1024, device=DEV, generator=g)
    res, x_n = start.clone(), torch.empty(16, 1024, dtype=torch.bfloat16, device=DEV)

    def both():
        a.forward(res, next_w=b.pre_w, res_out=res, next_out=x_n)
        b.forward(res, x_n=x_n, res_out=res)

    both()
    want = _by_hand(lmoe, b, *(lambda rn: (rn[0], rn[1]))(_by_hand(lmoe, a, start, None, None, b.pre_w)), None, None)[0]
    assert torch.equal(res, want)
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        both()
    for s in (2.0, 1.0):
        res.copy_(start * s)
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(res, want)


def test_one_block_in_two_graphs_at_once(cuda_lib):
    """The same block captured into two graphs, replayed on two streams at the same time, and run eagerly beside them
    on a workspace of the caller's."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    layer, wl = _layer(lmoe)
    b = _block(lmoe, layer, wl, 1024, True, g)
    xs = [torch.randn(16, 1024, device=DEV, generator=g) for _ in range(3)]
    want = [b.forward(x)[0] for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(b.forward(x)[0])
        graphs.append(gr)
    streams = [torch.cuda.Stream(DEV) for _ in range(3)]
    ws = torch.empty(b.workspace_size(16), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            eager = b.forward(xs[2], ws=ws)[0]
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(eager, want[2])
    with pytest.raises(lmoe.LmoeError):
        b.forward(xs[0], ws=ws[:256])


def test_block_refusals(cuda_lib):
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    layer, wl = _layer(lmoe)
    b = _block(lmoe, layer, wl, 1024, True, g)
    res = torch.randn(4, 1024, device=DEV, generator=g)
    with pytest.raises(ValueError):
        lmoe.ResidualBlock(layer, b.W_in, b.W_in)
    with pytest.raises(ValueError):
        b.forward(res.half())
    with pytest.raises(ValueError):
        b.forward(res, next_out=torch.empty(4, 1024, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        b.forward(res[:, :512].contiguous())
    with pytest.raises(ValueError):
        b.forward(res, gate=torch.ones(1, 7, device=DEV))
    with pytest.raises(lmoe.LmoeError):
        lmoe.ResidualBlock(layer, b.W_in, b.W_out, pre_w=b.pre_w, eps=-1.0).forward(res)
    with pytest.raises(ValueError):
        lmoe.ResidualBlock(layer, b.W_in, b.W_out).forward(res)  # neither x_n nor pre_w


@pytest.mark.parametrize("T,E,k,d,I", [(1, 40, 4, 256, 72), (64, 48, 6, 384, 136), (700, 12, 3, 256, 128)])
def test_bf16_experts_between_router_and_combine(cuda_lib, T, E, k, d, I):
    """route -> permute -> gated products -> weighted products -> combine, against
    fp64 on the GPU's routing.  Per element, with the errors of the parts as in
    the operator tests: h off by half a bf16 step and its fp32 sums' errors, the
    down sums by (I + 2) u of their magnitudes, the combine's k sums by k u, and
    the output by half a step."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    randn = lambda *s, sc=1.0: (torch.randn(*s, device=DEV, generator=g) * sc).to(torch.bfloat16)
    x = randn(T, d)
    bank = lmoe.ExpertBankBf16(randn(E, I, d, sc=d ** -0.5), randn(E, I, d, sc=d ** -0.5), randn(E, d, I, sc=I ** -0.5))
    _, idx, w = lmoe.route(x, torch.randn(E, d, device=DEV, generator=g) * d ** -0.5, k)
    counts, offsets, perm, inv, _ = lmoe.permute(idx, E)
    ws = torch.zeros(lmoe.grouped_workspace_size(), dtype=torch.uint8, device=DEV)
    y = lmoe.combine(lmoe.expert_ffn_bf16(x, bank, offsets, perm, w, k, ws=ws), inv, T, k)
    assert lmoe.last_device_status(ws) == lmoe.OK
    ref, tol = torch.zeros(T, d, dtype=D, device=DEV), torch.zeros(T, d, dtype=D, device=DEV)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        xe, wg, wu, wd = x[t].to(D), bank.gate[e].to(D), bank.up[e].to(D), bank.down[e].to(D)
        a, b = xe @ wg.t(), xe @ wu.t()
        da, db = (d + 2) * U * (xe.abs() @ wg.abs().t()), (d + 2) * U * (xe.abs() @ wu.abs().t())
        s = a * torch.sigmoid(a)
        h = s * b
        dh = 1.1 * da * (b.abs() + db) + (s.abs() + 1.1 * da) * db + 16 * U * h.abs()
        dh = h.abs() * HALF + dh * (1 + HALF)
        wt = w[t, j].to(D)[:, None]
        mag = (h.abs() + dh) @ wd.abs().t()
        ref.index_add_(0, t, wt * (h @ wd.t()))
        tol.index_add_(0, t, wt * (dh @ wd.abs().t() + (I + 2 + 1 + k) * U * mag))
    out = y.to(D)
    assert bool(((out - ref).abs() <= tol + (ref.abs() + tol) * HALF).all())
    # the bound above takes every error of h to be worst and of one sign; as a whole h's and y's roundings show
    assert float((out - ref).norm()) <= 2 * HALF * float(ref.norm())
