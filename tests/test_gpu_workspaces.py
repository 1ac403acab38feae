"""Memory that layers and blocks hold: the workspaces kept between calls, across
streams and captures, and weights that have to lie on the call's device."""
import pytest
import torch

from test_gpu_residual_block import _block, _layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _made(lmoe, kind):
    """(object with a kept workspace, a call of it on T rows)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    layer, wl = _layer(lmoe)
    if kind == "layer":
        return layer, lambda T, **a: layer.forward(torch.ones(T, wl.d, device=DEV, dtype=torch.bfloat16), **a)
    b = _block(lmoe, layer, wl, 1024, False, g)
    x = lambda T: torch.ones(T, 1024, device=DEV, dtype=torch.bfloat16)
    if kind == "residual_block":
        return b, lambda T, **a: b.forward(x(T), **a)
    c = lmoe.Block(b.W_in, layer, b.W_out)
    return c, lambda T, **a: c.forward(x(T), **a)


@pytest.mark.parametrize("kind", ["layer", "block", "residual_block"])
@pytest.mark.parametrize("how", ["current", "argument"])
def test_a_replaced_workspace_waits_for_its_last_stream(cuda_lib, kind, how):
    """A workspace made on one stream, used on another behind long work and then replaced by a larger one is not given
    to the first stream's next allocations while that work runs."""
    _made(cuda_lib, kind)[1](400)  # (kernels are loaded before the long work)
    obj, call = _made(cuda_lib, kind)
    a, b = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    with torch.cuda.stream(a):
        call(40)
    a.synchronize()
    old, n = obj._ws.data_ptr(), obj._ws.numel()
    run = (lambda T: call(T)) if how == "current" else (lambda T: call(T, stream=b))
    torch.cuda.synchronize()
    b.wait_stream(a)
    with torch.cuda.stream(b):
        torch.cuda._sleep(1_000_000_000)  # about half a second
        if how == "current":
            run(40)
    if how == "argument":
        with torch.cuda.stream(a):
            run(40)
            run(400)
    else:
        with torch.cuda.stream(b):
            run(400)
    assert obj._ws.numel() > n
    with torch.cuda.stream(a):
        got = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(20)]
    assert not b.query()  # still in the long work
    assert all(t.data_ptr() + n <= old or old + n <= t.data_ptr() for t in got)
    torch.cuda.synchronize()


def test_a_forward_captured_through_its_stream_argument_has_its_own_workspace(cuda_lib):
    """Whether a forward is captured is a question about the call's stream, not the current one: captured on `stream`
    with another stream current, the graph does not use the workspace that the block keeps for eager calls."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    layer, wl = _layer(lmoe)
    b = _block(lmoe, layer, wl, 1024, True, g)
    x = torch.randn(16, 1024, device=DEV, generator=g)
    want = b.forward(x)[0].clone()
    s, gr = torch.cuda.Stream(DEV), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        gr.capture_begin()
    out = b.forward(x, stream=s)[0]
    with torch.cuda.stream(s):
        gr.capture_end()
    b._ws.fill_(255)
    torch.cuda.synchronize()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert bool((b._ws == 255).all())
    # the other way round: an eager call beside a capture on the current stream keeps the block's workspace
    y = torch.zeros(64, device=DEV)
    gr, s2 = torch.cuda.CUDAGraph(), torch.cuda.Stream(DEV)
    with torch.cuda.graph(gr, stream=s, capture_error_mode="relaxed"):
        y.add_(1)
        out = b.forward(x, stream=s2)[0]
    s2.synchronize()
    assert torch.equal(out, want)
    assert not bool((b._ws == 255).all())
    assert b.device_status() == lmoe.OK


WEIGHTS = ["layer.Wr3", "layer.bias", "W_in.q", "W_in.s", "W_out.q", "W_out.s"] + \
    [f"layer.bank.{w}_{p}" for w in ("gate", "up", "down") for p in "qs"]


def _swap(b, path, change):
    obj = b
    *way, last = path.split(".")
    for p in way:
        obj = getattr(obj, p)
    old = getattr(obj, last)
    setattr(obj, last, change(old))
    return lambda: setattr(obj, last, old)


@pytest.mark.parametrize("mx", [True, False])
def test_weights_off_the_calls_device_are_refused(cuda_lib, mx):
    """Host addresses among the weights (a module moved by hand) are refused before anything is launched."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    layer, wl = _layer(lmoe)
    layer.bias = torch.zeros(wl.E, device=DEV)
    b = _block(lmoe, layer, wl, 1024, mx, g)
    x = torch.randn(4, 1024, device=DEV, generator=g)
    want = b.forward(x)[0]
    for path in WEIGHTS if mx else ["W_in", "W_out"]:
        back = _swap(b, path, lambda t: t.cpu())
        with pytest.raises(ValueError, match=path.split(".")[-1]):
            b.forward(x)
        back()
    for path, change in (("layer.bias", lambda t: t.double()), ("layer.bias", lambda t: t[:-1])):
        back = _swap(b, path, change)
        with pytest.raises(ValueError, match="bias"):
            b.forward(x)
        back()
    assert torch.equal(b.forward(x)[0], want)


def test_errors_of_calls_without_a_workspace_can_be_asked_for(cuda_lib):
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    randn = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()
    x, W, D = randn(40, 64), randn(3, 64, 64), randn(3, 64, 64)
    off = torch.tensor([0, 8, 24, 40], dtype=torch.int32, device=DEV)
    perm = torch.arange(40, dtype=torch.int32, device=DEV)
    bad = torch.tensor([0, 8, 24, 4000], dtype=torch.int32, device=DEV)
    w = torch.ones(40, device=DEV)
    lin = lmoe.LinearMxfp4(torch.randn(96, 64, device=DEV, generator=g))
    bank = lmoe.ExpertBankBf16(W, W, D)
    calls = [(lambda o: lmoe.grouped_linear_bf16(x, W, o), lmoe.ERR_DEVICE_CHECK),
             (lambda o: lmoe.grouped_swiglu_bf16(x, W, W, o), lmoe.ERR_DEVICE_CHECK),
             (lambda o: lmoe.expert_ffn_bf16(x, bank, o, perm, w, 1), lmoe.ERR_DEVICE_CHECK)]
    for call, code in calls:
        call(off)
        assert lmoe.last_call_status() == lmoe.OK
        call(bad)
        assert lmoe.last_call_status() == code
    # only the first of the two products reads x's rows
    lmoe.expert_ffn_bf16(x[:39], bank, off, perm, w, 1)
    assert lmoe.last_call_status() == lmoe.ERR_DEVICE_CHECK
    # a workspace of the caller's is asked by itself
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lmoe.grouped_linear_bf16(x, W, bad, ws=ws)
    lmoe.grouped_linear_bf16(x, W, off)
    assert lmoe.last_call_status() == lmoe.OK and lmoe.last_device_status(ws) == lmoe.ERR_DEVICE_CHECK
    for rows in (4, 40):
        lmoe.set_wait_test(True, 20_000_000)  # about 10 ms of SM clocks
        try:
            lin.forward(randn(rows, 64))
            torch.cuda.synchronize()
        finally:
            lmoe.set_wait_test(False, 0)
        assert lmoe.last_call_status() == lmoe.ERR_TIMEOUT
        lin.forward(randn(rows, 64))
        assert lmoe.last_call_status() == lmoe.OK
    # captured: of the latest replay
    gr, o = torch.cuda.CUDAGraph(), off.clone()
    lmoe.grouped_linear_bf16(x, W, o)
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        lmoe.grouped_linear_bf16(x, W, o)
    for now, code in ((bad, lmoe.ERR_DEVICE_CHECK), (off, lmoe.OK)):
        o.copy_(now)
        gr.replay()
        assert lmoe.last_call_status() == code


def test_what_a_call_on_another_stream_allocates_stays_its_own(cuda_lib, monkeypatch):
    """Outputs and workspaces that a call with a stream argument allocates, let go while the call is still to run: their
    memory goes to no allocation of the current stream before it has."""
    lmoe = cuda_lib
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    layer, wl = _layer(lmoe)
    T, d, E, k = 40, wl.d, wl.E, wl.k
    x = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    Wr = torch.randn(E, d, device=DEV, generator=g)
    w32 = torch.randn(1, 256, d, device=DEV, generator=g)
    Wl = torch.randn(256, d, device=DEV, generator=g).bfloat16()
    logits, idx, w = lmoe.route(x, Wr, k)
    _, off, perm, inv, _ = lmoe.permute(idx, E)
    xq, xs = lmoe.quant_mxfp8(x)
    qc, sc = lmoe.quant_mxfp4(w32, layout=lmoe.LAYOUT_CANONICAL)
    yp = lmoe.expert_ffn(xq, xs, layer.bank, off, perm, w, k)[0]
    block = lmoe.Block(torch.randn(d, 1024, device=DEV, generator=g).bfloat16(), layer,
                       torch.randn(1024, d, device=DEV, generator=g).bfloat16())
    xh = torch.randn(T, 1024, device=DEV, generator=g).bfloat16()
    calls = {
        "prepare_router": lambda **a: lmoe.prepare_router(Wr, **a), "route": lambda **a: lmoe.route(x, Wr, k, **a),
        "topk_from_logits": lambda **a: lmoe.topk_from_logits(logits, k, **a),
        "permute": lambda **a: lmoe.permute(idx, E, **a), "permute_noalloc": lambda **a: lmoe.permute_noalloc(idx, E, **a),
        "quant_mxfp4": lambda **a: lmoe.quant_mxfp4(w32, **a), "quant_mxfp8": lambda **a: lmoe.quant_mxfp8(x, **a),
        "repack_mxfp4": lambda **a: lmoe.repack_mxfp4(qc, sc, 1, 256, d, **a),
        "scale_histogram": lambda **a: lmoe.scale_histogram(sc, 1, 256, d, lmoe.LAYOUT_CANONICAL, **a),
        "expert_ffn": lambda **a: lmoe.expert_ffn(xq, xs, layer.bank, off, perm, w, k, **a),
        "combine": lambda **a: lmoe.combine(yp, inv, T, k, **a), "linear_bf16": lambda **a: lmoe.linear_bf16(x, Wl, **a),
        "layer": lambda **a: layer.forward(x, **a), "block": lambda **a: block.forward(xh, **a),
    }
    for f in calls.values():
        f()  # (kernels are loaded, kept workspaces made)
    side, empty = torch.cuda.Stream(DEV), torch.empty
    torch.cuda.synchronize()
    wrong = []
    for name, f in calls.items():
        made = []

        def watched(*a, **kw):
            t = empty(*a, **kw)
            made.append((t.data_ptr(), t.numel() * t.element_size()))
            return t

        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # about 0.1 s
        with monkeypatch.context() as m:
            m.setattr(torch, "empty", watched)
            f(stream=side)
        got = [empty(n, dtype=torch.uint8, device=DEV) for _, n in made for _ in range(4)]
        assert not side.query() and made, name
        if any(p < t.data_ptr() + t.numel() and t.data_ptr() < p + n for p, n in made for t in got):
            wrong.append(name)
        side.synchronize()
        del got
    assert not wrong, wrong
