"""The linear layer with bias, function and residual, layer norm, the balance loss and
their gradients, against plain torch in 64 bits.

Tolerances (u = 2^-24, half a step of fp32; a bf16 result is off by at most half a
step, 2^-8 of its value):
  products    each term passes at most K additions and one rounding of its product, in
              any order: |error| <= (K + 2) u sum |a b|.
  functions   slopes stay below 1.2, so an error of z enters the value with at most that
              factor; their own evaluation: the exponential's or erfc's argument is off
              by a few u of itself, which they turn into (8 |argument|) u of the value,
              the rest (exponential, division, products) below 16 u.  A slope's terms
              stay below 2 and their arguments' errors times the terms below 8 u, so it
              is off by less than 64 u.
  dz          is rounded to bf16 for the two products: half a bf16 step of every term.
  layer norm  a row's sums have at most 64 + 11 additions on any element's way, with
              the roundings of the terms below 84 u of the sum of magnitudes.
  balance     exponentials are off by 2 u |l - max| + 4 u of themselves, a row's sum by
              as much and 72 additions: with |l - max| <= 60, p by less than 400 u of itself.
Sums over rows: at most one addition a row on a term's way, and 300 where blocks and
warps are added up.
"""
import math

import pytest
import torch

from test_gpu_operators import D, DEV, HALF, U, gen, guarded, randn, within

pytestmark = pytest.mark.gpu
TINY = 1e-36
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
C = math.sqrt(8 / math.pi)


def phi(z):
    return torch.special.erfc(-z / 2 ** 0.5) / 2


def act_ref(z, act):
    """(value, argument of the exponential or of erfc) in 64 bits."""
    if act == "relu":
        return z.clamp_min(0), 0 * z
    if act == "silu":
        return z * torch.sigmoid(z), z.abs()
    if act == "gelu":
        return z * phi(z), z * z
    if act == "gelu_tanh":
        u = C * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(u), u.abs()
    return z, 0 * z


def slope_ref(z, act):
    if act == "relu":
        return (z > 0).to(D)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        u = C * (z + 0.044715 * z ** 3)
        return torch.sigmoid(u) + z * torch.sigmoid(u) * torch.sigmoid(-u) * C * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def half_of(dt):
    return HALF if dt == torch.bfloat16 else U


# ---- linear ---------------------------------------------------------------------------

def check_linear(lmoe, x, W, bias, act, res, pre, out_dt=None, ws=None):
    rows, K = x.shape
    N = W.shape[0]
    out_dt = out_dt or (torch.bfloat16 if res is None else res.dtype)
    out, intact = guarded((rows, N), out_dt)
    po, intact_p = guarded((rows, N), torch.bfloat16)
    if ws is None:
        ws = torch.zeros(lmoe.linear_act_workspace_size(rows, K, N), dtype=torch.uint8, device=DEV)
    r = lmoe.linear_act_bf16(x, W, bias=bias, act=act, res=res, out=out, pre=po if pre else None, ws=ws)
    z = x.to(D) @ W.to(D).t()
    tz = (K + 2) * U * (x.to(D).abs() @ W.to(D).abs().t())
    if bias is not None:
        z = z + bias.to(D)
        tz = tz + z.abs() * U
    a, arg = act_ref(z, act)
    ta = 1.2 * tz + (16 + 8 * arg) * U * a.abs() + TINY
    ref = a if res is None else a + res.to(D)
    if res is not None:
        ta = ta + ref.abs() * U
    within(r[0] if pre else r, ref, ta + (ref.abs() + ta) * half_of(out_dt))
    if pre:
        assert r[1] is po
        within(po, z, tz + (z.abs() + tz) * HALF)
    assert lmoe.last_device_status(ws) == lmoe.OK
    assert intact() and intact_p()
    return out, ref


SIZES = [(1, 8, 1), (1, 64, 7), (3, 72, 130), (17, 264, 64), (64, 512, 250), (65, 136, 129), (128, 1024, 256),
         (130, 96, 1000), (200, 1056, 33), (333, 520, 300), (513, 256, 520)]


@pytest.mark.parametrize("rows,K,N", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_act(cuda_lib, rows, K, N, act):
    g = gen(rows + 3 * K + 7 * N)
    x, W = randn(g, rows, K), randn(g, N, K, scale=2 * K ** -0.5)
    b = {0: None, 1: randn(g, N, dtype=torch.float32), 2: randn(g, N)}[(rows + N) % 3]
    res = {0: None, 1: randn(g, rows, N, dtype=torch.float32), 2: randn(g, rows, N)}[(rows + K // 8) % 3]
    check_linear(cuda_lib, x, W, b, act, res, pre=N % 2 == 0)


@pytest.mark.parametrize("bias", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("res", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,N", [(5, 72), (150, 40), (150, 45)])
def test_linear_act_types(cuda_lib, bias, res, out_dt, rows, N):
    g = gen(rows + N)
    K = 136
    x, W = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5)
    b = None if bias is None else randn(g, N, dtype=bias)
    r = None if res is None else randn(g, rows, N, dtype=res, scale=3.0)
    check_linear(cuda_lib, x, W, b, "gelu", r, True, out_dt)
    check_linear(cuda_lib, x, W, b, "silu", r, False, out_dt)


@pytest.mark.parametrize("rows,K,N", [(1, 3584, 7168), (1, 7168, 3584), (7, 7168, 3584), (64, 7168, 3584), (100, 7168, 520),
                                      (331, 1056, 1000), (512, 7168, 3584), (700, 2048, 4104), (2048, 3584, 7168),
                                      (2, 16, 40000), (9000, 72, 136), (40, 16384, 72)])
def test_linear_act_wide(cuda_lib, rows, K, N):
    g = gen(rows + K)
    x, W = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5)
    check_linear(cuda_lib, x, W, randn(g, N, dtype=torch.float32), "gelu_tanh", randn(g, rows, N), True)


@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_linear_act_in_place_on_the_residual_and_repeats(cuda_lib, rows, dt):
    g = gen(rows)
    x, W, b = randn(g, rows, 520), randn(g, 264, 520, scale=0.05), randn(g, 264)
    res = randn(g, rows, 264, dtype=dt)
    want = cuda_lib.linear_act_bf16(x, W, b, "silu", res)
    r2 = res.clone()
    got = cuda_lib.linear_act_bf16(x, W, b, "silu", r2, out=r2)
    assert got is r2 and torch.equal(want, r2)
    for _ in range(5):
        assert torch.equal(cuda_lib.linear_act_bf16(x, W, b, "silu", res), want)
    assert cuda_lib.last_call_status() == cuda_lib.OK


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [4, 200])
def test_linear_act_far_values_and_nan_rows(cuda_lib, act, rows):
    """Pre-activations far out on both sides: values and tails as the function has them; a NaN stays in its row."""
    K = N = 64
    x = torch.zeros(rows, K, device=DEV, dtype=torch.bfloat16)
    x[:, 0] = 1
    W = torch.zeros(N, K, device=DEV, dtype=torch.bfloat16)
    W[:, 0] = torch.cat([torch.linspace(-14, 14, 52), torch.tensor([-3e4, 3e4, -120., 120., -88., 88., -1e18, 1e18, 0., -0.,
                                                                   1e-30, -1e-30])]).to(DEV).bfloat16()
    check_linear(cuda_lib, x, W, None, act, None, True, torch.float32)
    x[2, 5] = float("nan")
    out = cuda_lib.linear_act_bf16(x, W, act=act)
    keep = [i for i in range(rows) if i != 2]
    assert bool(out[2].isnan().all()) and not bool(out[keep].isnan().any())


def test_linear_act_without_rows(cuda_lib):
    W = torch.zeros(40, 64, device=DEV, dtype=torch.bfloat16)
    x = torch.zeros(0, 64, device=DEV, dtype=torch.bfloat16)
    assert cuda_lib.linear_act_bf16(x, W).shape == (0, 40)
    dout = torch.zeros(0, 40, device=DEV, dtype=torch.bfloat16)
    dW, db = torch.ones(40, 64, device=DEV), torch.ones(40, device=DEV)
    dx, dW, db = cuda_lib.linear_act_bf16_backward(dout, x, W, "gelu", None, dW=dW, dbias=db)
    assert dx.shape == (0, 64) and not bool(dW.any()) and not bool(db.any())


def test_linear_act_beyond_2_31_outputs(cuda_lib):
    rows, K, N = 66000, 8, 33000
    g = gen(3)
    x, W, b = randn(g, rows, K), randn(g, N, K), randn(g, N)
    out, pre = cuda_lib.linear_act_bf16(x, W, b, "relu", pre=True)
    for r0 in (0, 40000, rows - 65):
        z = x[r0:r0 + 65].to(D) @ W.to(D).t() + b.to(D)
        tol = 12 * U * (x[r0:r0 + 65].to(D).abs() @ W.to(D).abs().t() + b.to(D).abs())
        within(out[r0:r0 + 65], z.clamp_min(0), tol + (z.abs() + tol) * HALF)
        within(pre[r0:r0 + 65], z, tol + (z.abs() + tol) * HALF)


def check_back(lmoe, dout, x, W, act, pre, dW_dt):
    rows, K = x.shape
    N = W.shape[0]
    dx, i0 = guarded((rows, K), torch.bfloat16)
    dW, i1 = guarded((N, K), dW_dt)
    db, i2 = guarded((N,), torch.float32)
    ws = torch.zeros(lmoe.linear_act_backward_workspace_size(rows, K, N), dtype=torch.uint8, device=DEV)
    lmoe.linear_act_bf16_backward(dout, x, W, act, pre, dx=dx, dW=dW, dbias=db, ws=ws)
    assert lmoe.last_device_status(ws) == lmoe.OK
    d = dout.to(D)
    dz = d if pre is None else d * slope_ref(pre.to(D), act)
    exact = act == "none" and dout.dtype == torch.bfloat16
    te = d.abs() * (0 if act == "none" else 65 * U)       # dz in fp32
    tz = te if exact else te + (dz.abs() + te) * HALF  # as rounded for the products
    for got, a, b, ta, n, half in ((dx, dz, W.to(D), tz, N, HALF), (dW, dz.t(), x.to(D), tz.t(), rows, half_of(dW_dt))):
        ref = a @ b
        tol = ta @ b.abs() + (n + 2) * U * ((a.abs() + ta) @ b.abs())
        within(got, ref, tol + (ref.abs() + tol) * half + TINY)
        if ref.numel() > 1000:  # roundings of the terms and of the result, each half a step at most, fall either way
            assert float((got.to(D) - ref).norm()) <= 2 * HALF * float(ref.norm())
    ref = dz.sum(0)
    within(db, ref, te.sum(0) + (rows + 2) * U * dz.abs().sum(0) + TINY)
    assert i0() and i1() and i2()
    return dx, dW, db


@pytest.mark.parametrize("rows,K,N", SIZES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_act_backward(cuda_lib, rows, K, N, act):
    g = gen(rows + 5 * K + N)
    x, W = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5)
    dout = randn(g, rows, N, dtype=torch.float32 if (rows + N) % 2 else torch.bfloat16, scale=0.1)
    pre = None if act == "none" else randn(g, rows, N, scale=2.0)
    check_back(cuda_lib, dout, x, W, act, pre, torch.float32 if N % 2 else torch.bfloat16)


@pytest.mark.parametrize("rows,K,N", [(1, 7168, 3584), (64, 3584, 7168), (333, 1056, 1000), (1500, 2048, 4104),
                                      (20000, 64, 72), (3000, 512, 512), (4096, 3584, 512), (600, 7168, 256)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_linear_act_backward_wide(cuda_lib, rows, K, N, dt):
    g = gen(rows + K)
    x, W = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5)
    act = "silu" if dt == torch.bfloat16 else "none"
    check_back(cuda_lib, randn(g, rows, N, dtype=dt, scale=0.1), x, W, act, None if act == "none" else randn(g, rows, N), dt)


def test_linear_act_backward_parts(cuda_lib):
    """Each gradient by itself is the one of the whole call."""
    g = gen(9)
    x, W, dout, pre = randn(g, 140, 264), randn(g, 200, 264), randn(g, 140, 200), randn(g, 140, 200)
    whole = cuda_lib.linear_act_bf16_backward(dout, x, W, "gelu", pre)
    for i in range(3):
        want = [j == i for j in range(3)]
        part = cuda_lib.linear_act_bf16_backward(dout, x, W, "gelu", pre, *want)
        assert [p is not None for p in part] == want and torch.equal(part[i], whole[i])
    assert cuda_lib.linear_act_bf16_backward(dout, x, W, "gelu", pre, False, False, False) == (None, None, None)


@pytest.mark.parametrize("rows,K,N", [(1, 8, 33), (65, 16, 20011), (300, 8, 9000), (6000, 72, 40), (8192, 64, 257),
                                      (2048, 512, 1024)])
def test_dbias_of_many_groups(cuda_lib, rows, K, N):
    """dbias has the same bits whether it comes by itself or on the way of one product or both."""
    g = gen(rows + N)
    x, W = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5)
    dout, pre = randn(g, rows, N, scale=0.1), randn(g, rows, N)
    dx, dW, db = check_back(cuda_lib, dout, x, W, "silu", pre, torch.float32)
    for want in ((False, False), (True, False), (False, True)):
        part = cuda_lib.linear_act_bf16_backward(dout, x, W, "silu", pre, *want)
        assert torch.equal(part[2], db)
        assert not want[0] or torch.equal(part[0], dx)
        assert cuda_lib.last_call_status() == cuda_lib.OK


@pytest.mark.parametrize("act", ACTS)
def test_slopes_far_out(cuda_lib, act):
    """dbias of one row is dout times the slope: finite and right for every pre-activation."""
    z = torch.cat([torch.linspace(-12, 12, 200), torch.tensor([-1e38, 1e38, -3e4, 3e4, -90., 90., 0., -0., 1e-38])])
    pre = z.to(DEV).bfloat16()[None]
    n = pre.shape[1]
    dout = torch.ones(1, n, device=DEV)
    x, W = torch.zeros(1, 8, device=DEV, dtype=torch.bfloat16), torch.zeros(n, 8, device=DEV, dtype=torch.bfloat16)
    _, _, db = cuda_lib.linear_act_bf16_backward(dout, x, W, act, None if act == "none" else pre)
    within(db[None], torch.nan_to_num(slope_ref(pre.to(D), act)), torch.full_like(pre, 64 * U, dtype=D))


# ---- layer norm -----------------------------------------------------------------------

NORM_SIZES = [(1, 8), (1, 7168), (3, 40), (5, 256), (4, 264), (2500, 520), (2, 1024), (3, 1032), (7, 4104), (400, 7168),
              (305, 3584), (700, 2048), (2, 8192), (3, 8200), (310, 8200), (2, 16384), (2, 16392), (5, 32768)]


def stream_rows(g, T, H, dt):
    amp = torch.exp(torch.randn(T, 1, device=DEV, generator=g))
    return (torch.randn(T, H, device=DEV, generator=g) * amp + 0.5 * amp).to(dt)


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("params", ["wb", "w", "b", ""])
def test_layer_norm(cuda_lib, T, H, dt, params):
    g = gen(T * 3 + H)
    x = stream_rows(g, T, H, dt)
    w = randn(g, H, dtype=torch.float32) if "w" in params else None
    b = randn(g, H, dtype=torch.float32) if "b" in params else None
    out, i0 = guarded((T, H), torch.bfloat16)
    mean, i1 = guarded((T,), torch.float32)
    rstd, i2 = guarded((T,), torch.float32)
    cuda_lib.layer_norm(x, w, b, 1e-5, out=out, mean=mean, rstd=rstd)
    v = x.to(D)
    m = v.mean(1, keepdim=True)
    c = v - m
    var = c.square().mean(1, keepdim=True)
    rs = 1 / (var + 1e-5).sqrt()
    dm = 84 * U * v.abs().mean(1, keepdim=True)  # error of the mean
    dr = 60 * U + 0.5 * dm.square() / (var + 1e-5)  # of rstd, relative
    within(mean[:, None], m, dm)
    within(rstd[:, None], rs, rs * dr)
    y = c * rs * (1 if w is None else w.to(D))
    ref = y if b is None else y + b.to(D)
    tol = y.abs() * (dr + 4 * U) + dm * rs * (1 if w is None else w.to(D).abs()) + ref.abs() * U
    within(out, ref, tol + (ref.abs() + tol) * HALF)
    assert torch.equal(cuda_lib.layer_norm(x, w, b, 1e-5), out)
    assert i0() and i1() and i2()


def test_layer_norm_of_rows_without_spread(cuda_lib):
    """Constant rows give b; a NaN or an infinity stays in its row."""
    x = torch.full((6, 512), 3.0, device=DEV)
    x[1] = 0
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    b = torch.arange(512, device=DEV, dtype=torch.float32)
    out = cuda_lib.layer_norm(x, None, b)
    assert torch.equal(out[[0, 1, 2, 5]], b.bfloat16()[None].expand(4, 512))
    assert bool(out[[3, 4]].isnan().all())


def check_norm_back(lmoe, T, H, dt, w, add, dy, x, mean, rstd, params=True):
    dx, i0 = guarded((T, H), dt)
    dw, i1 = guarded((H,), torch.float32)
    db, i2 = guarded((H,), torch.float32)
    r = lmoe.layer_norm_backward(dy, x, mean, rstd, w, add, params, dx=dx, dw=dw if params else None,
                                 db=db if params else None)
    h = (x.to(D) - mean.to(D)[:, None]) * rstd.to(D)[:, None]
    g = dy.to(D) * (1 if w is None else w.to(D))
    mg, mgh = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    rs = rstd.to(D)[:, None]
    ref = rs * (g - mg - h * mgh)
    tol = rs * 100 * U * (g.abs() + g.abs().mean(1, keepdim=True) + h.abs() * (g * h).abs().mean(1, keepdim=True))
    if add is not None:
        ref = ref + add.to(D)
    tol = tol + ref.abs() * U
    within(r[0], ref, tol + (ref.abs() + tol) * half_of(dt) + TINY)
    if params:
        within(r[1], (dy.to(D) * h).sum(0), (T + 8) * U * (dy.to(D) * h).abs().sum(0) + TINY)
        within(r[2], dy.to(D).sum(0), (T + 8) * U * dy.to(D).abs().sum(0) + TINY)
    else:
        assert r[1] is None and r[2] is None
    assert i0() and i1() and i2()
    return r


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weighted,added,params", [(True, True, True), (True, False, True), (False, True, True),
                                                   (True, True, False), (False, False, False)])
def test_layer_norm_backward(cuda_lib, T, H, dt, weighted, added, params):
    g = gen(T * 5 + H)
    x = stream_rows(g, T, H, dt)
    dy, w = randn(g, T, H, scale=0.1), randn(g, H, dtype=torch.float32) if weighted else None
    add = randn(g, T, H, dtype=dt, scale=0.1) if added else None
    _, mean, rstd = cuda_lib.layer_norm(x, w, stats=True)
    r = check_norm_back(cuda_lib, T, H, dt, w, add, dy, x, mean, rstd, params)
    again = cuda_lib.layer_norm_backward(dy, x, mean, rstd, w, add, params)
    assert torch.equal(again[0], r[0]) and (not params or (torch.equal(again[1], r[1]) and torch.equal(again[2], r[2])))
    if added:
        a = add.clone()
        inplace = cuda_lib.layer_norm_backward(dy, x, mean, rstd, w, a, params, dx=a)
        assert inplace[0] is a and torch.equal(a, r[0])
        assert not params or (torch.equal(inplace[1], r[1]) and torch.equal(inplace[2], r[2]))


@pytest.mark.parametrize("T,H", [(303, 1024), (305, 1024), (609, 640), (1216, 520), (1217, 2048), (2431, 640), (2433, 1024),
                                 (3649, 1000)])
def test_layer_norm_backward_by_blocks(cuda_lib, T, H):
    """Row counts about those where a block takes one row, two or four."""
    g = gen(T + H)
    x, dy, w = stream_rows(g, T, H, torch.float32), randn(g, T, H, scale=0.1), randn(g, H, dtype=torch.float32)
    _, mean, rstd = cuda_lib.layer_norm(x, w, stats=True)
    check_norm_back(cuda_lib, T, H, torch.float32, w, randn(g, T, H, dtype=torch.float32), dy, x, mean, rstd)


def test_layer_norm_backward_without_rows(cuda_lib):
    z = torch.zeros(0, 256, device=DEV, dtype=torch.bfloat16)
    s = torch.zeros(0, device=DEV)
    dw, db = torch.ones(256, device=DEV), torch.ones(256, device=DEV)
    dx, dw, db = cuda_lib.layer_norm_backward(z, z, s, s, dw=dw, db=db)
    assert dx.shape == (0, 256) and not bool(dw.any()) and not bool(db.any())


# ---- balance loss -----------------------------------------------------------------------

def balance_ref(l, idx, keep, coef, w=None, dw=None, scale=1.0):
    """(loss, counts, probs, dlogits, tolerance of dlogits) in 64 bits, on rows that count."""
    T, E = l.shape
    k = idx.shape[1]
    n = int(keep.sum())
    counts = torch.bincount(idx[keep].reshape(-1).long(), minlength=E)
    d, tol = torch.zeros(T, E, dtype=D, device=l.device), torch.zeros(T, E, dtype=D, device=l.device)
    if n == 0:
        return torch.zeros(2, dtype=D, device=l.device), counts, torch.zeros(E, dtype=D, device=l.device), d, tol
    v = l[keep].to(D)
    lse = torch.logsumexp(v, 1)
    p = torch.exp(v - lse[:, None])
    f = counts.to(D) * E / (k * n)
    probs = p.sum(0) / n
    loss = torch.stack([(f * probs).sum(), lse.square().sum() / n])
    sf = (p * f).sum(1, keepdim=True)
    cb, cz = scale * coef[0] / n, scale * coef[1] * 2 / n
    dd = cb * p * (f - sf) + cz * lse[:, None] * p
    tt = 400 * U * p * (abs(cb) * (f + sf) + abs(cz) * (lse.abs()[:, None] + 1))
    if w is not None:
        ww, gg = w[keep].to(D), dw[keep].to(D)
        ii = idx[keep].long()
        dd.scatter_add_(1, ii, ww * (gg - (ww * gg).sum(1, keepdim=True)))
        tt.scatter_add_(1, ii, 48 * U * ww.abs() * (gg.abs() + (ww * gg).abs().sum(1, keepdim=True)))
    d[keep], tol[keep] = dd, tt + dd.abs() * U + TINY
    return loss, counts, probs, d, tol


def check_balance(lmoe, l, idx, mask=None, coef=(0.01, 0.002), w=None, dw=None, scale=None, grad=True):
    T, E = l.shape
    k = idx.shape[1]
    ws = torch.zeros(lmoe.balance_loss_workspace_size(T, E, k), dtype=torch.uint8, device=DEV)
    ws[256:] = 0xA5  # nothing but the status word has to be cleared
    d, intact = guarded((T, E), torch.float32)
    r = lmoe.balance_loss(l, idx, mask=mask, coef=coef, grad=grad, topk_w=w, dtopk_w=dw, scale=scale,
                          dlogits=d if grad else None, ws=ws)
    assert lmoe.last_device_status(ws) == lmoe.OK
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if mask is None else mask
    loss, counts, probs, dref, dtol = balance_ref(l, idx, keep, coef, w, dw, 1.0 if scale is None else float(scale))
    n = max(int(keep.sum()), 1)
    lse = torch.logsumexp(l[keep].to(D), 1)
    assert r[1].dtype == torch.int32 and torch.equal(r[1].long(), counts)
    within(r[2], probs, (T + 700) * U * probs + TINY)
    tol = torch.stack([(T + E + 800) * U * loss[0], (T + 900) * U * loss[1] + 900 * U * lse.abs().sum() / n]) + TINY
    within(r[0], loss, tol)
    if grad:
        assert r[3] is d
        within(d, dref, dtol)
        assert not bool(d[~keep].any())
    assert intact()
    return r


def picks(g, T, E, k):
    return torch.rand(T, E, device=DEV, generator=g).topk(k, 1).indices.to(torch.int32).contiguous()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 896, 16), (2, 7, 7), (5, 32, 32), (64, 896, 16), (333, 130, 3),
                                   (151, 384, 8), (1000, 257, 4), (1100, 896, 16), (2100, 60, 8), (700, 2048, 32),
                                   (513, 1023, 5), (3000, 4, 2),
                                   (73, 1149, 20), (125, 1032, 25), (2000, 128, 8), (2000, 129, 8), (1500, 256, 4),
                                   (1500, 255, 4), (128, 128, 32), (129, 16, 4), (20000, 8, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss(cuda_lib, T, E, k, masked):
    g = gen(T + E + k)
    l = 2 * torch.randn(T, E, device=DEV, generator=g)
    idx = picks(g, T, E, k)
    mask = torch.rand(T, device=DEV, generator=g) < 0.7 if masked else None
    w = torch.softmax(torch.randn(T, k, device=DEV, generator=g), 1).contiguous()
    dw = torch.randn(T, k, device=DEV, generator=g)
    a = check_balance(cuda_lib, l, idx, mask, w=w, dw=dw)
    b = check_balance(cuda_lib, l, idx, mask, grad=False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))  # the gradient changes none of the rest
    check_balance(cuda_lib, l, idx, mask, scale=torch.full((1,), 0.25, device=DEV))
    check_balance(cuda_lib, l, idx, mask, coef=(0.0, 1.0))
    again = cuda_lib.balance_loss(l, idx, mask=mask, coef=(0.01, 0.002), grad=True, topk_w=w, dtopk_w=dw)
    assert all(torch.equal(x, y) for x, y in zip(a, again))
    assert cuda_lib.last_call_status() == cuda_lib.OK


@pytest.mark.parametrize("E", [896, 130, 61])
def test_balance_loss_padding_holds_anything(cuda_lib, E):
    """Rows that do not count are not looked at: NaN, infinities and ids out of range in them change nothing."""
    g = gen(E)
    T, k = 400, 4
    l, idx = torch.randn(T, E, device=DEV, generator=g), picks(g, T, E, k)
    w, dw = torch.rand(T, k, device=DEV, generator=g), torch.randn(T, k, device=DEV, generator=g)
    mask = torch.rand(T, device=DEV, generator=g) < 0.5
    want = check_balance(cuda_lib, l, idx, mask, w=w, dw=dw)
    l[~mask] = torch.tensor([float("nan"), float("inf"), -float("inf")], device=DEV)[torch.arange(int((~mask).sum()), device=DEV) % 3][:, None]
    idx[~mask] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31], device=DEV, dtype=torch.int32)
    w[~mask] = float("nan")
    dw[~mask] = float("inf")
    got = check_balance(cuda_lib, l, idx, mask, w=w, dw=dw)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T,k", [(50, 2), (9000, 2)])
def test_balance_loss_special_rows(cuda_lib, T, k):
    """Experts masked by -infinity or the type's lowest value have no probability; a row of nothing else adds nothing
    and has no gradient; all rows masked gives zeros."""
    g = gen(T)
    E = 96
    l, idx = torch.randn(T, E, device=DEV, generator=g), picks(g, T, E, k)
    l[:, 7] = -float("inf")
    l[3, 9] = torch.finfo(torch.float32).min
    r = check_balance(cuda_lib, l, idx)
    assert float(r[2][7]) == 0 and not bool(r[3][:, 7].any()) and float(r[3][3, 9]) == 0
    l2 = l.clone()
    l2[11] = -float("inf")
    loss, counts, probs, d = cuda_lib.balance_loss(l2, idx, coef=(0.01, 0.002), grad=True)
    assert torch.equal(counts, r[1]) and not bool(d[11].any())
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(d).all())
    rest = [t for t in range(T) if t != 11]
    within(probs, torch.softmax(l[rest].to(D), 1).sum(0) / T, (T + 700) * U * probs.to(D) + TINY)
    l2[12, 5] = float("nan")
    d = cuda_lib.balance_loss(l2, idx, coef=(0.01, 0.002), grad=True)[3]
    rest.remove(12)
    assert bool(d[12].isnan().all()) and not bool(d[rest].isnan().any())
    l2[13, :] = float("nan")
    l2[14, 3] = float("inf")
    d = cuda_lib.balance_loss(l2, idx, coef=(0.01, 0.002), grad=True)[3]
    assert bool(d[13:15].isnan().all())
    none = torch.zeros(T, dtype=torch.bool, device=DEV)
    for t in cuda_lib.balance_loss(l2, idx, mask=none, grad=True):
        assert not bool(t.any())


def test_balance_loss_without_tokens(cuda_lib):
    r = cuda_lib.balance_loss(torch.zeros(0, 64, device=DEV), torch.zeros(0, 2, device=DEV, dtype=torch.int32), grad=True)
    assert [tuple(t.shape) for t in r] == [(2,), (64,), (64,), (0, 64)] and not any(bool(t.any()) for t in r)


def test_balance_loss_same_expert_twice_and_in_place(cuda_lib):
    g = gen(4)
    T, E, k = 77, 40, 8
    l = torch.randn(T, E, device=DEV, generator=g)
    idx = torch.randint(0, E // 4, (T, k), device=DEV, generator=g).to(torch.int32)  # most rows have an expert twice
    w, dw = torch.rand(T, k, device=DEV, generator=g), torch.randn(T, k, device=DEV, generator=g)
    r = check_balance(cuda_lib, l, idx, w=w, dw=dw)
    l2 = l.clone()
    out = cuda_lib.balance_loss(l2, idx, coef=(0.01, 0.002), topk_w=w, dtopk_w=dw, grad=True, dlogits=l2)
    assert out[3] is l2 and all(torch.equal(a, b) for a, b in zip(r, out))


@pytest.mark.parametrize("T", [40, 3000])
def test_balance_loss_reports_bad_ids(cuda_lib, T):
    g = gen(T)
    E, k = 64, 8
    l, idx = torch.randn(T, E, device=DEV, generator=g), picks(g, T, E, k)
    good = cuda_lib.balance_loss(l, idx, grad=True)
    bad = idx.clone()
    bad[5, 2], bad[T - 1, 0] = E, -1
    ws = torch.zeros(cuda_lib.balance_loss_workspace_size(T, E, k), dtype=torch.uint8, device=DEV)
    w = torch.rand(T, k, device=DEV, generator=g)
    _, counts, probs, _ = cuda_lib.balance_loss(l, bad, grad=True, topk_w=w, dtopk_w=w, ws=ws)
    assert cuda_lib.last_device_status(ws) == cuda_lib.ERR_DEVICE_CHECK
    want = good[1].clone()
    want[int(idx[5, 2])] -= 1
    want[int(idx[T - 1, 0])] -= 1
    assert torch.equal(counts, want) and torch.equal(probs, good[2])


# ---- streams, graphs ---------------------------------------------------------------------

def _calls(lmoe, g, T=96, H=512, N=264, E=64, k=4):
    x = randn(g, T, H)
    W, b = randn(g, N, H, scale=0.05), randn(g, N, dtype=torch.float32)
    res, dout = randn(g, T, N, dtype=torch.float32), randn(g, T, N)
    pre = randn(g, T, N)
    w = randn(g, H, dtype=torch.float32)
    mean, rstd = torch.randn(T, device=DEV, generator=g), torch.rand(T, device=DEV, generator=g)
    l, idx = torch.randn(T, E, device=DEV, generator=g), picks(g, T, E, k)
    tw = torch.rand(T, k, device=DEV, generator=g)
    return [lambda **a: lmoe.linear_act_bf16(x, W, b, "gelu", res, pre=True, **a),
            lambda **a: lmoe.linear_act_bf16_backward(dout, x, W, "silu", pre, **a),
            lambda **a: lmoe.layer_norm(x, w, stats=True, **a),
            lambda **a: lmoe.layer_norm_backward(x, x, mean, rstd, w, **a),
            lambda **a: lmoe.balance_loss(l, idx, grad=True, topk_w=tw, dtopk_w=tw, **a)]


@pytest.mark.parametrize("which", range(5))
def test_on_another_stream_and_in_a_graph(cuda_lib, which):
    call = _calls(cuda_lib, gen(1))[which]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    got = call(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = call()
        out2 = call()
    for _ in range(3):
        for t in [*out, *out2]:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)) and all(torch.equal(a, b) for a, b in zip(want, out2))


# ---- together -------------------------------------------------------------------------------

def test_a_training_step_of_a_routers_neighbourhood(cuda_lib):
    """Norm -> projection with function -> router -> losses, and back through the gate weights, the projection and
    the norm to the stream; every step against its formula in 64 bits on the values the step was given, the whole
    against 64-bit automatic differentiation."""
    lmoe = cuda_lib
    g = gen(12)
    T, H, d, E, k = 200, 520, 256, 64, 8
    stream = stream_rows(g, T, H, torch.float32)
    w, b = 1 + 0.1 * torch.randn(H, device=DEV, generator=g), 0.1 * torch.randn(H, device=DEV, generator=g)
    W, bias = randn(g, d, H, scale=H ** -0.5), 0.1 * torch.randn(d, device=DEV, generator=g)
    Wr = torch.randn(E, d, device=DEV, generator=g) * d ** -0.5
    mask = torch.rand(T, device=DEV, generator=g) < 0.8
    coef = (0.5, 0.05)
    n, mean, rstd = lmoe.layer_norm(stream, w, b, stats=True)
    lat, pre = lmoe.linear_act_bf16(n, W, bias, "gelu", pre=True)
    logits, idx, gate = lmoe.route(lat, Wr, k)
    dgate = torch.randn(T, k, device=DEV, generator=g) * 0.01
    loss, counts, probs, dl = lmoe.balance_loss(logits, idx, mask, coef, True, gate, dgate)
    assert torch.equal(counts.long(), torch.bincount(idx[mask].reshape(-1).long(), minlength=E))
    Wrb = Wr.bfloat16()
    dlat, dWr, _ = lmoe.linear_act_bf16_backward(dl, lat, Wrb, want_dbias=False, dW=torch.empty(E, d, device=DEV))
    dn, dW, dbias = lmoe.linear_act_bf16_backward(dlat, n, W, "gelu", pre)
    add = torch.randn(T, H, device=DEV, generator=g) * 1e-4
    dstream, dw, db = lmoe.layer_norm_backward(dn, stream, mean, rstd, w, add)
    # the whole in 64 bits, by automatic differentiation
    leaf = lambda t: t.detach().to(D).requires_grad_()
    s6, w6, b6, W6, bias6, Wr6 = map(leaf, (stream, w, b, W, bias, Wr))
    c = s6 - s6.mean(1, keepdim=True)
    n6 = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w6 + b6
    z6 = n6 @ W6.t() + bias6
    l6 = (z6 * phi(z6)) @ Wr6.t()
    m = mask[:, None].to(D)
    N = int(mask.sum())
    f = counts.to(D) * E / (k * N)
    p6 = torch.softmax(l6, 1) * m
    bal = (p6.sum(0) / N * f).sum()
    zl = (torch.logsumexp(l6, 1).square() * m[:, 0]).sum() / N
    total = coef[0] * bal + coef[1] * zl + (torch.softmax(l6.gather(1, idx.long()), 1) * dgate.to(D) * m).sum() + (s6 * add.to(D)).sum()
    total.backward()
    # the losses: logits carry the roundings of n and lat (bf16), 2^-7 relative each in norm
    bal, zl = float(bal.detach()), float(zl.detach())
    assert abs(float(loss[0]) - bal) < 1e-3 * bal and abs(float(loss[1]) - zl) < 1e-2 * zl
    # gradients: five bf16 roundings on the way (n, lat, dl or Wr, dlat, dz), below 2^-8 in norm each, and W's products
    # keep norms apart by at most their condition, measured here by the ratio of 1: 6 half steps with room for two
    for got, ref in ((dWr, Wr6.grad), (dW, W6.grad), (dbias, bias6.grad), (dw, w6.grad), (db, b6.grad), (dstream, s6.grad)):
        assert float((got.to(D) - ref).norm()) < 8 * HALF * float(ref.norm())


@pytest.mark.parametrize("E", [896, 50])
def test_balance_loss_rows_of_extreme_logits(cuda_lib, E):
    """Rows of one value have even probabilities whatever the value, the type's lowest and largest among them; a
    difference that overflows is a probability of zero."""
    T, k = 30, 2
    big = torch.finfo(torch.float32).max
    l = torch.zeros(T, E, device=DEV)
    l[0], l[1], l[2], l[3] = -big, big, -1e38, 300.0
    l[4], l[4, 3] = -big, big
    idx = picks(gen(E), T, E, k)
    _, counts, probs, d = cuda_lib.balance_loss(l, idx, coef=(1.0, 0.0), grad=True)
    p = torch.softmax(l.to(D), 1)
    f = counts.to(D) / (k * T) * E
    within(probs, p.mean(0), 800 * U * p.mean(0))
    within(d, p * (f - (p * f).sum(1, keepdim=True)) / T, 400 * U / T * p * (f + (p * f).sum(1, keepdim=True)) + TINY)


# ---- offsets beyond 32 bits ------------------------------------------------------------------

def test_linear_act_backward_beyond_2_31_elements(cuda_lib):
    rows, K, N = 66000, 8, 33000
    g = gen(5)
    x, W, pre = randn(g, rows, K), randn(g, N, K), randn(g, rows, N)
    dout = randn(g, rows, N, scale=0.01)
    dx, dW, db = cuda_lib.linear_act_bf16_backward(dout, x, W, "relu", pre)
    assert cuda_lib.last_call_status() == cuda_lib.OK
    for r0 in (0, rows - 33):
        dz = dout[r0:r0 + 33].to(D) * (pre[r0:r0 + 33] > 0)  # bf16 as it is: relu's slope rounds nothing
        ref = dz @ W.to(D)
        tol = (N + 2) * U * (dz.abs() @ W.to(D).abs())
        within(dx[r0:r0 + 33], ref, tol + (ref.abs() + tol) * HALF)
    for n0 in (0, N - 9):
        dz = dout[:, n0:n0 + 9].to(D) * (pre[:, n0:n0 + 9] > 0)
        ref = dz.t() @ x.to(D)
        tol = (rows + 2) * U * (dz.abs().t() @ x.to(D).abs())
        within(dW[n0:n0 + 9], ref, tol + (ref.abs() + tol) * HALF)
        within(db[n0:n0 + 9], dz.sum(0), (rows + 2) * U * dz.abs().sum(0))


def test_layer_norm_beyond_2_31_elements(cuda_lib):
    T, H = 263000, 8192
    x = torch.empty(T, H, device=DEV, dtype=torch.bfloat16).normal_(generator=gen(6))
    out, mean, rstd = cuda_lib.layer_norm(x, stats=True)
    dx, _, _ = cuda_lib.layer_norm_backward(out, x, mean, rstd, want_params=False)
    for t0 in (0, T - 5):
        v = x[t0:t0 + 5].to(D)
        m, var = v.mean(1, keepdim=True), v.var(1, unbiased=False, keepdim=True)
        ref = (v - m) / (var + 1e-5).sqrt()
        within(out[t0:t0 + 5], ref, ref.abs() * (HALF + 80 * U) + 100 * U)
        small = cuda_lib.layer_norm_backward(out[t0:t0 + 5].contiguous(), x[t0:t0 + 5].contiguous(), mean[t0:t0 + 5].contiguous(),
                                             rstd[t0:t0 + 5].contiguous(), want_params=False)[0]
        assert torch.equal(dx[t0:t0 + 5], small)


def test_balance_loss_beyond_2_31_logits(cuda_lib):
    T, E, k = 1_060_000, 2048, 1
    l = torch.empty(T, E, device=DEV).normal_(generator=gen(7))
    first, last = l[:3].clone(), l[-3:].clone()
    idx = torch.randint(0, E, (T, k), device=DEV, generator=gen(8)).to(torch.int32)
    loss, counts, probs, d = cuda_lib.balance_loss(l, idx, coef=(1.0, 0.5), grad=True, dlogits=l)
    assert d is l and torch.equal(counts.long(), torch.bincount(idx[:, 0].long(), minlength=E))
    f = counts.to(D) * E / (k * T)
    for rows, got in ((first, d[:3]), (last, d[-3:])):
        lse = torch.logsumexp(rows.to(D), 1, keepdim=True)
        p = torch.exp(rows.to(D) - lse)
        sf = (p * f).sum(1, keepdim=True)
        ref = p * ((f - sf) + lse) / T
        within(got, ref, 400 * U * p * (f + sf + lse.abs() + 1) / T + TINY)
    assert abs(float(probs.sum()) - 1) < 1e-4 and abs(float(loss[0]) - 1) < 1e-2


# ---- edges ---------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,N", [(5, 45), (200, 45), (700, 1001), (300, 1004), (64, 264), (65, 264)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_linear_act_in_place_where_rows_start_anywhere(cuda_lib, rows, N, dt):
    g = gen(rows + N)
    x, W, b = randn(g, rows, 200), randn(g, N, 200, scale=0.07), randn(g, N, dtype=torch.float32)
    res = randn(g, rows, N, dtype=dt)
    want = cuda_lib.linear_act_bf16(x, W, b, "gelu_tanh", res, pre=True)
    r2 = res.clone()
    got = cuda_lib.linear_act_bf16(x, W, b, "gelu_tanh", r2, out=r2, pre=True)
    assert torch.equal(want[0], r2) and torch.equal(want[1], got[1])


def test_workspaces_may_hold_anything_behind_the_status(cuda_lib):
    """One workspace for all the calls, full of NaN patterns: each writes what it reads of it, and none touches the
    status word."""
    lmoe = cuda_lib
    g = gen(21)
    x, W, d = randn(g, 128, 7168), randn(g, 200, 7168, scale=0.01), randn(g, 128, 200)
    l, idx = torch.randn(9000, 64, device=DEV, generator=g), picks(g, 9000, 64, 4)
    mean, rstd = torch.randn(128, device=DEV, generator=g), torch.rand(128, device=DEV, generator=g)
    calls = [(lambda ws: lmoe.linear_act_bf16(x, W, act="silu", pre=True, ws=ws), lmoe.linear_act_workspace_size(128, 7168, 200)),
             (lambda ws: lmoe.linear_act_bf16_backward(d, x, W, "gelu", d, ws=ws),
              lmoe.linear_act_backward_workspace_size(128, 7168, 200)),
             (lambda ws: lmoe.layer_norm_backward(x, x, mean, rstd, ws=ws), lmoe.layer_norm_backward_workspace_size(128, 7168)),
             (lambda ws: lmoe.balance_loss(l, idx, grad=True, ws=ws), lmoe.balance_loss_workspace_size(9000, 64, 4))]
    ws = torch.full((max(n for _, n in calls),), 0xFF, dtype=torch.uint8, device=DEV)
    ws[:256] = 0
    for call, n in calls:
        want = [t.clone() for t in call(torch.zeros(n, dtype=torch.uint8, device=DEV))]
        got = call(ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert lmoe.last_device_status(ws) == lmoe.OK
        ws[256:] = 0xFF


def test_calls_at_once_on_two_streams(cuda_lib):
    """Calls that overlap on the GPU, each on a workspace of its own."""
    a, b = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    calls = _calls(cuda_lib, gen(31), T=700, H=1032, N=1000, E=96, k=4)
    want = [[t.clone() for t in c()] for c in calls]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(a):
            got.append([c() for c in calls])
        with torch.cuda.stream(b):
            got.append([c() for c in reversed(calls)][::-1])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for w, o in zip(want, g) for x, y in zip(w, o))


def test_the_binding_refuses_strides_types_and_shapes(cuda_lib):
    lmoe = cuda_lib
    g = gen(41)
    x, W, f = randn(g, 6, 64), randn(g, 16, 64), torch.zeros(6, 64, device=DEV)
    d, i = randn(g, 6, 16), torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    s = torch.zeros(6, device=DEV)
    wide = randn(g, 6, 128)[:, :64]
    bad = [lambda: lmoe.linear_act_bf16(wide, W), lambda: lmoe.linear_act_bf16(f, W), lambda: lmoe.linear_act_bf16(x, W[:, :32]),
           lambda: lmoe.linear_act_bf16(x, W, bias=torch.zeros(8, device=DEV)), lambda: lmoe.linear_act_bf16(x, W, res=f),
           lambda: lmoe.linear_act_bf16(x, W, out=torch.zeros(6, 16, device=DEV, dtype=torch.float16)),
           lambda: lmoe.linear_act_bf16(x, W, pre=f), lambda: lmoe.linear_act_bf16(x, W, ws=f),
           lambda: lmoe.linear_act_bf16(x.cpu(), W), lambda: lmoe.linear_act_bf16(x, W.cpu()),
           lambda: lmoe.linear_act_bf16_backward(d, x, W, "silu"), lambda: lmoe.linear_act_bf16_backward(d, x, W, "none", d),
           lambda: lmoe.linear_act_bf16_backward(d.t().contiguous(), x, W), lambda: lmoe.layer_norm(wide),
           lambda: lmoe.layer_norm(x, w=x[0]), lambda: lmoe.layer_norm(x, mean=s[:3], rstd=s),
           lambda: lmoe.layer_norm_backward(f, f, s, s), lambda: lmoe.layer_norm_backward(x, f, s, s, add=x),
           lambda: lmoe.layer_norm_backward(x, f, s[:5], s), lambda: lmoe.balance_loss(x, i), lambda: lmoe.balance_loss(f, i.long()),
           lambda: lmoe.balance_loss(f, i, mask=s), lambda: lmoe.balance_loss(f, i, grad=True, topk_w=torch.zeros(6, 2, device=DEV)),
           lambda: lmoe.balance_loss(f, i, scale=s[:1]), lambda: lmoe.balance_loss(f, i, grad=True, scale=s),
           lambda: lmoe.balance_loss(f[:5], i)]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")
    for call in (lambda: lmoe.linear_act_bf16(randn(g, 6, 60), randn(g, 16, 60)), lambda: lmoe.layer_norm(randn(g, 6, 60)),
                 lambda: lmoe.balance_loss(f, torch.zeros(6, 33, dtype=torch.int32, device=DEV)),
                 lambda: lmoe.linear_act_bf16(x, W, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(lmoe.LmoeError):
            call()
