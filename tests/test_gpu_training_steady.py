"""The linear layer with functions, layer norm and the balance loss where their kernels settle into their steady state:
warps and blocks that walk over several rows, weights kept in registers, rows of four columns more than eights, and
functions far out held to their tails.  Tolerances as in test_gpu_training_operators."""
import pytest
import torch

import test_gpu_training_operators as ops
from test_gpu_operators import D, DEV, U, gen, randn, within

pytestmark = pytest.mark.gpu


# ---- balance loss: from 152 x 24 rows (up to 256 experts), x 16 (512), x 12 (1024) and x 8 on a warp has several rows ----

ROWS = [(3800, 60, 8), (8000, 130, 4), (12000, 256, 8), (5000, 300, 8), (6000, 512, 4), (4000, 640, 16), (4000, 896, 16),
        (6000, 896, 16), (4100, 1023, 5), (4000, 1024, 32), (3000, 1149, 20), (2600, 2048, 32)]


@pytest.mark.parametrize("T,E,k", ROWS)
@pytest.mark.parametrize("mask", ["none", "random", "early", "late", "turns"])
def test_balance_loss_of_several_rows_a_warp(cuda_lib, T, E, k, mask):
    g = gen(T + E)
    l = 2 * torch.randn(T, E, device=DEV, generator=g)
    idx = ops.picks(g, T, E, k)
    w = torch.softmax(torch.randn(T, k, device=DEV, generator=g), 1).contiguous()
    dw = torch.randn(T, k, device=DEV, generator=g)
    t = torch.arange(T, device=DEV)
    keep = {"none": None, "random": torch.rand(T, device=DEV, generator=g) < 0.5, "early": t >= T // 2, "late": t < T // 3,
            "turns": t // 900 % 2 == 1}[mask]
    if keep is not None:  # padding holds anything
        l[~keep], w[~keep], dw[~keep], idx[~keep] = float("nan"), float("inf"), float("nan"), 2 ** 31 - 1
        l[~keep, ::2] = float("inf")
    a = ops.check_balance(cuda_lib, l, idx, keep, w=w, dw=dw)
    b = ops.check_balance(cuda_lib, l, idx, keep, grad=False)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    l2 = l.clone()
    c = cuda_lib.balance_loss(l2, idx, keep, coef=(0.01, 0.002), topk_w=w, dtopk_w=dw, dlogits=l2)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


@pytest.mark.parametrize("T,E,k", [(256, 896, 16), (257, 896, 16), (767, 300, 16), (768, 896, 16), (769, 896, 16), (768, 61, 16),
                                   (769, 61, 16), (384, 2048, 32), (385, 2048, 32)])
def test_balance_loss_about_the_picks_that_a_block_counts(cuda_lib, T, E, k):
    """4096 and 12288 picks: counted by every block or by a kernel of their own."""
    g = gen(T + E)
    l, idx = torch.randn(T, E, device=DEV, generator=g), ops.picks(g, T, E, k)
    w, dw = torch.rand(T, k, device=DEV, generator=g), torch.randn(T, k, device=DEV, generator=g)
    ops.check_balance(cuda_lib, l, idx, torch.rand(T, device=DEV, generator=g) < 0.8, w=w, dw=dw)


@pytest.mark.parametrize("T,E,k", [(6000, 896, 16), (9000, 130, 32), (4000, 2048, 8)])
def test_balance_loss_of_several_rows_with_experts_twice(cuda_lib, T, E, k):
    """A row that names an expert twice, then one that does not, in one warp: the gate weights' share of one row does
    not reach the next."""
    g = gen(T)
    l, idx = torch.randn(T, E, device=DEV, generator=g), ops.picks(g, T, E, k)
    twice = torch.rand(T, device=DEV, generator=g) < 0.5
    idx[twice] = torch.randint(0, max(k // 2, 1), (int(twice.sum()), k), device=DEV, generator=g).to(torch.int32)
    w, dw = torch.rand(T, k, device=DEV, generator=g), torch.randn(T, k, device=DEV, generator=g)
    ops.check_balance(cuda_lib, l, idx, torch.rand(T, device=DEV, generator=g) < 0.8, w=w, dw=dw)


# ---- layer norm: bf16 rows that a block walks over (more than 1216, 1032 to 8192 columns) ----

@pytest.mark.parametrize("T,H", [(1217, 1032), (2500, 1032), (1300, 2056), (5000, 2048), (3000, 3584), (1217, 7168),
                                 (2500, 7168), (1500, 8184), (1300, 8192)])
@pytest.mark.parametrize("params", ["wb", "w", "b", ""])
def test_layer_norm_of_several_rows_a_block(cuda_lib, T, H, params):
    ops.test_layer_norm(cuda_lib, T, H, torch.bfloat16, params)


@pytest.mark.parametrize("H", [1032, 7168])
def test_layer_norm_of_several_rows_keeps_bad_rows_to_themselves(cuda_lib, H):
    g = gen(H)
    x = randn(g, 3000, H)
    w, b = randn(g, H, dtype=torch.float32), randn(g, H, dtype=torch.float32)
    want = cuda_lib.layer_norm(x, w, b)
    bad = torch.tensor([0, 7, 608, 1216, 2998], device=DEV)
    x[bad, H - 1] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan"), float("inf")], device=DEV).bfloat16()
    out = cuda_lib.layer_norm(x, w, b)
    good = torch.ones(3000, dtype=torch.bool, device=DEV)
    good[bad] = False
    assert torch.equal(out[good], want[good]) and bool(out[bad].isnan().all())


# ---- linear: rows of outputs and residual that start on 16 bytes though N % 8 == 4 (fp32 both, no pre) ----

@pytest.mark.parametrize("rows,K,N", [(65, 264, 300), (200, 72, 1004), (700, 512, 1004), (128, 7168, 1004), (100, 7168, 516),
                                      (5000, 128, 260), (3, 264, 300), (40, 4096, 1004)])
@pytest.mark.parametrize("res", [False, True])
def test_linear_act_fp32_rows_of_fours(cuda_lib, rows, K, N, res):
    g = gen(rows + N)
    x, W, b = randn(g, rows, K), randn(g, N, K, scale=K ** -0.5), randn(g, N, dtype=torch.float32)
    r = randn(g, rows, N, dtype=torch.float32) if res else None
    out, _ = ops.check_linear(cuda_lib, x, W, b, "gelu", r, False, torch.float32)
    if res:
        r2 = r.clone()
        assert torch.equal(cuda_lib.linear_act_bf16(x, W, b, "gelu", r2, out=r2), out)


# ---- functions far out ----

@pytest.mark.parametrize("act", ops.ACTS)
@pytest.mark.parametrize("rows", [4, 200])
def test_linear_act_far_values_by_their_tails(cuda_lib, act, rows):
    """fn(z) = max(z, 0) - |z| tail(|z|): the argument's error (8 of its own u a unit, 16 u beside) is one of the tail
    alone, the sum is rounded twice at most.  z is one product by 1, so exact."""
    K = N = 64
    x = torch.zeros(rows, K, device=DEV, dtype=torch.bfloat16)
    x[:, 0] = 1
    W = torch.zeros(N, K, device=DEV, dtype=torch.bfloat16)
    W[:, 0] = torch.cat([torch.linspace(-14, 14, 50), torch.tensor([-3e4, 3e4, -120., 120., -88., 88., -1e18, 1e18, -30., 30.,
                                                                   1e30, -1e30, 1e-30, -1e-30])]).to(DEV).bfloat16()
    out, pre = cuda_lib.linear_act_bf16(x, W, act=act, out=torch.empty(rows, N, device=DEV), pre=True)
    z = W[:, 0].to(D)[None].expand(rows, N)
    assert torch.equal(pre.to(D), z)
    a = z.abs()
    if act in ("none", "relu"):
        assert torch.equal(out.to(D), z if act == "none" else z.clamp_min(0))
        return
    u = ops.C * (a + 0.044715 * a ** 3)
    arg, tail = {"silu": (a, a * torch.sigmoid(-a)), "gelu": (a * a, a * ops.phi(-a)), "gelu_tanh": (u, a * torch.sigmoid(-u))}[act]
    tail = torch.where(tail > 0, tail, torch.zeros_like(tail))  # (infinity times zero far out)
    factor = torch.where(tail > 0, (16 + 8 * arg) * U, torch.zeros_like(arg))
    ref = z.clamp_min(0) - tail
    within(out, ref, 2 * U * ref.abs() + factor * tail + ops.TINY)


@pytest.mark.parametrize("act", ops.ACTS)
@pytest.mark.parametrize("N", [16, 13])
def test_values_and_slopes_at_infinity(cuda_lib, act, N):
    """A column whose bias is -infinity (masked) or infinity: the function's limit, and 0 or 1 for its slope, so that the
    gradients of a masked column are zero and no other column's change.  A NaN stays a NaN."""
    g = gen(N)
    rows, K = 70, 24
    x, W, bias = randn(g, rows, K), randn(g, N, K), randn(g, N, dtype=torch.float32)
    dout = randn(g, rows, N)
    want = cuda_lib.linear_act_bf16(x, W, bias, act, pre=True)
    bias[3], bias[7], bias[9] = -float("inf"), float("inf"), float("nan")
    out, pre = cuda_lib.linear_act_bf16(x, W, bias, act, pre=True)
    rest = [n for n in range(N) if n not in (3, 7, 9)]
    assert torch.equal(out[:, rest], want[0][:, rest])
    assert bool((out[:, 3] == (-float("inf") if act == "none" else 0)).all()) and bool((out[:, 7] == float("inf")).all())
    assert bool(out[:, 9].isnan().all())
    saved = None if act == "none" else pre
    _, _, db = cuda_lib.linear_act_bf16_backward(dout, x, W, act, saved)
    low = 1.0 if act == "none" else 0.0
    within(db[[3]], low * dout[:, 3].to(D).sum()[None], (rows + 2) * U * dout[:, 3].to(D).abs().sum()[None])
    within(db[[7]], dout[:, 7].to(D).sum()[None], (rows + 2) * U * dout[:, 7].to(D).abs().sum()[None])
    if act == "none":
        return
    assert bool(db[9].isnan())
    pre[:, 9] = 0  # without the NaN: masked columns add nothing to dx, and their dW is zero
    dx, dW, _ = cuda_lib.linear_act_bf16_backward(dout, x, W, act, pre)
    pre[:, 3], masked = -200.0, W.clone()
    masked[3] = 0
    also = cuda_lib.linear_act_bf16_backward(dout, x, masked, act, pre)
    assert torch.equal(dx, also[0]) and not bool(dW[3].any()) and bool(torch.isfinite(dW).all())
