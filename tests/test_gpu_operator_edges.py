"""Values at the edges of the formats, and arguments that are no plain value, in
the norms, the MXFP4 linear and the grouped products.

Tolerances as in test_gpu_operators.py: U = 2^-24, a bf16 result off by at most
half a step (2^-8 of its value, or 2^-134 among the subnormals)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U, HALF = 2.0 ** -24, 2.0 ** -8
D = torch.float64


@pytest.mark.parametrize("rows", [3, 40, 300])
def test_gated_pair_far_below_zero(cuda_lib, rows):
    """silu(g) u where exp(-g) comes near fp32's largest value and passes it.  One product a gate, so g and u are exact:
    what is left is the exponential (2 ulp, absolute 2^-148 where it is subnormal), the add, the division and the
    products (below 16 U), and the output's rounding."""
    n = 128
    gate = -torch.linspace(80, 104, n, device=DEV).bfloat16()
    up = torch.tensor([1.0, -3.0, 8.0, 0.5], device=DEV).bfloat16().repeat(n // 4)
    Wg, Wu = torch.zeros(1, n, 8, device=DEV).bfloat16(), torch.zeros(1, n, 8, device=DEV).bfloat16()
    Wg[0, :, 0], Wu[0, :, 1] = gate, up
    x = torch.zeros(rows, 8, device=DEV).bfloat16()
    x[:, :2] = 1
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    h = cuda_lib.grouped_swiglu_bf16(x, Wg, Wu, off)
    g, u = gate.to(D), up.to(D)
    ref = g * torch.exp(g) / (1 + torch.exp(g)) * u
    tol = ref.abs() * (HALF + 16 * U) + 2.0 ** -134 + 2.0 ** -148 * (g * u).abs()
    assert bool(((h.to(D) - ref).abs() <= tol).all())


def test_gated_pair_far_above_zero(cuda_lib):
    """silu(g) = g up to fp32's exponential's end and beyond."""
    n = 64
    gate = torch.linspace(20, 200, n, device=DEV).bfloat16()
    Wg, Wu = torch.zeros(1, n, 8, device=DEV).bfloat16(), torch.zeros(1, n, 8, device=DEV).bfloat16()
    Wg[0, :, 0], Wu[0, :, 1] = gate, 1
    x = torch.zeros(2, 8, device=DEV).bfloat16()
    x[:, :2] = 1
    h = cuda_lib.grouped_swiglu_bf16(x, Wg, Wu, torch.tensor([0, 2], dtype=torch.int32, device=DEV))
    assert torch.equal(h, gate.expand(2, n))


@pytest.mark.parametrize("rows", [2, 20, 200])
def test_linear_mxfp4_near_the_largest_values(cuda_lib, rows):
    """bf16's largest magnitudes and the smallest ones through weights of 1/2 and 1/4: sums as large as are sure to stay
    finite, exact (one or two terms an output)."""
    lmoe, K, N = cuda_lib, 64, 32
    big = torch.finfo(torch.bfloat16).max
    # output n: x[n] / 2 + x[n + 32] / 4
    q = torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV)
    n = torch.arange(N, device=DEV)
    for c in (n, n + 32):
        q[n, c // 2] = torch.where(c % 2 == 0, 0x02, 0x20).to(torch.uint8)  # 1.0
    s = torch.tensor([126, 125], dtype=torch.uint8, device=DEV).expand(N, 2).contiguous()
    qt, st = lmoe.repack_mxfp4(q, s, 1, N, K)
    x = torch.zeros(rows, K, device=DEV).bfloat16()
    x[:, :32] = torch.tensor([big, -big, 2.0 ** 127, -(2.0 ** 126)], device=DEV).bfloat16().repeat(8)
    x[1, 32:] = x[1, :32]
    out = lmoe.linear_mxfp4(x, qt, st, N).to(D)
    xd = x.to(D)
    ref = xd[:, :32] / 2 + xd[:, 32:] / 4
    assert torch.equal(out, ref.bfloat16().to(D)) and bool(torch.isfinite(out).all())
    # the smallest: subnormal elements beside nothing larger are held exactly; half of one is rounded once
    tiny = torch.finfo(torch.bfloat16).smallest_normal
    x[:, :32] = torch.tensor([tiny, -tiny * 1.5, tiny * 2.0 ** -4, 4 * tiny], device=DEV).bfloat16().repeat(8)
    x[:, 32:] = 0
    out, ref = lmoe.linear_mxfp4(x, qt, st, N).to(D), x[:, :32].to(D) / 2
    # a product below fp32's normal range may be flushed by the tensor core: 2^-126
    assert bool(((out - ref).abs() <= 2.0 ** -126 + 2.0 ** -134).all())
    assert torch.equal(out[:, 3::4], ref[:, 3::4])


def test_gather_without_a_truth_value_is_refused(cuda_lib):
    """An argument whose truth value raises: that error, and no result beside it."""
    x, W = torch.ones(4, 64, device=DEV).bfloat16(), torch.ones(1, 16, 64, device=DEV).bfloat16()
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    perm = torch.arange(4, dtype=torch.int32, device=DEV)
    with pytest.raises(RuntimeError, match="ambiguous"):
        cuda_lib.grouped_linear_bf16(x, W, off, perm, gather=torch.ones(2))
    for gather in (True, torch.ones(1), 1):
        assert bool((cuda_lib.grouped_linear_bf16(x, W, off, perm, gather=gather) == 64).all())
