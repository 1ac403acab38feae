"""Batches of changing size through the linear layer with functions, layer norm and the balance loss: one workspace
for the largest serves them all."""
import pytest
import torch

from test_gpu_operators import DEV, gen, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,N", [(1056, 1000), (3584, 520), (520, 3584)])
def test_one_workspace_for_the_largest_batch(cuda_lib, K, N):
    lmoe = cuda_lib
    most = 6000
    g = gen(K + N)
    W = randn(g, N, K, scale=K ** -0.5)
    fwd = torch.zeros(lmoe.linear_act_workspace_size(most, K, N) + 256, dtype=torch.uint8, device=DEV)
    back = torch.zeros(lmoe.linear_act_backward_workspace_size(most, K, N) + 256, dtype=torch.uint8, device=DEV)
    for ws in (fwd, back):
        ws[-256:] = 0x5A  # behind its end: not written
    for rows in (most, 4901, 1300, 769, 512, 333, 299, 130, 65, 64, 3, 1, most):
        x, dout, pre = randn(g, rows, K), randn(g, rows, N), randn(g, rows, N)
        want = lmoe.linear_act_bf16(x, W, act="silu")
        assert torch.equal(lmoe.linear_act_bf16(x, W, act="silu", ws=fwd[:-256]), want)
        want = lmoe.linear_act_bf16_backward(dout, x, W, "silu", pre)
        got = lmoe.linear_act_bf16_backward(dout, x, W, "silu", pre, ws=back[:-256])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for ws in (fwd, back):
        assert lmoe.last_device_status(ws) == lmoe.OK and bool((ws[-256:] == 0x5A).all())
