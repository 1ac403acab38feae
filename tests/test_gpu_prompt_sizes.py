"""The MXFP4 linear and the block on a residual stream at a prompt's sizes."""
import pytest
import torch

import lmoe_inputs as gen
from _util import device_bank
from test_gpu_operators import check_linear, gen as generator, mx_weights, randn
from test_gpu_residual_block import _block, _by_hand

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("rows,K,N", [(8192, 7168, 3584), (2049, 3584, 7168), (20000, 512, 136)])
def test_linear_mxfp4_of_a_prompt(cuda_lib, rows, K, N):
    g = generator(rows)
    q, s, W = mx_weights(cuda_lib, g, N, K)
    check_linear(cuda_lib, randn(g, rows, K), W, q, s)


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("T,dt", [(300, torch.float32), (2050, torch.bfloat16), (9000, torch.bfloat16)])
def test_block_of_a_prompt_is_its_calls(cuda_lib, mx, T, dt):
    """As for few tokens, with the layer's combine fused into the expert GEMM.  That one adds a token's experts in any
    order; with one expert a token there is no order, and the block equals its calls bit for bit."""
    lmoe = cuda_lib
    g = generator(T)
    wl = gen.WORKLOADS["tiny"]
    layer = lmoe.Layer(torch.from_numpy(gen.router_f32(wl)).to(DEV), device_bank(wl, DEV), k=1)
    b = _block(lmoe, layer, wl, 1088, mx, g)
    res, nw = torch.randn(T, 1088, device=DEV, generator=g).to(dt), torch.rand(1088, device=DEV, generator=g) + 0.5
    tok = torch.rand(T, 1, device=DEV, generator=g)
    for gate, next_w in ((None, nw), (tok, None)):
        r, n = b.forward(res, gate=gate, next_w=next_w)
        assert b.device_status() == lmoe.OK
        r2, n2 = _by_hand(lmoe, b, res, None, gate, next_w)
        assert torch.equal(r, r2)
        assert (n is None and n2 is None) or torch.equal(n, n2)
