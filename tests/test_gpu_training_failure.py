"""The failure path of the linear layer with bias, function and residual and of its
gradients: the first pipeline stage of every CTA is withheld (lmoe_set_wait_test, 10 ms
limit), the waits run out, the status word says so, and the next calls in the same
context are right.  One case for each kernel form: few rows with K shared by a cluster or
not, 64-, 128- and 256-column tiles, single CTAs and pairs, the reduction in parts, and
the three orders of operands."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _forward(lmoe, rows, K, N):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    x, W = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((rows, K), (N, K)))
    return (lambda ws: [lmoe.linear_act_bf16(x, W, act="silu", ws=ws)]), lmoe.linear_act_workspace_size(rows, K, N)


def _backward(lmoe, rows, K, N, dx, dW):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    x, W, d = (torch.randn(*s, device=DEV, generator=g).bfloat16() for s in ((rows, K), (N, K), (rows, N)))
    call = lambda ws: [t for t in lmoe.linear_act_bf16_backward(d, x, W, "silu", d, dx, dW, True, ws=ws) if t is not None]
    return call, lmoe.linear_act_backward_workspace_size(rows, K, N)


CASES = {
    "few_1_clustered": lambda m: _forward(m, 1, 4096, 256),
    "few_20": lambda m: _forward(m, 20, 192, 512),
    "few_64_clustered": lambda m: _forward(m, 64, 2048, 1024),
    "narrow_tiles": lambda m: _forward(m, 300, 512, 512),
    "parts": lambda m: _forward(m, 128, 7168, 3584),
    "pairs_128": lambda m: _forward(m, 1000, 1024, 2048),
    "pairs_256": lambda m: _forward(m, 4096, 512, 3584),
    "dx": lambda m: _backward(m, 3000, 512, 512, True, False),
    "dW": lambda m: _backward(m, 3000, 512, 520, False, True),
    "dx_dW_pairs": lambda m: _backward(m, 4096, 3584, 1024, True, True),
}


@pytest.mark.parametrize("name", list(CASES))
def test_waits_run_out_and_the_context_stays_usable(cuda_lib, name):
    lmoe = cuda_lib
    call, need = CASES[name](lmoe)
    new_ws = lambda: torch.zeros(need, dtype=torch.uint8, device=DEV)
    want = call(new_ws())
    ws = new_ws()
    lmoe.set_wait_test(True, 20_000_000)  # about 10 ms of SM clocks
    try:
        call(ws)
        torch.cuda.synchronize()
    finally:
        lmoe.set_wait_test(False, 0)
    assert lmoe.last_device_status(ws) == lmoe.ERR_TIMEOUT
    ws = new_ws()
    assert all(torch.equal(a, b) for a, b in zip(call(ws), want))
    assert lmoe.last_device_status(ws) == lmoe.OK
