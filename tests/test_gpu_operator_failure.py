"""The failure path of the MXFP4 linear and the grouped products: the first
pipeline stage of every CTA is withheld (lmoe_set_wait_test, 10 ms limit), the
waits run out, the status word says so, and the next calls in the same context
are right.  One case for each kernel form: rows split in the kernel or before
it, K shared by a cluster or not, single CTAs and pairs, rows in order and
gathered."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _linear(lmoe, rows, K, N):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    lin = lmoe.LinearMxfp4(torch.randn(N, K, device=DEV, generator=g))
    x = torch.randn(rows, K, device=DEV, generator=g).bfloat16()
    return (lambda ws: lin.forward(x, ws=ws)), lmoe.linear_mxfp4_workspace_size(rows, K, N)


def _grouped(lmoe, rows, E, K, N, gather, swiglu):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    P = rows * E
    off = torch.arange(0, P + 1, rows, dtype=torch.int32, device=DEV)
    perm = torch.randperm(P, device=DEV, generator=g).to(torch.int32) if gather else None
    x = torch.randn(P, K, device=DEV, generator=g).bfloat16()
    W, V = ((torch.randn(E, N, K, device=DEV, generator=g) * K ** -0.5).bfloat16() for _ in range(2))
    if swiglu:
        return (lambda ws: lmoe.grouped_swiglu_bf16(x, W, V, off, perm, 1, ws=ws)), 256
    return (lambda ws: lmoe.grouped_linear_bf16(x, W, off, perm, 1, ws=ws)), 256


CASES = {
    "linear_1_clustered": lambda m: _linear(m, 1, 7168, 256),
    "linear_12": lambda m: _linear(m, 12, 1024, 40000),
    "linear_40_clustered": lambda m: _linear(m, 40, 4096, 512),
    "linear_400": lambda m: _linear(m, 400, 1024, 7168),
    "grouped_1_clustered": lambda m: _grouped(m, 1, 2, 2048, 256, False, False),
    "grouped_20_gathered": lambda m: _grouped(m, 20, 40, 1024, 640, True, False),
    "swiglu_100": lambda m: _grouped(m, 100, 20, 1024, 320, True, True),
    "grouped_300_pairs": lambda m: _grouped(m, 300, 8, 1024, 1100, True, False),
    "swiglu_300_pairs": lambda m: _grouped(m, 300, 8, 1024, 640, False, True),
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
    assert torch.equal(call(ws), want)
    assert lmoe.last_device_status(ws) == lmoe.OK
