"""The failure path of the kernel forms that tests/test_gpu_operator_failure.py
does not reach: items handed out by the counter (the feeding warp's wait, the
wait for an item, a pair's barriers across its two CTAs), 16-row tiles with K
shared by two, four and no other CTAs, 64-row tiles.  The first pipeline stage of
every CTA is withheld with a 10 ms limit (lmoe_set_wait_test); the short
reductions leave the producers waiting for an item rather than for a stage.  The
status says so and the next call in the same context is right."""
import pytest
import torch

from test_gpu_operator_failure import _grouped

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# rows an expert, experts, K, N (weight tiles of 128, gated 64, pairs twice that), gathered, gated.  At 152 SMs the
# counter takes over from 608 items on (304 for pairs).
CASES = {
    "fed_16": (1, 64, 64, 1300, True, False),             # 704 items
    "fed_16_gated": (1, 64, 128, 700, False, True),       # 704
    "fed_32_gathered": (20, 40, 64, 2050, True, False),   # 680 tiles and more
    "fed_128_gated": (100, 64, 128, 700, True, True),     # 704
    "fed_pairs": (500, 4, 64, 10000, True, False),        # 320
    "fed_pairs_in_order": (500, 4, 128, 10000, False, False),
    "fed_pairs_gated": (500, 4, 64, 5000, True, True),    # 320
    "one_cta_16": (1, 100, 1024, 256, True, False),       # 200 items
    "two_ranks_16": (1, 30, 512, 256, True, False),       # 60
    "four_ranks_16": (1, 10, 1024, 192, False, True),     # 30, four chunks a rank
    "tiles_64": (50, 20, 1024, 320, True, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_waits_run_out_in_every_form(cuda_lib, name):
    lmoe = cuda_lib
    call, need = _grouped(lmoe, *CASES[name])
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
    for _ in range(3):
        ws = new_ws()
        assert torch.equal(call(ws), want)
        assert lmoe.last_device_status(ws) == lmoe.OK
