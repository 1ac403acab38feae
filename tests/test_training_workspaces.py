"""A workspace for the largest batch serves every smaller one: the sizes that the linear layer's, layer norm's and the
balance loss' calls ask for never fall as the rows grow (no GPU needed)."""
import pytest

ROWS = sorted({*range(0, 2200), *range(2200, 20000, 37), *range(20000, 400000, 1777), 1 << 20, 1 << 22})


@pytest.fixture(scope="module")
def lmoe():
    from top_routing_mxfp4_gb300 import build
    build.build()
    from top_routing_mxfp4_gb300 import lmoe
    return lmoe


def check(size):
    most = 0
    for r in ROWS:
        n = size(r)
        assert n >= most, f"{n} bytes for {r} rows, {most} for fewer"
        most = n


@pytest.mark.parametrize("K,N", [(3584, 7168), (7168, 3584), (1056, 1000), (512, 512), (7168, 256), (128, 3000), (8, 1),
                                 (256, 20011), (16384, 72)])
def test_linear(lmoe, K, N):
    check(lambda r: lmoe.linear_act_workspace_size(r, K, N))
    check(lambda r: lmoe.linear_act_backward_workspace_size(r, K, N))


@pytest.mark.parametrize("H", [8, 256, 512, 520, 1024, 3584, 7168, 8192, 8200, 32768])
def test_layer_norm(lmoe, H):
    check(lambda r: lmoe.layer_norm_backward_workspace_size(r, H))


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (64, 8), (896, 16), (2048, 32)])
def test_balance_loss(lmoe, E, k):
    check(lambda r: lmoe.balance_loss_workspace_size(r, E, k))
