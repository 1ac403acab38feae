"""Bounded waits of the linear layer's kernels: all roles are whole warps, whose waits
answer by one vote of the warp (mbar_wait_warp); only the drain is waited for by one
elected thread.  Read from the sources: no GPU is made to run into the fault."""
import pytest

from test_warp_waits import waits


@pytest.mark.parametrize("name", ["k_linear_act.cu", "k_linear_few.cu"])
def test_linear_kernels_wait_by_warps(name):
    alone = [w for w in waits(name) if "mbar_wait(drain," not in w[1]]
    assert not alone, alone
