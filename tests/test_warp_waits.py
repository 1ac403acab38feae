"""Bounded waits in front of warp-wide instructions.  A wait on an mbarrier may
run out for one lane of a warp and not for another (the barrier completes as the
limit is reached); where the whole warp goes on to elect.sync, __syncwarp, votes
or tcgen05 loads, all lanes have to take the same branch, so the wait's answer is
the warp's (mbar_wait_warp).  Read from the sources: no GPU is made to
run into the fault."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routing_mxfp4_gb300", "csrc")


def waits(name):
    """(line number, line) of every wait by single lanes in a source file, comments taken out."""
    src = open(os.path.join(CSRC, name)).read()
    src = re.sub(r"/\*.*?\*/", lambda m: re.sub(r"[^\n]", " ", m.group()), src, flags=re.S)
    lines = [re.sub(r"//.*", "", l) for l in src.split("\n")]
    return [(i + 1, l.strip()) for i, l in enumerate(lines) if re.search(r"\bmbar_(try_)?wait(_cluster)?\(", l)]


def test_the_warp_wait_branches_by_votes():
    src = open(os.path.join(CSRC, "tc_ptx.cuh")).read()
    for f, look in (("mbar_wait_warp", "mbar_try_wait"), ("mbar_wait_cluster_warp", "mbar_try_wait_cluster")):
        body = re.search(r"bool %s\([^)]*\)\s*\{(.*?)\n\}" % f, src, flags=re.S)
        assert body
        branches = re.findall(r"\b(?:if|while) \((.*)\)", body.group(1))
        assert len(branches) == 3
        for b in branches:
            assert re.match(r"!?__all_sync\(0xFFFFFFFFu, %s\(bar, parity\)\)|__any_sync\(0xFFFFFFFFu, clock64\(\)" % look, b), b


@pytest.mark.parametrize("name", ["k_grouped.cu", "k_linear_mxfp4.cu", "cluster_sum.cuh"])
def test_operator_kernels_wait_by_warps(name):
    """All roles of these kernels are whole warps; only the drain is waited for by one elected thread."""
    alone = [w for w in waits(name) if "mbar_wait(drain," not in w[1]]
    assert not alone, alone


def test_a_lost_item_is_not_the_end_of_the_items():
    """A wait for the next item that runs out sends producers and the MMA warp down their failure path (copies and
    MMAs in flight are waited for before shared and tensor memory go), unlike the end of the items."""
    src = open(os.path.join(CSRC, "k_grouped.cu")).read()
    src = re.sub(r"//.*", "", src)
    fetch = re.search(r"auto next_item = .*?\n    \};", src, flags=re.S).group()
    assert re.search(r"LMOE_ERR_TIMEOUT\);\s*return LOST;", fetch)
    assert re.search(r"constexpr int NO_MORE = -1, LOST = -2;", src)
    takers = re.findall(r"const int it = next_item\(\);\s*if \(it < 0\) \{\s*ok = it != LOST;\s*break;", src)
    assert len(takers) == 2  # the producers, the MMA warp


@pytest.mark.parametrize("name,whole", [("k_ffn_tc.cu", r"&acc_full\["), ("k_gemm_bf16.cu", r"&acc_full\["),
                                        ("k_small.cu", r"&bar\["), ("k_route.cu", r"&bar\[buf\]")])
def test_layer_kernels_wait_by_warps_where_warps_go_on(name, whole):
    """The layer's kernels: producers and MMA issuers are single threads, but the epilogues' tcgen05 loads and the
    small-batch and selection kernels' warp-wide products, sums and votes follow waits of whole warps."""
    alone = [w for w in waits(name) if re.search(r"mbar_wait\(" + whole, w[1])]
    assert not alone, alone
