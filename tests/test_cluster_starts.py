"""Access to another CTA's shared memory is defined from the moment that CTA is known to run: every kernel that maps
an address into another CTA of its cluster has all its threads pass a cluster barrier first.  Read from the sources: no
GPU is made to run into the fault."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routing_mxfp4_gb300", "csrc")
# what makes or takes such an address (ClusterSum's exchange among them), on its own or through a pair's barrier
REMOTE = r"\b(?:cluster_map|tc_commit_pair|mma_bf16_pair|tma_load_2d_pair|exchange)\("


def kernels(path):
    """(name, body) of every kernel of a source file, comments taken out."""
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    src = re.sub(r"//[^\n]*", "", src)
    for m in re.finditer(r"__global__[^;{]*?\b(k_\w+)\(", src):
        start = src.index("{", m.end())
        depth, end = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
        yield m.group(1), src[start:end]


FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu")))


def test_the_kernels_that_reach_into_other_ctas_are_seen():
    found = {n for f in FILES for n, body in kernels(os.path.join(CSRC, f)) if re.search(REMOTE, body)}
    assert {"k_balance_count", "k_balance_rows", "k_balance_final", "k_linear_act", "k_linear_few", "k_linear_mx",
            "k_grouped"} <= found


@pytest.mark.parametrize("name", FILES)
def test_a_cluster_barrier_stands_before_the_first_access(name):
    for kernel, body in kernels(os.path.join(CSRC, name)):
        first = [m.start() for m in re.finditer(REMOTE, body)
                 # a lambda that only forms the address is used behind the barrier it is checked with below
                 if not re.search(r"auto \w+ = \[&\]\([^)]*\) \{ return (?:tc::)?$", body[:m.start()])]
        named = re.search(r"auto (\w+) = \[&\]\([^)]*\) \{ return (?:tc::)?cluster_map\(", body)
        if named:
            first += [m.start() for m in re.finditer(r"\b%s\((?!float)" % named.group(1), body)]
        if not first:
            continue
        barrier = re.search(r"\b(?:tc::)?cluster_sync\(\)", body)
        assert barrier and barrier.start() < min(first), f"{kernel} reaches into another CTA before a cluster barrier"
