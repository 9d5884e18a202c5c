"""Shared memory of another CTA may be used from the time that CTA has begun until
it ends, which only a barrier of the cluster says. On the sources, since a missing
barrier may show in no run: every kernel of clusters has one before it begins its work,
ahead of any access of its own to another CTA, and one at its end."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "newton_schulz_gram_gb300", "csrc")


def kernels():
    """name: body, without comments."""
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in re.split(r"\b__global__\b", text)[1:]:
            name = re.search(r"(\w+)\s*\(\w", re.sub(r"__launch_bounds__\([^)]*\)", "", part)).group(1)
            found[name] = part[:part.index("\n}\n")]
    return found


CLUSTERS = {name: body for name, body in kernels().items() if "cluster_sync()" in body or "map_to_rank(" in body}


def test_the_kernels_of_clusters_are_found():
    assert {"moe_balance_join_kernel", "layer_norm_ring_kernel", "layer_norm_backward_ring_kernel", "gemm_tc_kernel"} <= set(CLUSTERS)


@pytest.mark.parametrize("name", sorted(CLUSTERS))
def test_barriers_at_both_ends(name):
    entry, *rest = CLUSTERS[name].split("cluster_sync()")
    assert len(rest) >= 2, "a barrier at either end"
    # gemm_tc_kernel's lambdas name the accesses that its loops make; no statement may.
    for access in ("shared::cluster", "row_sums<", "st_cluster_v4(", "send_sums("):
        assert access not in entry, access
