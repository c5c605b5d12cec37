"""Blocks of a cluster touch one another's shared memory only behind a barrier of the cluster: a block that has not started yet
has none, and whether it has shows in no result.  So the order is read off the kernels' source (no GPU needed)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_gb300", "csrc")
BARRIERS = r"wait_for_cluster\(\)|cluster\.sync\(\)|this_cluster\(\)\.sync\(\)"


def kernels():
    """(name, body) of every kernel that names another block's shared memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        for body in open(path).read().split("__global__")[1:]:
            body = re.sub(r"//[^\n]*", "", body)
            if re.search(r"map_shared_rank|mapa\b", body):
                yield re.search(r"(\w+)\((?:const )?\w+Params", body).group(1), body


@pytest.mark.parametrize("name, body", list(kernels()), ids=lambda v: v if v.isidentifier() else "")
def test_remote_shared_memory_follows_a_barrier(name, body):
    first = re.search(r"map_shared_rank|mapa\b", body).start()
    barrier = re.search(BARRIERS, body)
    assert barrier and barrier.start() < first, f"{name} names another block's shared memory before a barrier of its cluster"
    # an arrival for the split barrier, on entry
    if barrier.group().startswith("wait"):
        assert 0 <= body.find("cluster_started()") < barrier.start()
    # and the block whose memory it is does not end before the others' last access
    assert len(re.findall(BARRIERS, body)) >= 2


def test_there_is_such_a_kernel():
    assert "select_kernel" in [name for name, _ in kernels()]
