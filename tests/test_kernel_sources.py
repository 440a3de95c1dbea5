"""What the kernels' sources may not hold.  The library also serves replicas on
several GPUs and takes any device address from its callers, so no copy may be
a cluster multicast: its source would have to lie in the same GPU's memory.
Cluster barriers follow branches of single threads, so they are not the forms
that need the whole warp to arrive as one."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(f for e in ("*.cu", "*.cuh", "*.h") for f in
                 glob.glob(os.path.join(ROOT, "quantized_mixture_experts_router_gb300", "**", e), recursive=True))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_multicast(path):
    with open(path) as f:
        assert "multicast::cluster" not in f.read()


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_aligned_cluster_barrier(path):
    with open(path) as f:
        assert not re.search(r"barrier\.cluster\.(arrive|wait)[.\w]*\.aligned", f.read())
