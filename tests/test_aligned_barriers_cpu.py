"""Cluster barriers in their aligned form take whole warps: some lanes may come from a branch of their
own, so a __syncwarp stands directly before each.  Checked on the sources; a warp that arrives in parts
is undefined, which is nothing to try on a GPU."""
import os
import re

import pytest

from selective_state_space_56_b200 import build as s6build

SOURCES = sorted(f for f in os.listdir(s6build.CSRC) if f.endswith((".cu", ".cuh")))


@pytest.mark.parametrize("name", SOURCES)
def test_whole_warps_reach_cluster_barriers(name):
    lines = [s.strip() for s in open(os.path.join(s6build.CSRC, name))]
    lines = [s for s in lines if s and not s.startswith("//")]
    for i, line in enumerate(lines):
        if re.search(r"barrier\.cluster\.arrive\S*\.aligned", line):
            assert lines[i - 1] == "__syncwarp();", (name, line)


def test_there_are_cluster_barriers():
    text = "".join(open(os.path.join(s6build.CSRC, f)).read() for f in SOURCES)
    assert text.count("barrier.cluster.arrive") >= 3
