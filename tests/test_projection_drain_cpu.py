"""The projection's kernels end only after the copies into their shared memory and the products in
tensor memory have: the waits for them stand on the way that every role takes to its end, not only
where that role itself gave up (another one may have, long after the last copy was issued).  Checked on
the source: making a device-side wait run out while copies are in flight is nothing to do on a GPU."""
import os
import re

from selective_state_space_56_b200 import build as s6build

LINES = open(os.path.join(s6build.CSRC, "fp8_linear.cu")).read().split("\n")


def around(i):
    """The lines that open the blocks (by indentation) around line i, innermost first."""
    depth = len(LINES[i]) - len(LINES[i].lstrip())
    for j in range(i - 1, -1, -1):
        line = LINES[j]
        here = len(line) - len(line.lstrip())
        if line.strip() and here < depth and not line.lstrip().startswith("//"):
            depth = here
            yield line
        if line.startswith("__global__"):
            return


def test_last_copies_and_products_are_waited_for_by_every_way_to_the_end():
    waits = [i for i, line in enumerate(LINES) if re.search(r"mbar_wait_bounded\(&bars\.(full|drain)", line)]
    kinds = [re.search(r"&bars\.(\w+)", LINES[i]).group(1) for i in waits]
    assert sorted(kinds) == ["drain", "drain", "full", "full"]  # either kernel, copies and products
    for i in waits:
        for line in around(i):
            assert "!ok" not in line and "wait_or_abort" not in line, (LINES[i].strip(), line.strip())


def test_the_products_are_committed_whatever_ended_their_loop():
    commits = [i for i, line in enumerate(LINES) if re.search(r"tc_commit(_pair)?\(&bars\.drain\)", line)]
    assert len(commits) == 2
    for i in commits:
        for line in around(i):
            assert "!ok" not in line and "wait_or_abort" not in line and "for (" not in line, line.strip()
