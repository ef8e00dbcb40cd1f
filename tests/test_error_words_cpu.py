"""Host checks of the probe of the device error words (nothing is launched)."""
import os

import pytest

from selective_state_space_56_b200 import build as s6build
from selective_state_space_56_b200 import ops

DIMS = -2


@pytest.mark.parametrize("part,limit", [(-1, 1000), (3, 1000), (0, 0), (1, 0), (2, -5), (1, 5_000_000_000)])
def test_probe_refusals(part, limit):
    s6build.build()
    assert ops.load_library().mamba_diag_wait_timeout_in(part, limit, None) == DIMS


def test_a_check_copies_to_the_host_once():
    """Each copy makes the host wait for the stream; the words of all parts come with one."""
    text = "".join(open(os.path.join(s6build.CSRC, f)).read() for f in sorted(os.listdir(s6build.CSRC))
                   if f.endswith((".cu", ".cuh")))
    assert text.count("cudaMemcpyFromSymbol") == 1 and text.count("cudaMemcpyDeviceToHost") == 1
