"""Kernels that start before the kernel whose results they read has ended (programmatic dependent
launch): the read-only path (__ldg, ld.global.nc) is defined for data that nothing writes while the
kernel runs, and those results are written while it runs.  The rule is checked on the sources."""
import os
import re

import pytest

from selective_state_space_56_b200 import build as s6build

SOURCES = sorted(f for f in os.listdir(s6build.CSRC) if f.endswith((".cu", ".cuh")))


def early_kernels(text):
    """Bodies of the functions that wait for the kernel before them."""
    for wait in re.finditer(r"cudaGridDependencySynchronize\(\)|griddepcontrol\.wait", text):
        start = text.rindex("\n__global__", 0, wait.start())
        end = text.index("\n}\n", wait.start())
        yield text[start:end]


def test_there_are_early_kernels():
    assert sum(len(list(early_kernels(open(os.path.join(s6build.CSRC, f)).read()))) for f in SOURCES) >= 2


@pytest.mark.parametrize("name", SOURCES)
def test_early_kernels_read_results_coherently(name):
    for body in early_kernels(open(os.path.join(s6build.CSRC, name)).read()):
        signature, code = body.split("{", 1)
        assert "__ldg(" not in code and "ld.global.nc" not in code, body[:120]
        assert "__restrict__" not in signature, body[:120]
