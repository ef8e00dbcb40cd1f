"""Each part's device error word (scans, projection, gated recurrence) is reported until it is cleared,
and cleared when it is reported.  The waits are bounded, about a millisecond; nothing faults."""
import ctypes
import itertools

import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
TIMEOUT, ERR_CUDA = -7, -6


def status(clear):
    try:
        ops.check_device_error(clear=clear)
    except ops.MambaError as e:
        return e.status
    return 0


@pytest.mark.parametrize("parts", [p for n in (1, 2, 3) for p in itertools.combinations(range(3), n)], ids=str)
def test_words_are_reported_and_cleared(cuda_ok, parts):
    assert status(True) == 0
    for part in parts:
        ops.diag_wait_timeout(1_000_000, part=part)
    assert status(False) == TIMEOUT
    assert status(True) == TIMEOUT
    assert status(True) == 0 and status(False) == 0


@pytest.mark.parametrize("part", [0, 1, 2])
def test_a_read_that_fails_loses_no_report(cuda_ok, part):
    """A stream under capture refuses the read; the word is still there for the next one."""
    lib, driver = ops.load_library(), ctypes.CDLL("libcuda.so.1")
    ops.diag_wait_timeout(1_000_000, part=part)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(handle, 2) == 0
    failed = lib.mamba_check_device_error(1, handle)
    driver.cuStreamEndCapture(handle, ctypes.byref(graph))
    if graph.value:
        driver.cuGraphDestroy(graph)
    assert failed == ERR_CUDA
    assert status(True) == TIMEOUT and status(True) == 0
