"""An error that one call reports is not reported again by the next: a launch's status is its own.

The error is made on the host: reading the device error word synchronises its stream, which a
stream under capture refuses.  Nothing faults on the device."""
import ctypes

import pytest
import torch

from selective_state_space_56_b200 import inputs, ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
ERR_CUDA = -6


def leave_an_error():
    """A library call that fails on the host; the stream and its capture are given up again."""
    lib, driver = ops.load_library(), ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert driver.cuStreamBeginCapture_v2(handle, 2) == 0  # relaxed: other streams go on
    status = lib.mamba_check_device_error(0, handle)
    driver.cuStreamEndCapture(handle, ctypes.byref(graph))
    if graph.value:
        driver.cuGraphDestroy(graph)
    assert status == ERR_CUDA
    torch.cuda.synchronize()


@pytest.mark.parametrize("native", [True, False])
def test_update_after_an_error_moves_the_state_one_step(cuda_ok, native, monkeypatch):
    ops.load_library()
    if not native:
        monkeypatch.setattr(ops, "_native", None)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, gate, state = (torch.randn(3, 64, generator=g, device=DEV) for _ in range(3))
    want_state = state.clone()
    want = ops.gated_state_update(want_state, x, gate)
    leave_an_error()
    y = ops.gated_state_update(state, x, gate)
    assert torch.equal(state, want_state) and torch.equal(y, want)


def test_other_calls_after_an_error(cuda_ok):
    x3, x2, w = torch.randn(1, 16, 4, device=DEV), torch.randn(4, 16, device=DEV), torch.ones(16, device=DEV)
    p = inputs.scan_inputs(1, 16, 16, 64, torch.float32, seed=3, device=DEV)
    q, s = ops.fp8_quantize(x2)
    wq, ws = ops.fp8_quantize_weight(x2)
    for call in (lambda: ops.gated_scan_fwd(x3, x3), lambda: ops.gated_scan_bwd(x3, x3, x3),
                 lambda: ops.add_rms_norm_fwd(x2, w), lambda: ops.add_rms_norm_bwd(x2, x2, w),
                 lambda: ops.fp8_quantize(x2), lambda: ops.fp8_quantize_weight(x2),
                 lambda: ops.fp8_linear(q, s, wq, ws), lambda: ops.causal_conv1d_fwd(x3, torch.ones(16, 4, device=DEV)),
                 lambda: ops.selective_scan_fwd(p["u"], p["delta"], p["A"], p["B"], p["C"])):
        leave_an_error()
        call()
    torch.cuda.synchronize()
