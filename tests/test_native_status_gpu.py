"""What the native marshalling does once the library has been called: its status is the caller's,
and the call is never made a second time."""
import ctypes

import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
ERR_CUDA = -6


def addresses(lib):
    return {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ops._native.names()}


@pytest.fixture
def bound(cuda_ok):
    """Binds the native module to a stub of one entry point, and back afterwards."""
    lib = ops.load_library()
    assert ops._native is not None
    kept = []

    def stub(name, status):
        fn = getattr(lib, name)
        calls = []
        kind = ctypes.CFUNCTYPE(fn.restype, *fn.argtypes)
        kept.append(kind(lambda *a: calls.append(a) or status))
        ops._native.bind(dict(addresses(lib), **{name: ctypes.cast(kept[-1], ctypes.c_void_p).value}))
        return calls

    yield stub
    ops._native.bind(addresses(lib))


def test_a_failed_update_is_raised_and_not_repeated(bound):
    state, x = torch.ones(2, 8, device=DEV), torch.ones(2, 8, device=DEV)
    calls = bound("mamba_gated_state_update", ERR_CUDA)
    with pytest.raises(ops.MambaError) as e:
        ops.gated_state_update(state, x, x)
    assert e.value.status == ERR_CUDA and len(calls) == 1
    # the interpreter's path was not taken either: the state is as it was
    assert torch.equal(state, torch.ones_like(state))


@pytest.mark.parametrize("name", ["gated_scan_fwd", "gated_scan_bwd", "add_rms_norm_fwd", "add_rms_norm_fp8",
                                  "add_rms_norm_bwd", "fp8_quantize", "fp8_linear"])
def test_every_failed_call_is_raised(bound, name):
    x3, x2, w = torch.ones(1, 16, 4, device=DEV), torch.ones(4, 16, device=DEV), torch.ones(16, device=DEV)
    q, s = ops.fp8_quantize(x2)
    wq, ws = ops.fp8_quantize_weight(x2)
    run = dict(gated_scan_fwd=lambda: ops.gated_scan_fwd(x3, x3), gated_scan_bwd=lambda: ops.gated_scan_bwd(x3, x3, x3),
               add_rms_norm_fwd=lambda: ops.add_rms_norm_fwd(x2, w), add_rms_norm_fp8=lambda: ops.add_rms_norm_fp8(x2, w),
               add_rms_norm_bwd=lambda: ops.add_rms_norm_bwd(x2, x2, w), fp8_quantize=lambda: ops.fp8_quantize(x2),
               fp8_linear=lambda: ops.fp8_linear(q, s, wq, ws))[name]
    calls = bound("mamba_" + name, ERR_CUDA)
    with pytest.raises(ops.MambaError) as e:
        run()
    assert e.value.status == ERR_CUDA and len(calls) == 1
