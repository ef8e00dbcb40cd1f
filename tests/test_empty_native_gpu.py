"""Sizes of zero through the native marshalling: the same outputs as the interpreter's path."""
import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_backward_of_an_empty_sequence_has_every_gradient(cuda_ok, monkeypatch):
    x, h0, bias = torch.empty(2, 3, 0, device=DEV), torch.randn(2, 3, device=DEV), torch.zeros(3, device=DEV)
    ops.load_library()
    assert ops._native is not None
    results = []
    for native in (ops._native, None):
        monkeypatch.setattr(ops, "_native", native)
        results.append(ops.gated_scan_bwd(x, x, x, bias, x, h0, h0))
    for fast, slow in zip(results[0].values(), results[1].values()):
        assert fast is not None and fast.shape == slow.shape and torch.equal(fast, slow)


def test_other_calls_without_elements(cuda_ok, monkeypatch):
    x, rows, w = torch.empty(2, 3, 0, device=DEV), torch.empty(0, 32, device=DEV), torch.ones(32, device=DEV)
    wq, ws = ops.fp8_quantize_weight(torch.ones(8, 32, device=DEV))
    calls = [lambda: ops.gated_scan_fwd(x, x, torch.zeros(3, device=DEV), x, return_last_state=True),
             lambda: ops.add_rms_norm_fwd(rows, w, rows), lambda: ops.add_rms_norm_fp8(rows, w, rows.bfloat16()),
             lambda: ops.add_rms_norm_bwd(rows, rows.bfloat16(), w, rows.bfloat16()).values(),
             lambda: ops.fp8_quantize(rows), lambda: ops.fp8_quantize(torch.empty(2, 32, 0, device=DEV), True),
             lambda: [ops.fp8_linear(*ops.fp8_quantize(rows), wq, ws)],
             lambda: [ops.fp8_linear(*ops.fp8_quantize(rows), wq, ws, channel_major_seqlen=5)]]
    native = ops._native
    for call in calls:
        monkeypatch.setattr(ops, "_native", native)
        fast = call()
        monkeypatch.setattr(ops, "_native", None)
        for a, b in zip(fast, call()):
            assert a.shape == b.shape and a.dtype == b.dtype
