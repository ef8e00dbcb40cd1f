"""The native marshalling of the layer operators' calls against the interpreter's own path: equal
bits from both, the same refusals, and the current stream and device respected."""
import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def calls():
    g = torch.Generator(device=DEV).manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, gate, z, dy = (n(2, 48, 70).bfloat16() for _ in range(4))
    bias, h0, dl = n(48), n(2, 48), n(2, 48)
    rows, res, w = n(9, 256).bfloat16(), n(9, 256), 1 + 0.1 * n(256)
    q, s = ops.fp8_quantize(rows)
    wq, ws = ops.fp8_quantize_weight(n(130, 256))
    ck = torch.empty(ops.gated_scan_checkpoints_size(2, 48, 70), dtype=torch.uint8, device=DEV)
    return dict(
        update=lambda: (lambda st: [ops.gated_state_update(st, x[..., 0].contiguous(), gate[..., 0].contiguous(),
                                                           bias, z[..., 0].contiguous()), st])(h0.clone()),
        scan=lambda: ops.gated_scan_fwd(x, gate, bias, z, h0, return_last_state=True, checkpoints=ck),
        scan_plain=lambda: [ops.gated_scan_fwd(x, gate, given_decay=True)],
        scan_bwd=lambda: ops.gated_scan_bwd(x, gate, dy, bias, z, h0, dl),
        scan_bwd_decay=lambda: ops.gated_scan_bwd(x, gate.abs().clamp(max=1), dy, bias, given_decay=True),
        norm=lambda: ops.add_rms_norm_fwd(rows, w, res), norm_alone=lambda: ops.add_rms_norm_fwd(rows, w),
        norm3=lambda: ops.add_rms_norm_fp8(rows.view(3, 3, 256), w, res.view(3, 3, 256)),
        norm_fp8=lambda: ops.add_rms_norm_fp8(rows, w),
        norm_bwd=lambda: ops.add_rms_norm_bwd(rows, res, w, res),
        norm_bwd_same=lambda: ops.add_rms_norm_bwd(rows, rows, w),
        quantize=lambda: ops.fp8_quantize(rows), quantize_cm=lambda: ops.fp8_quantize(x, channel_major=True),
        linear=lambda: [ops.fp8_linear(q, s, wq, ws)],
        linear_cm=lambda: [ops.fp8_linear(q, s, wq, ws, out_dtype=torch.float32, channel_major_seqlen=3)])


def flat(r):
    items = r.items() if isinstance(r, dict) else enumerate(r)
    return {k: v for k, v in items}


@pytest.mark.parametrize("name", ["update", "scan", "scan_plain", "scan_bwd", "scan_bwd_decay", "norm", "norm_alone",
                                  "norm3", "norm_fp8", "norm_bwd", "norm_bwd_same", "quantize", "quantize_cm",
                                  "linear", "linear_cm"])
def test_native_equals_interpreter(cuda_ok, name, monkeypatch):
    ops.load_library()
    assert ops._native is not None
    call = calls()[name]
    fast = flat(call())
    monkeypatch.setattr(ops, "_native", None)
    slow = flat(call())
    assert fast.keys() == slow.keys()
    for k in slow:
        if slow[k] is None:
            assert fast[k] is None
            continue
        assert fast[k].shape == slow[k].shape and fast[k].dtype == slow[k].dtype
        assert torch.equal(fast[k].view(torch.uint8) if fast[k].element_size() == 1 else fast[k],
                           slow[k].view(torch.uint8) if slow[k].element_size() == 1 else slow[k]), (name, k)


def test_native_is_the_path_taken(cuda_ok, monkeypatch):
    """Plain calls do not reach the interpreter's path."""
    todo = calls()

    def fail(*a):
        raise AssertionError("the interpreter's path was taken")

    monkeypatch.setattr(ops, "_run", fail)
    for name, call in todo.items():
        call()


def test_refusals_are_the_interpreters(cuda_ok):
    x = torch.randn(2, 8, 16, device=DEV)
    w = torch.ones(16, device=DEV)
    for call, error in (
            (lambda: ops.gated_scan_fwd(x, x[..., :8].contiguous()), ValueError),
            (lambda: ops.gated_scan_fwd(x, x.bfloat16()), ValueError),
            (lambda: ops.gated_scan_fwd(x.half(), x.half()), ValueError),
            (lambda: ops.gated_scan_fwd(x.transpose(1, 2), x.transpose(1, 2)), ValueError),
            (lambda: ops.gated_scan_fwd(x, x, gate_bias=torch.zeros(8)), ValueError),
            (lambda: ops.gated_scan_fwd(x, None), TypeError),
            (lambda: ops.gated_scan_bwd(x, x, x[:1]), ValueError),
            (lambda: ops.gated_state_update(x[..., 0].contiguous().bfloat16(), x[..., 0].contiguous(),
                                            x[..., 0].contiguous()), ValueError),
            (lambda: ops.add_rms_norm_fwd(x, w[:8]), ValueError),
            (lambda: ops.add_rms_norm_fp8(x[..., :8].contiguous(), w[:8].contiguous()), ops.MambaError),
            (lambda: ops.add_rms_norm_fwd(torch.randn(2, 16385, device=DEV), torch.ones(16385, device=DEV)),
             ops.MambaError),
            (lambda: ops.fp8_quantize(torch.randn(2, 24, device=DEV)), ops.MambaError),
            (lambda: ops.fp8_quantize(x), ValueError),
            (lambda: ops.fp8_linear(x[0], w, x[0], w), ValueError)):
        with pytest.raises(error):
            call()
    base = torch.randn(2 * 64 + 1, device=DEV)
    with pytest.raises(ops.MambaError):  # a view that is not 16-byte aligned
        ops.add_rms_norm_fwd(base[1:].view(2, 64), torch.ones(64, device=DEV))


def test_calls_run_on_the_current_stream(cuda_ok):
    """A call made on a side stream waits for that stream's work and for nothing else."""
    rows, w = torch.zeros(4096, 1024, device=DEV), torch.ones(1024, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(50):
            rows.add_(1.0)  # the call must see all of these
        q, s = ops.fp8_quantize(rows)
        out, _ = ops.add_rms_norm_fwd(rows, w)
    side.synchronize()
    assert float(q.float().min()) == 448.0 and float((s * 448 - 50).abs().max()) < 1e-3
    assert float((out - 1).abs().max()) < 1e-3
