"""The layer operators where element offsets pass 32 bits (needs a B200: up to 25 GB on the
device), and with every output passed in by the caller.

A piece at the far end of a large call is compared with the same piece called by itself: equal
bits, since a row, a token or an output is computed alike wherever it lies (the pieces keep the
rows' alignment and take the same kernels)."""
import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def free():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_gated_scan_beyond_32_bits(cuda_ok):
    b, d, L = 1, 2400, 1 << 20  # 2.5e9 elements; a warp per row, as in the piece below
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(b, d, L, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    a = torch.empty_like(x).uniform_(0.5, 1.0, generator=g)
    ck = torch.empty(ops.gated_scan_checkpoints_size(b, d, L), dtype=torch.uint8, device=DEV)
    y, last = ops.gated_scan_fwd(x, a, given_decay=True, return_last_state=True, checkpoints=ck)
    part = slice(d - 4, d)
    want, last_part = ops.gated_scan_fwd(x[:, part].contiguous(), a[:, part].contiguous(), given_decay=True,
                                         return_last_state=True)
    # four rows are walked by teams: the same states, associated differently
    assert float((y[:, part].float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    torch.testing.assert_close(last[:, part], last_part, rtol=1e-4, atol=1e-4)
    grads = ops.gated_scan_bwd(x, a, y, given_decay=True, checkpoints=ck)
    w = ops.gated_scan_bwd(x[:, part].contiguous(), a[:, part].contiguous(), y[:, part].contiguous(), given_decay=True)
    for k in ("dx", "dgate"):
        assert float((grads[k][:, part].float() - w[k].float()).abs().max()) <= 2.0 ** -6 * float(w[k].float().abs().max())
    del x, a, y, ck, grads, want
    free()


def test_norm_and_quantize_beyond_32_bits(cuda_ok):
    rows, dim = 1_100_000, 2048  # 2.25e9 elements
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = torch.rand(dim, device=DEV) + 0.5
    tail = x[-300:].contiguous()
    out, v = ops.add_rms_norm_fwd(x, w, x)
    o, u = ops.add_rms_norm_fwd(tail, w, tail)
    assert torch.equal(out[-300:], o) and torch.equal(v[-300:], u)
    grad = ops.add_rms_norm_bwd(out, v, w)
    assert torch.equal(grad["dx"][-300:], ops.add_rms_norm_bwd(o, u, w)["dx"])
    del grad, v, out
    q, s = ops.fp8_quantize(x)
    qt, st = ops.fp8_quantize(tail)
    assert torch.equal(q[-300:].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s[-300:], st)
    del q, s
    cm = x.view(2, 1024, -1)  # (2, 1024, 1100000): channel-major rows of over a million tokens
    q, s = ops.fp8_quantize(cm, channel_major=True)
    qt, st = ops.fp8_quantize(cm[1:, :, -64:].contiguous(), channel_major=True)
    assert torch.equal(q[-64:].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s[-64:], st)
    del x, cm, q, s
    free()


@pytest.mark.parametrize("L", [None, 65536], ids=["tokens", "channels"])
def test_linear_beyond_32_bits(cuda_ok, L):
    tokens, n, k = 262144, 8448, 256  # 2.2e9 outputs
    g = torch.Generator(device=DEV).manual_seed(3)
    xq, xs = ops.fp8_quantize(torch.randn(tokens, k, generator=g, device=DEV).bfloat16())
    wq, ws = ops.fp8_quantize_weight(torch.randn(n, k, generator=g, device=DEV))
    out = ops.fp8_linear(xq, xs, wq, ws, channel_major_seqlen=L)
    part = ops.fp8_linear(xq[-2000:], xs[-2000:], wq, ws)
    got = out[-2000:] if L is None else out[-1, :, -2000:].t()
    assert torch.equal(got, part)
    del out
    free()


def test_outputs_of_the_caller(cuda_ok):
    g = torch.Generator(device=DEV).manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, gate, h0 = n(2, 32, 100), n(2, 32, 100), n(2, 32)
    y, last = torch.empty_like(x), torch.empty_like(h0)
    r = ops.gated_scan_fwd(x, gate, initial_state=h0, y=y, last_state=last, return_last_state=True)
    want = ops.gated_scan_fwd(x, gate, initial_state=h0, return_last_state=True)
    assert r[0] is y and r[1] is last and torch.equal(y, want[0]) and torch.equal(last, want[1])
    ws = torch.empty(ops.gated_scan_bwd_workspace_size(2, 32, 100), dtype=torch.uint8, device=DEV)
    a, b = ops.gated_scan_bwd(x, gate, y, workspace=ws), ops.gated_scan_bwd(x, gate, y)
    assert all(torch.equal(a[k], b[k]) for k in ("dx", "dgate", "dinitial_state"))
    with pytest.raises(ops.MambaError):
        ops.gated_scan_bwd(x, gate, y, workspace=ws[:16])
    st, yt = h0.clone(), torch.empty_like(h0)
    assert ops.gated_state_update(st, x[..., 0].contiguous(), gate[..., 0].contiguous(), y=yt) is yt
    rows, res, w = n(6, 128).bfloat16(), n(6, 128), torch.ones(128, device=DEV)
    out, v = torch.empty(6, 128, device=DEV), torch.empty_like(res)
    r = ops.add_rms_norm_fwd(rows, w, res, out_dtype=torch.float32, out=out, residual_out=v)
    assert r[0] is out and r[1] is v and torch.equal(v, rows.float() + res)
    kept = torch.empty_like(rows)  # a copy of the stream where there is no residual
    assert torch.equal(ops.add_rms_norm_fwd(rows, w, residual_out=kept)[1], rows) and torch.equal(kept, rows)
    q, s = torch.empty(6, 128, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(6, 1, device=DEV)
    assert ops.fp8_quantize(rows, q=q, scales=s)[0] is q
    wq, wsc = ops.fp8_quantize_weight(n(48, 128))
    o = torch.empty(6, 48, device=DEV)
    assert ops.fp8_linear(q, s, wq, wsc, out_dtype=torch.float32, out=o) is o
    assert torch.equal(o, ops.fp8_linear(q, s, wq, wsc, out_dtype=torch.float32))
