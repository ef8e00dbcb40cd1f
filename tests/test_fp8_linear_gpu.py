"""The 8-bit projection on the GPU against fp64 on the same e4m3 operands and scales, and the
layer's operators run together as a prefill and as decode steps.

Tolerance.  Products of two e4m3 values are exact in fp32 (8 bits of fraction).  A block's 128
products are summed in fp32; with at worst one truncation (2^-23 relative to the running
magnitude) an addition, a block sum is off by 128 * 2^-23 = 2^-16 of the sum of magnitudes S.
The scaled block sums are added in fp32: two roundings of the scale and one an addition,
(kb + 8) 2^-24 of S.  Plus half a step of the output's type."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def operands(tokens, n, k, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(tokens, k, generator=g, device=DEV) * torch.exp(torch.randn(tokens, 1, generator=g, device=DEV))
    w = torch.randn(n, k, generator=g, device=DEV) / k ** 0.5
    w[: n // 2] *= 3.0  # blocks of unlike scales
    return (*ops.fp8_quantize(x), *ops.fp8_quantize_weight(w))


def exact(xq, xs, wq, ws):
    k, n = xq.shape[1], wq.shape[0]
    at = torch.arange(k, device=DEV) // 128
    x = xq.float().double() * xs.double()[:, at]
    w = wq.float().double() * ws.double()[torch.arange(n, device=DEV) // 128][:, at]
    return x @ w.t(), x.abs() @ w.abs().t()


def compare(tokens, n, k, out="fp32", L=None, seed=0):
    o = operands(tokens, n, k, seed)
    got = ops.fp8_linear(*o, out_dtype=TYPES[out], channel_major_seqlen=L)
    want, mag = exact(*o)
    kb = -(-k // 128)
    tol = (2.0 ** -16 + (kb + 8) * 2.0 ** -24) * mag + want.abs() * (2.0 ** -8 if out == "bf16" else 2.0 ** -24)
    if L is not None:
        want, tol = (t.view(tokens // L, L, n).transpose(1, 2) for t in (want, tol))
    ref.check(got.double().cpu().numpy(), want.cpu().numpy(), tol.cpu().numpy(), "out")
    return o, got


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 33, 64, 65, 128, 200])
@pytest.mark.parametrize("nk", [(1, 16), (8, 128), (128, 256), (130, 272), (848, 1536), (1000, 2064)],
                         ids=lambda v: "%dx%d" % v)
def test_fp8_linear_few_tokens(cuda_ok, tokens, nk):
    compare(tokens, *nk, seed=tokens)


@pytest.mark.parametrize("shape", [(128, 256 * 148, 128), (2500, 2000, 400), (128 * 148, 200, 1040),
                                   (4100, 1288, 2560), (3333, 1531, 272)], ids=lambda s: "%dx%dx%d" % s)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_fp8_linear_many_tokens(cuda_ok, shape, out):
    compare(*shape, out=out, seed=1)


@pytest.mark.parametrize("shape", [(61, 5120, 2560), (77, 4000, 2576), (59, 10240, 2560), (150, 4999, 2064),
                                   (231, 2555, 4112), (1001, 130, 1536)], ids=lambda s: "%dx%dx%d" % s)
def test_fp8_linear_between(cuda_ok, shape):
    """Tiles of 16, 32 and 64 tokens, with one piece of the inputs and with several."""
    tokens, n, k = shape
    o, got = compare(*shape, out="bf16", seed=3)
    if tokens % 7 == 0:
        cm = ops.fp8_linear(*o, channel_major_seqlen=tokens // 7)
        assert torch.equal(cm, got.view(7, tokens // 7, n).transpose(1, 2))


@pytest.mark.parametrize("shape", [(3, 1, 300, 256), (2, 7, 130, 272), (3, 431, 848, 1536), (2, 2050, 1400, 384)],
                         ids=lambda s: "%dx%dx%dx%d" % s)
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_fp8_linear_channel_major(cuda_ok, shape, out):
    b, L, n, k = shape
    o, got = compare(b * L, n, k, out=out, L=L, seed=2)
    rows = ops.fp8_linear(*o, out_dtype=TYPES[out])
    assert torch.equal(got, rows.view(b, L, n).transpose(1, 2))


def test_fp8_linear_no_tokens(cuda_ok):
    o = operands(4, 32, 64, 1)
    assert ops.fp8_linear(o[0][:0], o[1][:0], o[2], o[3]).shape == (0, 32)


def test_fp8_linear_nan_stays_in_its_token(cuda_ok):
    xq, xs, wq, ws = operands(40, 300, 256, 3)
    clean = ops.fp8_linear(xq, xs, wq, ws)
    bad = xq.clone()
    bad.view(torch.uint8)[7, 9] = 0x7F
    got = ops.fp8_linear(bad, xs, wq, ws)
    keep = [i for i in range(40) if i != 7]
    assert torch.isnan(got[7]).all() and torch.equal(got[keep], clean[keep])


def test_fp8_linear_many_inputs(cuda_ok):
    compare(5, 40, 33008, seed=4)
    compare(70, 40, 110000, seed=5)


def test_fp8_linear_graph_and_two_streams(cuda_ok):
    sets = [operands(20, 700, 512, 1), operands(3000, 2100, 512, 2)]
    eager = [ops.fp8_linear(*o) for o in sets]
    graphs, outs = [], []
    for o in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.fp8_linear(*o))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert torch.equal(e, o)
    del graphs


def test_layer_prefill_then_decode(cuda_ok):
    """The operators as a layer uses them: norm to e4m3 -> projections into the channel-major
    layout -> causal conv1d -> gated recurrence -> e4m3 -> output projection; a prefill of L
    tokens in one pass equals a prefill of the first tokens followed by decode steps."""
    b, L, dm, di, cut = 2, 37, 256, 384, 33
    g = torch.Generator(device=DEV).manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, residual = n(b, L, dm).bfloat16(), n(b, L, dm)
    norm_w = 1 + 0.1 * n(dm)
    proj = [ops.fp8_quantize_weight(n(di, dm) / dm ** 0.5) for _ in range(3)]
    w_out = ops.fp8_quantize_weight(n(dm, di) / di ** 0.5)
    conv_w, conv_b, gate_b = 0.5 * n(di, 4), 0.1 * n(di), n(di) - 2

    def inputs(xp, rp, steps):
        q, s, stream = ops.add_rms_norm_fp8(xp, norm_w, rp)
        q, s = q.view(-1, dm), s.view(-1, s.shape[-1])
        return [ops.fp8_linear(q, s, *w, channel_major_seqlen=steps) for w in proj], stream

    def prefill(xp, rp):
        steps = xp.shape[1]
        (u, gate, z), stream = inputs(xp, rp, steps)
        u, conv_state = ops.causal_conv1d_fwd(u, conv_w, conv_b, return_final_state=True)
        y, state = ops.gated_scan_fwd(u, gate, gate_b, z, return_last_state=True)
        q, s = ops.fp8_quantize(y, channel_major=True)
        return ops.fp8_linear(q, s, *w_out).view(b, steps, dm), stream, conv_state, state

    whole, stream, conv_end, state_end = prefill(x, residual)
    out, _, conv_state, state = prefill(x[:, :cut].contiguous(), residual[:, :cut].contiguous())
    assert torch.equal(out, whole[:, :cut])
    for t in range(cut, L):
        (u, gate, z), st = inputs(x[:, t].contiguous(), residual[:, t].contiguous(), 1)
        assert torch.equal(st, stream[:, t])
        u = ops.causal_conv1d_update(conv_state, u.view(b, di), conv_w, conv_b)
        y = ops.gated_state_update(state, u, gate.view(b, di), gate_b, z.view(b, di))
        q, s = ops.fp8_quantize(y)
        step = ops.fp8_linear(q, s, *w_out)
        # y may round to the other neighbour in bf16 (the recurrence is associated differently),
        # and then one e4m3 step: 2^-3 of a value in a few of 384 summed terms
        a, r = step.double(), whole[:, t].double()
        assert float((a - r).abs().max()) <= 2.0 ** -4 * float(r.abs().max())
    assert torch.equal(conv_state, conv_end)
    ref.check(state.double().cpu().numpy(), state_end.double().cpu().numpy(),
              2.0 ** -16 * (1 + state_end.abs().double().cpu().numpy()), "state")
    # the same layer in fp64 from the definitions, on the quantised weights
    de = lambda w: (w[0].float().double() * w[1].double().repeat_interleave(128, 0)[:w[0].shape[0]]  # noqa: E731
                    .repeat_interleave(128, 1)[:, :w[0].shape[1]]).cpu().numpy()
    v = stream.double().cpu().numpy().reshape(b * L, dm)
    a, _ = ref.rms_norm(v, norm_w.double().cpu().numpy(), 1e-5)
    q, s = ref.e4m3_groups(a)
    a = q * s[:, np.arange(dm) // 128]
    u, gate, z = ((a @ de(w).T).reshape(b, L, di).transpose(0, 2, 1) for w in proj)
    cw, cb = conv_w.double().cpu().numpy(), conv_b.double().cpu().numpy()
    up = np.concatenate([np.zeros((b, di, 3)), u], 2)
    c = sum(up[..., k:k + L] * cw[:, k][:, None] for k in range(4)) + cb[:, None]
    f = ref.gated_forward(c * ref.sigmoid(c), gate, gate_b.double().cpu().numpy(), z)
    q, s = ref.e4m3_groups(f["y"].transpose(0, 2, 1).reshape(b * L, di))
    want = ((q * s[:, np.arange(di) // 128]) @ de(w_out).T).reshape(b, L, dm)
    err = np.linalg.norm(whole.double().cpu().numpy() - want) / np.linalg.norm(want)
    # bf16 between the operators (2^-8 each of four, some amplified by the gates) may move an
    # e4m3 rounding of y by a step (2^-3 relative) in under a tenth of the terms: 0.03 in norm
    assert err <= 0.04, err
