"""Residual addition with RMS norm (forward, e4m3 output, backward) and the e4m3 quantisation
on the GPU against fp64.

Tolerances (u = 2^-24).  The stream v is one fp32 addition rounded to its type: equal bits to
torch's.  The sum of dim squares passes at most 40 fp32 additions a term in a thread, 5 in a
warp and 16 over the CTA, so mean v^2 is off by at most 64 u relative, rstd by 32 u + 2^-22
(rsqrt) and an output by two more roundings: 2^-18 relative in all, plus half a step of its type.
The backward's second sum is off by 64 u of its terms' magnitudes.  A column sum over rows adds
at most rows / blocks + blocks / 32 + 32 terms in sequence; with the term's own error of 2^-18
relative, (2^-18 + (rows + 64) u) times the sum of magnitudes bounds it.
e4m3: a value lies within half a step (2^-4 relative, 2^-10 absolute below 2^-6) of the exact
quotient, whose numerator and scale are each off by 2^-18 relative."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
REL = 2.0 ** -18


def n64(t):
    return None if t is None else t.detach().float().double().cpu().numpy()


def problem(rows, dim, xt, rt, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(x=n(rows, dim).to(TYPES[xt]), weight=1 + 0.2 * n(dim), dout=n(rows, dim).to(TYPES[xt]),
             residual=None if rt is None else (2 * n(rows, dim)).to(TYPES[rt]),
             dres=None if rt is None else n(rows, dim).to(TYPES[rt]))
    return {k: None if v is None else v.to(DEV) for k, v in p.items()}


def check_e4m3(q, scales, v, what):
    """q (rows, dim), scales against exact rows v within the bounds above."""
    want, ws = ref.e4m3_groups(v)
    ref.check(n64(scales), ws, 2 * REL * ws, what + " scales")
    cols = np.arange(v.shape[1]) // 128
    s = n64(scales)[:, cols]
    got = n64(q)
    half = np.maximum(np.abs(got) * 2.0 ** -4, 2.0 ** -10)
    ref.check(got * s, v, half * s + 4 * REL * np.abs(v) + 1e-36, what)
    assert np.abs(got).max() <= 448


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 48), (4, 130), (7, 768), (3, 1001), (2, 2560), (3, 5120),
          (2, 8200), (2, 16383), (1, 16384)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"),
                                   ("fp32", "bf16"), ("bf16", None)], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%dx%d" % s)
def test_add_rms_norm(cuda_ok, shape, types):
    rows, dim = shape
    xt, rt = types
    p = problem(rows, dim, xt, rt, seed=dim)
    st = rt or xt
    for ot in ("bf16", "fp32"):
        out, v = ops.add_rms_norm_fwd(p["x"], p["weight"], p["residual"], out_dtype=TYPES[ot])
        total = p["x"] if rt is None else (p["x"].float() + p["residual"].float()).to(TYPES[rt])
        assert torch.equal(v, total)
        want, _ = ref.rms_norm(n64(total), n64(p["weight"]), 1e-5)
        ref.check(n64(out), want, REL * np.abs(want) + ref.half_step(ot, want), "out")
    if dim % 16 == 0:
        q, s, v = ops.add_rms_norm_fp8(p["x"], p["weight"], p["residual"])
        assert torch.equal(v, total)
        check_e4m3(q, s, want, "out e4m3")
    g = ops.add_rms_norm_bwd(p["dout"], total, p["weight"], p["dres"])
    d, v64, w = n64(p["dout"]), n64(total), n64(p["weight"])
    dv, dw = ref.rms_norm_backward(d, v64, w, n64(p["dres"]), 1e-5)
    _, rstd = ref.rms_norm(v64, w, 1e-5)
    xhat = v64 * rstd
    mag = rstd * (np.abs(d * w) + np.abs(xhat) * np.mean(np.abs(d * w * xhat), -1, keepdims=True))
    tol = 2 * REL * mag + 2 * ref.U * np.abs(dv)
    ref.check(n64(g["dx"]), dv, tol + ref.half_step(xt, dv), "dx")
    ref.check(n64(g["dresidual"]), dv, tol + ref.half_step(st, dv), "dresidual")
    ref.check(n64(g["dweight"]), dw, (REL + (rows + 64) * ref.U) * np.abs(d * xhat).sum(0), "dweight")


@pytest.mark.parametrize("shape", [(5000, 768), (3001, 101), (2500, 2560)], ids=lambda s: "%dx%d" % s)
def test_add_rms_norm_backward_many_rows(cuda_ok, shape):
    """More rows than CTAs: each CTA sums dweight over several; equal calls give equal bits."""
    rows, dim = shape
    p = problem(rows, dim, "bf16", "fp32", seed=1)
    g = ops.add_rms_norm_bwd(p["dout"], p["residual"], p["weight"], p["dres"])
    d, v64, w = n64(p["dout"]), n64(p["residual"]), n64(p["weight"])
    dv, dw = ref.rms_norm_backward(d, v64, w, n64(p["dres"]), 1e-5)
    _, rstd = ref.rms_norm(v64, w, 1e-5)
    ref.check(n64(g["dweight"]), dw, (REL + (rows + 64) * ref.U) * np.abs(d * v64 * rstd).sum(0), "dweight")
    ref.check(n64(g["dx"]), dv, 2.0 ** -7 * np.abs(dv) + 4 * REL * (np.abs(rstd * d * w) + np.abs(v64)), "dx")
    again = ops.add_rms_norm_bwd(p["dout"], p["residual"], p["weight"], p["dres"])
    assert all(torch.equal(g[k], again[k]) for k in g)


def test_norm_and_quantize_in_graphs_and_streams(cuda_ok):
    """Captured training steps, replayed on two streams side by side with workspaces of their
    own, equal the eager calls (dweight's sum starts early there too)."""
    probs = [problem(3000, 768, "bf16", "bf16", seed=1), problem(700, 2560, "bf16", "fp32", seed=2)]

    def step(p):
        out, v = ops.add_rms_norm_fwd(p["x"], p["weight"], p["residual"])
        q, s, _ = ops.add_rms_norm_fp8(p["x"], p["weight"], p["residual"])
        g = ops.add_rms_norm_bwd(p["dout"], v, p["weight"], p["dres"])
        return [out, v, q.view(torch.uint8), s, *g.values(), *[t.view(torch.uint8) for t in ops.fp8_quantize(out)]]

    eager = [step(p) for p in probs]
    graphs, outs = [], []
    for p in probs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(p))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for e, o in zip(eager, outs):
        assert all(torch.equal(a, b) for a, b in zip(e, o))
    del graphs


def test_rms_norm_gradient_against_differences(cuda_ok):
    p = problem(3, 40, "fp32", "fp32", seed=2)
    g = ops.add_rms_norm_bwd(p["dout"], p["residual"], p["weight"], p["dres"])

    def loss(v, w):
        out, _ = ops.add_rms_norm_fwd(v, w)
        return float((out.double() * p["dout"].double()).sum() + (v.double() * p["dres"].double()).sum())

    eps = 2.0 ** -7
    for name, grad in (("residual", "dx"), ("weight", "dweight")):
        e = torch.randn(p[name].shape, generator=torch.Generator().manual_seed(3)).to(DEV)
        args = lambda k: ((p["residual"] + k * e, p["weight"]) if name == "residual"  # noqa: E731
                          else (p["residual"], p["weight"] + k * e))
        diff = (loss(*args(eps)) - loss(*args(-eps))) / (2 * eps)
        want = float((g[grad].double() * e.double()).sum())
        scale = float((g[grad].double() * e.double()).abs().sum())
        # eps^2 / 6 of a third derivative of order |e / v|^3 a term, and 120 outputs off by 4e-6
        assert abs(diff - want) <= 2e-3 * scale + 120 * 4e-6 / eps, (name, diff, want)


def test_rms_norm_zero_rows_and_zero_values(cuda_ok):
    w = torch.ones(64, device=DEV)
    empty = torch.empty(0, 64, device=DEV)
    out, v = ops.add_rms_norm_fwd(empty, w, empty)
    assert out.shape == (0, 64)
    assert float(ops.add_rms_norm_bwd(empty, empty, w)["dweight"].abs().max()) == 0.0
    q, s, _ = ops.add_rms_norm_fp8(torch.zeros(3, 64, device=DEV), w)
    assert float(q.float().abs().max()) == 0.0 and torch.isfinite(s).all() and (s > 0).all()
    x = torch.randn(4, 64, device=DEV)
    x[1, 5] = float("nan")
    out, _ = ops.add_rms_norm_fwd(x, w)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[[0, 2, 3]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 16, 1), (2, 48, 7), (1, 128, 64), (3, 272, 65), (1, 2560, 8),
                                   (2, 144, 200), (1, 5120, 3)], ids=lambda s: "%dx%dx%d" % s)
def test_fp8_quantize(cuda_ok, shape, dtype):
    b, d, L = shape
    g = torch.Generator().manual_seed(d + L)
    x = (torch.randn(b, d, L, generator=g) * torch.exp(2 * torch.randn(b, d, 1, generator=g))).to(TYPES[dtype])
    rows = x.transpose(1, 2).reshape(b * L, d).contiguous()
    q, s = ops.fp8_quantize(x.to(DEV), channel_major=True)
    check_e4m3(q, s, n64(rows), "channel-major")
    q2, s2 = ops.fp8_quantize(rows.to(DEV))
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


def test_fp8_quantize_special_values(cuda_ok):
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1))
    x[0, :128] = 0.0
    x[1, 3] = float("nan")
    x[2, 130] = float("inf")
    x[3, 0] = 1e-38
    q, s = ops.fp8_quantize(x.to(DEV))
    q, s = q.float().cpu(), s.cpu()
    assert (q[0, :128] == 0).all() and s[0, 0] > 0
    assert torch.isnan(q[1, 3]) and torch.isfinite(q[1, :3]).all() and torch.isfinite(s[1]).all()
    assert torch.isinf(s[2, 1]) and torch.isfinite(q[2, :128]).all()
    assert torch.isfinite(q[3]).all()


@pytest.mark.parametrize("shape", [(1, 16), (130, 272), (128, 128), (300, 1040)], ids=lambda s: "%dx%d" % s)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_fp8_quantize_weight(cuda_ok, shape, dtype):
    n, k = shape
    w = torch.randn(n, k, generator=torch.Generator().manual_seed(n)).to(TYPES[dtype])
    q, s = ops.fp8_quantize_weight(w.to(DEV))
    w64 = n64(w)
    for i in range(0, n, 128):
        for j in range(0, k, 128):
            blk = w64[i:i + 128, j:j + 128]
            sc = max(np.abs(blk).max(), 1e-30) / 448
            got_s = float(s[i // 128, j // 128])
            assert abs(got_s - sc) <= 2.0 ** -22 * sc
            got = n64(q[i:i + 128, j:j + 128])
            half = np.maximum(np.abs(got) * 2.0 ** -4, 2.0 ** -10)
            ref.check(got * got_s, blk, half * got_s + 2.0 ** -21 * np.abs(blk), "block")
